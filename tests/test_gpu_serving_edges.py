"""Operators for serving many requests where the ordinary problems do not reach."""
import numpy as np
import pytest
import torch

from tests import attention_check as A
from tests import serve_check as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


# ------------------------------------------------------------------ trees
def _tree(ctx, p, see):
    words = max((int(np.diff(p["cu"]).max()) + 63) // 64, 1)
    mask = np.concatenate([S.packed(m, words) for m in see])
    q = S.dev(p["q"]).bfloat16()
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = ctx.kv_tree_attention(S.cache_of(p), q, S.dev(mask), S.dev(np.asarray(p["cu"], np.int32)), S.dev(p["table"]),
                                S.dev(np.asarray(p["lens"], np.int32)), int(np.diff(p["cu"]).max()), max(p["lens"]),
                                scale=p["scale"], lse=lse)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("rows,n", [(8, 30), (16, 200), (30, 60), (32, 300), (40, 60), (150, 400), (700, 800)])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_far_values_of_other_branches(ctx, rows, n, D):
    """Two branches whose nodes lie among each other: a far value of one leaves the other's rows their bits,
    whether those see far values of their own or not."""
    print("tree", rows, n, D, flush=True)
    rng = np.random.default_rng(rows + D)
    branch = rng.integers(0, 2, rows)
    branch[:2] = 0, 1
    see = (branch[:, None] == branch[None]) & np.tril(np.ones((rows, rows), bool))
    p = A.steep_problem(rows, n, rows, 2, D, 32, lambda _, shape: np.full(shape, 127))
    scales = p["arr"]["v_scales"]

    def far(nodes, b):
        j = n - rows + np.asarray(nodes)
        scales[p["table"][0, j // 16], :, j % 16, 1] = b

    ones, zeros = np.flatnonzero(branch == 1), np.flatnonzero(branch == 0)
    for own, others in ((0, 240), (0, 20), (240, 20), (20, 240), (240, 240)):
        scales[...] = 127
        if own:
            far(rng.permutation(ones)[:max(len(ones) // 30, 1)], own)
        clean = _tree(ctx, p, [see])
        far(rng.permutation(zeros)[:max(len(zeros) // 20, 1)], others)
        got = _tree(ctx, p, [see])
        A.check(*got, S.tree_want(p, [see]))
        assert np.array_equal(got[0][ones], clean[0][ones]) and np.array_equal(got[1][ones], clean[1][ones]), (own, others)


@pytest.mark.parametrize("rows", [8, 30, 150])
@pytest.mark.parametrize("byte", [253, 255])
def test_values_that_are_no_number_in_other_branches(ctx, rows, byte):
    """A node whose value is none makes NaN of the rows that see it and leaves the others their bits."""
    p = A.problem(rows, [300], [rows], 2, 2, 128, 16, 32)
    rng = np.random.default_rng(rows)
    branch = rng.integers(0, 2, rows)
    see = (branch[:, None] == branch[None]) & np.tril(np.ones((rows, rows), bool))
    clean = _tree(ctx, p, [see])
    node = rows // 2
    j = 300 - rows + node
    p["arr"]["v_scales"][p["table"][0][j // 16], :, j % 16, 2] = byte
    got = _tree(ctx, p, [see])
    touched = see[:, node]
    assert np.isnan(got[0][touched]).all() and touched.any() and not touched.all()
    assert np.array_equal(got[0][~touched], clean[0][~touched]) and np.array_equal(got[1][~touched], clean[1][~touched])


# ------------------------------------------------------------------ adapters
def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16().to(DEV)


@pytest.mark.parametrize("rows", [1, 5, 200])
def test_columns_of_one_matrix(ctx, rows):
    """x, y and out beside each other in one matrix: the bits of separate ones, and nothing else is written."""
    rng = np.random.default_rng(rows)
    K, N = 64, 96
    whole = _bf(rng, rows, 8 + N + K + N)
    x, y = whole[:, 8 + N:8 + N + K], whole[:, 8 + N + K:]
    bank = T.Adapters(_bf(rng, 2, 16, K, scale=0.1), _bf(rng, 2, N, 16))
    cu, which = S.dev(np.array([0, rows // 2, rows], np.int32)), S.dev(np.array([1, 0], np.int32))
    want = ctx.adapter_linear(bank, x.contiguous(), y.contiguous(), cu, which)
    before = whole.clone()
    ctx.adapter_linear(bank, x, y, cu, which, out=whole[:, 8:8 + N])
    assert torch.equal(whole[:, 8:8 + N], want)
    assert torch.equal(whole[:, :8], before[:, :8]) and torch.equal(whole[:, 8 + N:], before[:, 8 + N:])
    with pytest.raises(T.TabitError):
        ctx.adapter_linear(bank, x, y, cu, which, out=whole[:, 16:16 + N])


def test_masks_of_more_words_than_any_tree_has(ctx):
    """Rows of more than 2^25 words, whose bits pass 32 bits: the node itself and its parent, then zeros."""
    words = (1 << 25) + 1
    mask = torch.full((2, words), -1, dtype=torch.int64, device=DEV)
    parents, cu = S.dev(np.array([-1, 0], np.int32)), S.dev(np.array([0, 2], np.int32))
    depth = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    assert T.load().tabit_tree_mask(ctx.handle, parents.data_ptr(), 2, cu.data_ptr(), 1, 2, mask.data_ptr(), words, depth.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream) == T.OK
    torch.cuda.synchronize()
    assert mask[:, 0].tolist() == [1, 3] and depth.tolist() == [0, 1]
    assert not mask[:, 1:].any()


SHAPES = {                 # rows, segments, rank: one kernel for both products, two for single tokens, two of larger tiles
    "one kernel, rank 16": (20, 5, 16), "one kernel, rank 32": (9, 9, 32), "two kernels, few rows": (40, 8, 64),
    "two kernels, rank 128": (200, 1, 128), "two kernels, rank 16": (150, 2, 16),
}


def _product(rng, shape, fmt, K=96, N=1184):
    rows, segments, rank = SHAPES[shape]
    cu = np.linspace(0, rows, segments + 1).astype(np.int32)
    which = rng.integers(0, 3, segments).astype(np.int32)
    bank = T.Adapters(_bf(rng, 3, rank, K, scale=0.1), _bf(rng, 3, N, rank))
    if fmt == "bf16":
        x, xs = _bf(rng, rows, K), None
    elif fmt == "int8":
        x, xs = S.dev(rng.integers(-127, 128, (rows, K)).astype(np.int8)), S.dev(rng.uniform(0.001, 0.1, rows).astype(np.float32))
    else:
        x, xs = S.dev(rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)), S.dev(rng.integers(120, 128, (rows, K // 32), dtype=np.uint8))
    return bank, x, xs, _bf(rng, rows, N), S.dev(cu), S.dev(which)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "mxfp4"])
def test_rows_that_are_no_number(ctx, shape, fmt):
    """They make NaN of themselves alone, wherever in a tile of rows they lie."""
    rng = np.random.default_rng(len(shape))
    bank, x, xs, y, cu, which = _product(rng, shape, fmt)
    clean = ctx.adapter_linear(bank, x, y, cu, which, x_scale=xs)
    bad = rng.permutation(len(y))[:2]
    for t in bad:
        if fmt == "bf16":
            x[t, 90] = float("nan")
        elif fmt == "int8":
            xs[t] = float("nan")
        else:
            xs[t, 2] = 255
    out = ctx.adapter_linear(bank, x, y, cu, which, x_scale=xs)
    rest = torch.ones(len(y), dtype=torch.bool, device=DEV)
    rest[S.dev(bad)] = False
    assert out[~rest].isnan().all() and torch.equal(out[rest], clean[rest]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "mxfp4"])
def test_products_captured(ctx, shape, fmt):
    """Replays in place, with eager calls on the same workspace in between."""
    rng = np.random.default_rng(len(shape) + 1)
    bank, x, xs, y, cu, which = _product(rng, shape, fmt)
    want = ctx.adapter_linear(bank, x, y, cu, which, x_scale=xs)
    ws, out = ctx.adapter_workspace(bank, x, len(which)), y.clone()

    def call():
        ctx.adapter_linear(bank, x, out, cu, which, x_scale=xs, out=out, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.copy_(y)
        ws.fill_(255)
        g.replay()
        eager = ctx.adapter_linear(bank, x, y, cu, which, x_scale=xs, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)


@pytest.mark.parametrize("rows", [1, 30, 300])
def test_no_adapters_at_all(ctx, rows):
    """A bank of none: out = y."""
    rng = np.random.default_rng(rows)
    bank = T.Adapters(_bf(rng, 0, 16, 64), _bf(rng, 0, 96, 16))
    x, y = _bf(rng, rows, 64), _bf(rng, rows, 96)
    cu, which = S.dev(np.array([0, rows], np.int32)), S.dev(np.array([0], np.int32))
    assert torch.equal(ctx.adapter_linear(bank, x, y, cu, which), y)


# ------------------------------------------------------------------ another stream, moves of one list twice
def test_calls_on_another_stream(ctx):
    """Every operator on a side stream, while the default one works: the bits of calls by themselves."""
    p = A.problem(31, [2500, 90], [20, 8], 8, 2, 64, 16, 32)
    rng = np.random.default_rng(31)
    q = S.dev(np.asarray(p["q"], np.float32)).bfloat16()
    cu, table, lens = S.dev(np.asarray(p["cu"], np.int32)), S.dev(p["table"]), S.dev(np.array(p["lens"], np.int32))
    parents = S.dev(np.concatenate([S.random_parents(rng, n) for n in (20, 8)]))
    bank, x, y = T.Adapters(_bf(rng, 2, 16, 64), _bf(rng, 2, 96, 16)), _bf(rng, 28, 64), _bf(rng, 28, 96)
    which = S.dev(np.array([0, 1], np.int32))

    def run():
        cache = S.cache_of(p)
        mask, depth = ctx.tree_mask(parents, cu, 20)
        o = ctx.kv_tree_attention(cache, q, mask, cu, table, lens, 20, 2500)
        sums = ctx.kv_weigh(cache, ctx.kv_sums(cache), q, cu, table, lens, 20, 2500)
        weights = sums.clone()
        keep, new = ctx.kv_evict(cache, sums, table, lens, 2500, 64, sinks=2, recent=20)
        ctx.kv_compact(cache, table, keep, new, sums=sums)
        z = ctx.adapter_linear(bank, x, y, cu, which)
        return [mask, depth, o, weights, keep, new, sums, cache.k_codes, cache.v_scales, z]

    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    work = torch.randn(4096, 4096, device=DEV)
    for _ in range(4):
        work = work @ work * 1e-3
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


def test_a_token_named_twice(ctx):
    """A list that names a token twice puts it in both places; a head's list of one token many times as well."""
    rng = np.random.default_rng(5)
    arr = [rng.integers(0, 256, (80, 2, 16, w), dtype=np.uint8) for w in (32, 2, 32, 2)]
    table = rng.permutation(80).astype(np.int32)[None]
    for most in (12, 1100):
        keep = np.sort(rng.integers(most, 1280, (1, 2, most)), axis=2).astype(np.int32)
        keep[0, 1, most // 2:] = keep[0, 1, -1]
        cache = T.KVCache(*[S.dev(a) for a in arr], head_dim=64)
        ctx.kv_compact(cache, S.dev(table), S.dev(keep), S.dev(np.array([most], np.int32)))
        want = S.compact_want(arr, table, keep, np.array([most]))
        for n, w in zip(("k_codes", "k_scales", "v_codes", "v_scales"), want):
            assert np.array_equal(getattr(cache, n).cpu().numpy(), w), n


# ------------------------------------------------------------------ nothing there
@pytest.mark.parametrize("rows", [1, 2, 40])
@pytest.mark.parametrize("most", [0, 50, 2000])
def test_caches_without_pages_or_keys(ctx, rows, most):
    """Rows that have no key answer zeros and -infinity, whether there are no lengths or no pages; nothing is kept
    wrongly or written."""
    rng = np.random.default_rng(rows)
    cache = T.KVCache.empty(0 if most else 4, 16, 2, 64, 32, DEV)
    q = _bf(rng, 2 * rows, 8, 64)
    cu, lens = S.dev(np.array([0, rows, 2 * rows], np.int32)), S.dev(np.array([most, most // 2], np.int32))
    table = torch.full((2, 128), 3 if not most else 0, dtype=torch.int32, device=DEV)
    mask, _ = ctx.tree_mask(torch.full((2 * rows,), -1, dtype=torch.int32, device=DEV), cu, rows)
    lse = torch.full((2 * rows, 8), 7.0, device=DEV)
    out = ctx.kv_tree_attention(cache, q, mask, cu, table, lens, rows, most, lse=lse)
    assert not out.any() and lse.isneginf().all()
    for causal in (True, False):
        lse.fill_(7.0)
        sums = torch.full((cache.num_pages, 2, 16), 5.0, device=DEV)
        ctx.kv_weigh(cache, sums, q, cu, table, lens, rows, most, causal=causal, lse=lse)
        assert (sums == 5).all() and lse.isneginf().all()
    keep, new = ctx.kv_evict(cache, sums, table, lens, most, 20, sinks=2, recent=3)
    # (to the reference: one page, and tables that name another)
    want, wnew = S.evict_want(np.zeros((1, 2, 16), np.float32), np.full((2, 128), 9), lens.tolist(), 20, 2, 3)
    assert np.array_equal(keep.cpu().numpy(), want) and np.array_equal(new.cpu().numpy(), wnew)
    ctx.kv_compact(cache, table, keep, new, sums=sums)
    assert (sums == 5).all()
