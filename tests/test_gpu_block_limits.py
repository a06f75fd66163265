"""The cache, the attention and the norms at the far ends of what their entry points accept:
counts near 2^31, grids past 2^32 threads, bounds far beyond the lengths."""
import numpy as np
import pytest
import torch

from tests import attention_check as A
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


@pytest.fixture
def room():
    """room(gib): skips where the card has less free memory; all of it is given back after."""
    def need(gib):
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < gib << 30:
            pytest.skip(f"needs {gib} GiB of free device memory")
    yield need
    torch.cuda.empty_cache()


def test_append_and_read_of_more_tokens_than_seven_pieces(ctx, room):
    """One head of 64 elements or less goes in pieces of 2^28 tokens: the eighth begins at 7 * 2^28
    and its end is past 2^31."""
    room(100)
    n, D = 7 * (1 << 28) + 37, 8
    print("append", n, "tokens", flush=True)
    cache = T.KVCache.empty(1, 16, 1, D, 0, DEV)
    x = torch.zeros((n, 1, D), dtype=torch.bfloat16, device=DEV)
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    at = [0, (1 << 28) - 1, 1 << 28, 7 * (1 << 28) - 1, 7 * (1 << 28), n - 1]
    vals = torch.tensor([1.0, -2.0, 0.5, 3.0, 6.0, -1.5], dtype=torch.bfloat16, device=DEV)
    for i, t in enumerate(at):
        x[t], slots[t] = vals[i], 2 * i
    ctx.kv_append(cache, x, x, slots)
    rk, rv = ctx.kv_read(cache, torch.arange(16, device=DEV))
    want = torch.zeros(16, dtype=torch.bfloat16, device=DEV)
    want[0:12:2] = vals
    assert torch.equal(rk, want[:, None, None].expand(16, 1, D)) and torch.equal(rk, rv)
    print("read", n, "tokens", flush=True)
    v = torch.ones_like(x)
    x.fill_(1.0)
    ctx.kv_read(cache, slots, k=x, v=v)
    for i, t in enumerate(at):
        for r in (x, v):
            assert bool((r[t] == vals[i]).all()), t
            r[t] = 0
    for r in (x, v):                       # slots outside the cache: zeros, up to the last token
        for part in r.view(-1).split(1 << 30):
            assert not bool(part.any())


@pytest.mark.parametrize("rows,width", [((1 << 31) - 5, 32), ((1 << 22) + 3, 16384)])
def test_norm_of_rows_past_the_counts_of_one_launch(ctx, room, rows, width):
    """Rows whose share, rounded up, passes 2^31 rows; rows of a workgroup each past 2^32 threads."""
    room(132)
    print("block_norm", rows, width, flush=True)
    x = torch.ones((rows, width), dtype=torch.bfloat16, device=DEV)
    for r in (0, rows // 2, rows - 1):
        x[r] = 3.0
    ctx.block_norm(x, x_out=x, res_scale=2.0, want_h=False)
    for r in (0, rows // 2, rows - 1):
        assert bool((x[r] == 6).all()), r
        x[r] = 2.0
    step = (1 << 31) // width
    for part in x.split(step):
        assert not bool(part.ne(2.0).any())


def _one_page(heads, D, seed, pages=1, page=16):
    """A full cache of ordinary codes and scales."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dp = (D + 31) // 32 * 32
    codes = [torch.randint(0, 256, (pages, heads, page, dp // 2), generator=g, device=DEV).byte() for _ in range(2)]
    for c in codes:
        c[..., D // 2:] = 0
    scales = [torch.randint(124, 128, (pages, heads, page, dp // 32), generator=g, device=DEV).byte() for _ in range(2)]
    return T.KVCache(codes[0], scales[0], codes[1], scales[1], head_dim=D)


def test_attention_of_more_workgroups_than_one_launch(ctx):
    """65535 sequences x 257 heads of 17 rows are more than 2^32 threads; rows in three of them."""
    seqs, heads, D, n = 65535, 257, 8, 17
    print("attention", seqs, "sequences", heads, "heads", flush=True)
    cache = _one_page(heads, D, 1)
    some = [0, 40000, seqs - 1]
    rows = torch.zeros(seqs + 1, dtype=torch.int32)
    rows[[i + 1 for i in some]] = n
    q = torch.randn(n * len(some), heads, D, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    lens = torch.full((seqs,), 16, dtype=torch.int32)
    lens[some[1]] = 5
    table = torch.zeros((seqs, 1), dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 9.0)
    ctx.kv_attention(cache, q, rows.cumsum(0).int().to(DEV), table, lens.to(DEV), n, 16, out=out)
    cu = torch.arange(0, n * len(some) + 1, n, dtype=torch.int32, device=DEV)
    want = ctx.kv_attention(cache, q, cu, table[:3].contiguous(), lens[some].to(DEV), n, 16)
    assert torch.equal(out, want) and not bool((out == 9).any())


@pytest.mark.parametrize("rows", [1, 16, 17, 140])
@pytest.mark.parametrize("most", [(1 << 31) - 1, (1 << 31) - 63, (1 << 31) - 64, 1 << 30])
def test_a_bound_far_beyond_the_lengths(ctx, rows, most):
    """max_kv near 2^31 (a table of 2048 pages of 2^20 holds it) with some keys: all are seen."""
    D, ps = 8, 1 << 20
    rng = np.random.default_rng(3)
    cache = _one_page(1, D, 5, page=ps)
    cache.v_scales[:, :, 30000:] = 129            # later values are larger, and none is negative:
    cache.v_codes.bitwise_and_(0x77)              # what is left out shows
    for n in (1, 64, 40000):
        print("attention", rows, "rows", n, "keys, bound", most, flush=True)
        q = A.whole_queries(rng, rows, 1, D)
        arr = {x: getattr(cache, x)[:, :, :n].contiguous().cpu().numpy()
               for x in ("k_codes", "k_scales", "v_codes", "v_scales")}
        scale = A.exact_scale(3, 0)
        w = A.want(q, arr, np.zeros((1, 1), int), [n], [0, rows], scale, False, D, 0)
        lse = torch.empty(rows, 1, device=DEV)
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)      # noqa: E731
        out = ctx.kv_attention(cache, torch.from_numpy(q).bfloat16().to(DEV), i32(0, rows),
                               torch.zeros((1, 2048), dtype=torch.int32, device=DEV), i32(n), rows, most,
                               scale=scale, lse=lse)
        A.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), w)


@pytest.mark.parametrize("rows", [1, 17])
def test_as_many_keys_as_an_int_counts(ctx, rows):
    """2^31 - 1 keys: one page of 2^20 keys 2048 times (but for the last), so the softmax is that of
    the page, and the sum 2048 times its."""
    D, ps, n = 8, 1 << 20, (1 << 31) - 1
    print("attention", rows, "rows", n, "keys", flush=True)
    rng = np.random.default_rng(4)
    cache = _one_page(1, D, 6, page=ps)
    cache.v_scales[:, :, ps // 2:] = 129
    cache.v_codes.bitwise_and_(0x77)
    q = A.whole_queries(rng, rows, 1, D)
    arr = {x: getattr(cache, x).cpu().numpy() for x in ("k_codes", "k_scales", "v_codes", "v_scales")}
    scale = A.exact_scale(3, 0)
    ref, rlse, room, lroom = A.want(q, arr, np.zeros((1, 1), int), [ps], [0, rows], scale, False, D, 0)
    lse = torch.empty(rows, 1, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)      # noqa: E731
    out = ctx.kv_attention(cache, torch.from_numpy(q).bfloat16().to(DEV), i32(0, rows),
                           torch.zeros((1, 2048), dtype=torch.int32, device=DEV), i32(n), rows, n,
                           scale=scale, lse=lse)
    # the page's room has 2^-22 for each of its 2^20 keys: a quarter.  A lane's sum has at most 2^19
    # tiles of a rounding of 2^-24; a sum of values has some roundings a tile of either sign.  A lost
    # half of the keys moves lse by log 2
    assert A.outside(out.double().cpu().numpy(), ref, room) == 0.0
    assert A.outside(lse.double().cpu().numpy(), rlse + np.log(2048.0), lroom) == 0.0
    assert bool((np.abs(ref[..., :D]) > room).all())       # zeros would not pass
