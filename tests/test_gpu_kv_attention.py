"""Attention over the paged MXFP4 cache against fp64, at the lengths, masks, pages and
layouts where it can go wrong.

Tolerance, from what the kernel rounds: a weight p to bf16 (relative 2^-8 at most), a
block of a query to 2^-12 of its largest element (three FP6 terms leave at most 2^-13,
times two for the block's absolute sum), scores, exponentials and sums in fp32 (2^-21
relative of the score's absolute sum, 2^-22 a summed key at most), the output to bf16
(2^-8).  `weight` and `spread` of the oracle turn these into absolute bounds per output.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import tabit_oracle as O
import tabit_synth as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


def _problem(seed, lens, qs, hq, hk, D, ps, had, rope="none", slack=0, extra_pages=3, key_gain=1.0):
    """A cache of random codes with ordinary scales in the keys that lie inside the
    sequences; every other byte (tails of pages, free pages) is random garbage, NaN scales
    among it."""
    rng = np.random.default_rng(seed)
    dp = (D + 31) // 32 * 32
    need = [(n + ps - 1) // ps for n in lens]
    P = sum(need) + extra_pages
    arr = {n: rng.integers(0, 256, (P, hk, ps, w), dtype=np.uint8)
           for n, w in (("k_codes", dp // 2), ("k_scales", dp // 32), ("v_codes", dp // 2),
                        ("v_scales", dp // 32))}
    arr["k_scales"][...] = np.where(rng.random(arr["k_scales"].shape) < 0.5, 255, arr["k_scales"])
    arr["v_scales"][...] = np.where(rng.random(arr["v_scales"].shape) < 0.5, 255, arr["v_scales"])
    width = max(need + [1])
    table = np.full((len(lens), width), -1, np.int32)
    perm = rng.permutation(P)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
        for j in range(lens[b]):
            pg, o = table[b, j // ps], j % ps
            k = rng.standard_normal((1, hk, D)).astype(np.float32) * key_gain
            v = rng.standard_normal((1, hk, D)).astype(np.float32)
            kc, ks = B.mx_rows(k, had)
            vc, vs = B.mx_rows(v, had)
            arr["k_codes"][pg, :, o], arr["k_scales"][pg, :, o] = kc[0], ks[0]
            arr["v_codes"][pg, :, o], arr["v_scales"][pg, :, o] = vc[0], vs[0]
    cu = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
    tokens = int(cu[-1])
    wide = torch.from_numpy(rng.standard_normal((tokens, hq * D + slack)).astype(np.float32)).bfloat16()
    q = O.bf16_to_f32(S.bf16_bits(wide)[:, :hq * D]).reshape(tokens, hq, D)
    R = 0 if rope == "none" else D // 16 * 16
    r = None
    if R:
        a = rng.uniform(-50, 50, (23, R // 2))
        r = (np.cos(a).astype(np.float32), np.sin(a).astype(np.float32),
             rng.integers(0, 23, tokens).astype(np.int32), rope == "pairs")
    return dict(arr=arr, table=table, cu=cu, lens=np.array(lens, np.int32), wide=wide, q=q, rope=r,
                D=D, hq=hq, hk=hk, had=had, max_q=max(qs), max_kv=max(lens), ps=ps)


def _on_gpu(p):
    d = lambda x: torch.from_numpy(x).to(DEV)   # noqa: E731
    cache = T.KVCache(*[d(p["arr"][n]) for n in ("k_codes", "k_scales", "v_codes", "v_scales")],
                      head_dim=p["D"], had_block=p["had"])
    q = p["wide"].to(DEV)[:, :p["hq"] * p["D"]].unflatten(1, (p["hq"], p["D"]))
    kw = {}
    if p["rope"]:
        cos, sin, pos, inter = p["rope"]
        kw = dict(rope=T.Rope(d(cos), d(sin), inter), positions=d(pos))
    return cache, q, d(p["cu"]), d(p["table"]), d(p["lens"]), kw


def _run(ctx, p, causal, scale, **over):
    cache, q, cu, table, lens, kw = _on_gpu(p)
    lse = torch.full((q.shape[0], p["hq"]), 7.0, device=DEV)
    kw.update(over)
    max_q, max_kv = kw.pop("max_q", p["max_q"]), kw.pop("max_kv", p["max_kv"])
    out = ctx.kv_attention(cache, q, cu, table, lens, max_q, max_kv, scale=scale, causal=causal, lse=lse, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def _want(p, causal, scale, max_kv=None):
    return B.attention(p["q"].astype(np.float64), p["arr"], p["table"], p["lens"], p["cu"], scale, causal,
                       p["D"], p["had"], p["rope"], max_kv)


def _check(got, want, keys):
    out, lse = got
    ref, rlse, weight, spread = want
    slip = spread[..., None] * (2.0 ** -12 + 2.0 ** -21)         # error of a score
    moved = 2.0 * np.expm1(2 * slip) + 2.0 ** -8 + (keys + 64) * 2.0 ** -22
    assert np.all(np.isfinite(out))
    bad = np.abs(out - ref) > weight * moved + np.abs(ref) * 2.0 ** -8 + 1e-30
    assert not bad.any(), (bad.sum(), np.abs(out - ref).max())
    empty = np.isinf(rlse)
    assert np.array_equal(empty, np.isinf(lse)) and np.all(lse[empty] < 0) and not out[empty].any()
    room = slip[..., 0] * 2 + (keys + 64) * 2.0 ** -22 + np.abs(np.where(empty, 0, rlse)) * 2.0 ** -20
    assert np.all(np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rlse)) <= room)


CASES = [
    # lens, qs, hq, hk, D, page, had, rope, causal
    ([1], [1], 1, 1, 64, 16, 0, "none", True),
    ([0], [1], 4, 2, 64, 16, 32, "none", True),                   # no key at all
    ([17], [1], 8, 1, 128, 16, 32, "half", True),
    ([64, 65, 63], [1, 1, 1], 8, 2, 128, 16, 32, "half", True),
    ([1000, 1, 0, 333], [1, 1, 1, 1], 32, 8, 128, 16, 32, "half", True),
    ([129], [1], 16, 1, 96, 32, 0, "pairs", True),                # 16 heads on one key head
    ([200], [1], 20, 1, 112, 64, 32, "half", True),               # more heads than one row tile
    ([70, 300], [5, 1], 6, 2, 72, 16, 32, "none", False),
    ([150, 40], [33, 40], 4, 4, 64, 64, 32, "pairs", True),
    ([10, 100], [30, 7], 4, 2, 64, 16, 32, "half", True),         # more queries than keys: empty rows
    ([257], [130], 3, 3, 40, 128, 0, "half", True),
    ([31, 300, 128], [64, 129, 1], 2, 2, 80, 16, 32, "none", False),
    ([48], [17], 2, 1, 32, 16, 32, "pairs", False),
    ([48], [3], 2, 1, 8, 16, 32, "none", True),
    ([700], [200], 4, 1, 128, 32, 32, "half", True),
    ([90, 64], [0, 70], 2, 1, 64, 16, 32, "none", False),         # a sequence without queries
    ([2100], [2], 4, 2, 64, 16, 0, "none", False),                # split over workgroups
]


@pytest.mark.parametrize("lens,qs,hq,hk,D,ps,had,rope,causal", CASES)
def test_attention(ctx, lens, qs, hq, hk, D, ps, had, rope, causal):
    print(f"attention lens {lens} qs {qs} heads {hq}/{hk} D {D} page {ps} had {had} {rope}", flush=True)
    p = _problem(len(lens) + D, lens, qs, hq, hk, D, ps, had, rope, slack=8 * (D // 40))
    scale = D ** -0.5
    _check(_run(ctx, p, causal, scale), _want(p, causal, scale), max(lens))


def test_scores_far_apart(ctx):
    """Scores of some hundreds: one key takes nearly all the weight, running maxima jump."""
    for qs in ([1, 1], [40, 20]):
        p = _problem(5, [500, 129], qs, 4, 2, 64, 16, 32, "half", key_gain=40.0)
        _check(_run(ctx, p, True, 0.125), _want(p, True, 0.125), 500)
    p = _problem(6, [200], [50], 2, 2, 128, 16, 0)
    _check(_run(ctx, p, False, -0.3), _want(p, False, -0.3), 200)     # a negative scale
    _check(_run(ctx, p, False, 0.0), _want(p, False, 0.0), 200)       # plain means


def test_pages_outside_the_cache_are_not_seen(ctx):
    for qs in ([1, 1], [20, 50]):
        p = _problem(7, [300, 100], qs, 4, 2, 64, 16, 32)
        p["table"][0, 3], p["table"][0, 7], p["table"][1, 0] = -1, p["arr"]["k_codes"].shape[0], 2 ** 30
        _check(_run(ctx, p, True, 0.125), _want(p, True, 0.125), 300)


def test_lengths_are_cut_at_max_kv(ctx):
    for qs in ([1], [40]):
        p = _problem(8, [200], qs, 4, 2, 64, 16, 0)
        _check(_run(ctx, p, False, 0.125, max_kv=100), _want(p, False, 0.125, max_kv=100), 100)


def test_not_a_number_reaches_only_the_rows_that_see_it(ctx):
    """A poisoned token in the middle of a causal chunk, a query row that is not finite, a
    query position outside the tables."""
    for n, hk, D in ((40, 2, 64), (6, 1, 128), (150, 2, 96)):
        p = _problem(9, [n + 30], [n], 4, hk, D, 16, 32, "half")
        j = 30 + n // 2
        pg, o = p["table"][0, j // 16], j % 16
        p["arr"]["k_scales"][pg, 0, o], p["arr"]["v_codes"][pg, 0, o] = 255, 0
        p["arr"]["v_scales"][pg, 0, o] = 127
        cache, q, cu, table, lens, kw = _on_gpu(p)
        q[1, 3, 7] = float("inf")
        kw["positions"][0] = 23
        out = ctx.kv_attention(cache, q, cu, table, lens, n, n + 30, causal=True, **kw)
        nan = torch.isnan(out).all(-1).cpu().numpy()
        some = torch.isnan(out).any(-1).cpu().numpy()
        want = np.zeros((n, 4), bool)
        want[n // 2:, :4 // hk] = True      # heads of key head 0, from the token on
        want[0], want[1, 3] = True, True
        assert np.array_equal(nan, want) and np.array_equal(some, want), (n, D)


@pytest.mark.parametrize("n,hk,D", [(4, 1, 128), (8, 2, 64), (40, 2, 64), (150, 2, 96), (3, 1, 32), (64, 4, 128)])
def test_value_scales_beyond_bf16(ctx, n, hk, D):
    """A key whose value scale is NaN (255) or too large for bf16 (253, 254): rows that see it
    answer NaN, rows that do not are as without it."""
    for byte in (253, 255):
        p = _problem(12, [n + 30], [n], 4, hk, D, 16, 32)
        cache, q, cu, table, lens, kw = _on_gpu(p)
        a = ctx.kv_attention(cache, q, cu, table, lens, n, n + 30, causal=True)
        j = 30 + n // 2
        cache.v_scales[int(p["table"][0, j // 16]), hk - 1, j % 16, D // 32 - 1] = byte
        b = ctx.kv_attention(cache, q, cu, table, lens, n, n + 30, causal=True)
        sees = torch.zeros((n, 4), dtype=torch.bool, device=DEV)
        sees[n // 2:, 4 // hk * (hk - 1):] = True
        assert torch.isnan(b[sees]).all() and torch.equal(a[~sees], b[~sees]), (byte, n, D)


@pytest.mark.parametrize("n,hq,hk,D", [(4, 4, 1, 128), (16, 2, 2, 64), (17, 2, 2, 64), (2, 17, 1, 96),
                                       (1, 16, 1, 40), (1, 17, 1, 40), (31, 8, 2, 72)])
@pytest.mark.parametrize("keys", [5, 64, 700])
def test_around_sixteen_rows_a_key_head(ctx, n, hq, hk, D, keys):
    """Both sides of the change of kernel, with as few keys as queries and many."""
    print("attention rows", n * hq // hk, "keys", keys, flush=True)
    p = _problem(n + keys, [keys, 1], [n, 1], hq, hk, D, 16, 32, "half")
    _check(_run(ctx, p, True, D ** -0.5), _want(p, True, D ** -0.5), keys)


def test_ranges_of_many_tiles(ctx):
    """A workgroup that passes more tiles than it places at once, some of their pages missing:
    512 key heads, so that the 4500 keys stay one range; three heads against fp64."""
    rng = np.random.default_rng(21)
    n, hk, D, ps, keys = 20, 512, 16, 16, 4500
    pages = (keys + ps - 1) // ps
    arr = {"k_codes": rng.integers(0, 256, (pages, hk, ps, 16), dtype=np.uint8),
           "v_codes": rng.integers(0, 256, (pages, hk, ps, 16), dtype=np.uint8),
           "k_scales": rng.integers(122, 126, (pages, hk, ps, 1), dtype=np.uint8),
           "v_scales": rng.integers(124, 128, (pages, hk, ps, 1), dtype=np.uint8)}
    for name in ("k_codes", "v_codes"):
        arr[name][..., D // 2:] = 0            # past the head's elements
    table = rng.permutation(pages).astype(np.int32)[None]
    table[0, [70, 256, 270]] = -1, pages, -5
    wide = torch.from_numpy(rng.standard_normal((n, hk * D)).astype(np.float32)).bfloat16()
    p = dict(arr=arr, table=table, cu=np.array([0, n], np.int32), lens=np.array([keys], np.int32), wide=wide,
             rope=None, D=D, hq=hk, hk=hk, had=0, max_q=n, max_kv=keys, ps=ps)
    out, lse = _run(ctx, p, True, 0.25)
    pick = [0, 255, 511]
    part = dict(p, arr={k: np.ascontiguousarray(v[:, pick]) for k, v in arr.items()},
                q=O.bf16_to_f32(S.bf16_bits(wide)).reshape(n, hk, D)[:, pick])
    _check((out[:, pick], lse[:, pick]), _want(part, True, 0.25), keys)


def test_reference_rises_late(ctx):
    """Scores near nothing for the first tiles, then one of hundreds: what was summed so far has
    to be scaled away, in the tile where the reference rises and in the join of the ranges."""
    for n, D in ((1, 64), (3, 128), (70, 64), (130, 96)):
        p = _problem(13, [900], [n], 2, 1, D, 16, 0)
        for j, x in ((500, 127 + 6), (700, 127 + 8)):
            p["arr"]["k_scales"][p["table"][0, j // 16], :, j % 16] = x
        _check(_run(ctx, p, False, 0.5), _want(p, False, 0.5), 900)


def test_same_bits_every_time_and_other_streams(ctx):
    for qs in ([1, 1], [100, 30]):
        p = _problem(10, [900, 400], qs, 8, 2, 128, 16, 32, "half")
        a, b = _run(ctx, p, True, 0.1), _run(ctx, p, True, 0.1)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c = _run(ctx, p, True, 0.1)
        assert np.array_equal(a[0], c[0])


def test_rows_of_no_sequence_stay(ctx):
    p = _problem(11, [40, 50], [3, 2], 4, 2, 64, 16, 0)
    cache, q, cu, table, lens, kw = _on_gpu(p)
    cu = torch.tensor([1, 2, 4], dtype=torch.int32, device=DEV)     # rows 0 and 4 are nobody's
    out = torch.full((5, 4, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    ctx.kv_attention(cache, q, cu, table, lens, 3, 50, out=out)
    assert bool((out[0] == 9).all()) and bool((out[4] == 9).all()) and not bool((out[1:4] == 9).any())
    full = out.clone()
    out.fill_(9.0)          # rows past max_q are not computed
    ctx.kv_attention(cache, q, cu, table, lens, 1, 50, out=out)
    assert torch.equal(out[2], full[2]) and bool((out[3] == 9).all())


def test_long_cache_past_4_gib(ctx):
    """Pages whose byte offset passes 32 bits, in a split call and in a chunk of queries."""
    heads, D, ps = 8, 128, 64
    pages = (5 << 30) // (heads * ps * (D // 2))
    cache = T.KVCache(*[torch.empty((pages, heads, ps, w), dtype=torch.uint8, device=DEV)
                        for w in (D // 2, D // 32, D // 2, D // 32)], head_dim=D, had_block=32)
    small = T.KVCache.empty(40, ps, heads, D, 32, DEV)
    g = torch.Generator().manual_seed(2)
    n = 40 * ps - 5
    k, v = (torch.randn(n, heads, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    far = (pages - 1 - torch.arange(40)).int()
    ctx.kv_append(small, k, v, torch.arange(n, device=DEV))
    slots = far.long().to(DEV)[torch.arange(n, device=DEV) // ps] * ps + torch.arange(n, device=DEV) % ps
    ctx.kv_append(cache, k, v, slots)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    for rows in (1, 70):
        q = torch.randn(rows, 16, D, generator=g).bfloat16().to(DEV)
        cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        a = ctx.kv_attention(small, q, cu, torch.arange(40, dtype=torch.int32, device=DEV)[None], lens, rows, n, causal=True)
        b = ctx.kv_attention(cache, q, cu, far.to(DEV)[None], lens, rows, n, causal=True)
        assert torch.equal(a, b)


def test_graph_replays_match_eager(ctx):
    """Append and attention captured together, replayed on new inputs."""
    heads, D = 2, 64
    cache = T.KVCache.empty(8, 16, heads, D, 32, DEV)
    cos = torch.randn(128, 32, device=DEV).cos()
    rope = T.Rope(cos, (1 - cos * cos).sqrt(), True)
    k, v = (torch.zeros(2, heads, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros(2, 4, D, dtype=torch.bfloat16, device=DEV)
    slots = torch.zeros(2, dtype=torch.int64, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    out = torch.zeros_like(q)
    ws = ctx.kv_attention_workspace(cache, q, 2, 1, 64)

    def step():
        ctx.kv_append(cache, k, v, slots, rope=rope, positions=pos)
        ctx.kv_attention(cache, q, cu, table, lens, 1, 64, causal=True, rope=rope, positions=pos, out=out, ws=ws)

    def load(i):
        g = torch.Generator().manual_seed(i)
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())
        slots.copy_(torch.tensor([i, 64 + i]))
        pos.fill_(i)
        lens.fill_(i + 1)

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = []
    for i in range(20):
        load(i)
        step()
        torch.cuda.synchronize()
        want.append(out.clone())
    for t in (cache.k_codes, cache.v_codes):
        t.zero_()
    for i in range(20):
        load(i)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i


def test_binding_refusals(ctx):
    p = _problem(12, [20], [2], 4, 2, 64, 16, 0)
    cache, q, cu, table, lens, kw = _on_gpu(p)
    with pytest.raises(TypeError):
        ctx.kv_attention(cache, q.float(), cu, table, lens, 2, 20)
    with pytest.raises(TypeError):
        ctx.kv_attention(cache, q, cu.long(), table, lens, 2, 20)
    with pytest.raises(ValueError):
        ctx.kv_attention(cache, q, cu[:1], table, lens, 2, 20)
    with pytest.raises(ValueError):
        ctx.kv_attention(cache, q[:, :, :32], cu, table, lens, 2, 20)
    with pytest.raises(T.TabitError) as e:
        ctx.kv_attention(cache, q, cu, table, lens, 2, 33)      # two pages hold 32 tokens
    assert e.value.status == T.ESHAPE
    assert ctx.kv_attention(cache, q[:0], cu, table, lens, 2, 20).shape == (0, 4, 64)
