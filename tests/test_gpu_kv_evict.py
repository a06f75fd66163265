"""Eviction from the paged cache: accumulated attention weights against 64 bits, the kept lists and
the moves exactly."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
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


def _weigh(ctx, p, sums, causal, rope=None, positions=None, max_q=None, max_kv=None):
    cache = S.cache_of(p)
    q = S.dev(np.asarray(p["q"], np.float32)).bfloat16()
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    got = S.dev(sums.astype(np.float32))
    kw = {}
    if rope is not None:
        kw = dict(rope=T.Rope(S.dev(rope[0]), S.dev(rope[1]), rope[2]), positions=S.dev(positions))
    ctx.kv_weigh(cache, got, q, S.dev(np.asarray(p["cu"], np.int32)), S.dev(p["table"]),
                 S.dev(np.asarray(p["lens"], np.int32)), max_q or int(np.diff(p["cu"]).max()),
                 max(p["lens"]) if max_kv is None else max_kv, scale=p["scale"], causal=causal, lse=lse, **kw)
    return got.double().cpu().numpy(), lse.double().cpu().numpy()


def _near(got, want, room):
    assert np.isfinite(got).all()
    off = np.abs(got - want)
    assert (off <= room).all(), (off.max(), np.argwhere(off > room)[:5])


def _random(seed, lens, qs, hq, hk, D, ps, had):
    """Keys of a normal distribution and bf16 queries of one."""
    p = A.problem(seed, lens, qs, hq, hk, D, ps, had)
    rng = np.random.default_rng(seed + 1)
    q = torch.from_numpy(rng.standard_normal(p["q"].shape).astype(np.float32)).bfloat16().float().numpy()
    return dict(p, q=q, scale=float(np.float32(D ** -0.5))), rng


@pytest.mark.parametrize("lens,qs,hq,hk,D,ps", [
    ([1], [1], 1, 1, 64, 16), ([9], [1], 4, 1, 128, 16), ([300, 77], [1, 1], 8, 2, 64, 16),
    ([64, 65, 63, 128], [16, 1, 7, 64], 4, 2, 40, 16), ([130], [65], 2, 1, 72, 32), ([1000], [1], 32, 8, 128, 16),
    ([700, 200, 90], [63, 90, 33], 8, 4, 96, 64), ([513], [130], 4, 4, 32, 128), ([2500, 40], [12, 40], 12, 2, 112, 16),
    ([5000], [1], 4, 1, 128, 64), ([4100], [3], 2, 2, 8, 16), ([260], [260], 3, 3, 80, 16), ([700], [300], 16, 1, 64, 16),
])
@pytest.mark.parametrize("had", [0, 32])
@pytest.mark.parametrize("causal", [True, False])
def test_weights_against_64_bits(ctx, lens, qs, hq, hk, D, ps, had, causal):
    print("weigh", lens, qs, hq, hk, D, ps, had, causal, flush=True)
    p, rng = _random(sum(lens) + D, lens, qs, hq, hk, D, ps, had)
    shape = p["arr"]["k_codes"].shape[:3]
    sums = rng.random(shape).astype(np.float32)
    want, room, lse = S.weigh_want(p, sums, causal)
    got, glse = _weigh(ctx, p, sums, causal)
    _near(got, want, room)
    # typical errors: a query's terms leave 2^-21 / sqrt(3) of a block's largest element (2.5 of its rms),
    # 7e-7 of a weight; the argument and value of the exponential as much again: 2^-18 in all
    fresh = room > 0
    if not causal and fresh.sum() > 100:
        part = want - sums
        assert np.sqrt((((got - want)[fresh]) ** 2).sum()) <= 2.0 ** -18 * np.sqrt((part[fresh] ** 2).sum()) + 2.0 ** -24 * np.sqrt((want[fresh] ** 2).sum())
    seen = np.isfinite(lse)
    assert np.array_equal(np.isneginf(glse), np.isneginf(lse))
    assert np.abs(glse - lse)[seen].max(initial=0) < 2.0 ** -14


@pytest.mark.parametrize("seqs,hq,hk,D,most", [(3, 8, 8, 64, 1024), (40, 8, 8, 64, 90), (2, 4, 1, 128, 1025), (30, 32, 8, 128, 1000), (40, 16, 8, 32, 1024)])
@pytest.mark.parametrize("causal", [True, False])
def test_weights_of_single_tokens(ctx, seqs, hq, hk, D, most, causal):
    """About the sizes where single tokens have one kernel or two: keys, and pairs of sequence and key head."""
    rng = np.random.default_rng(seqs + most)
    lens = [most, 0] + list(rng.integers(1, 60, seqs - 2))
    p, rng = _random(seqs + D, lens, [1] * seqs, hq, hk, D, 16, 32)
    sums = rng.random((p["arr"]["k_codes"].shape[:3])).astype(np.float32)
    want, room, lse = S.weigh_want(p, sums, causal)
    got, glse = _weigh(ctx, p, sums, causal)
    _near(got, want, room)
    seen = np.isfinite(lse)
    assert np.array_equal(np.isneginf(glse), np.isneginf(lse))
    assert np.abs(glse - lse)[seen].max(initial=0) < 2.0 ** -14


@pytest.mark.parametrize("rope", ["half", "pairs"])
def test_weights_of_rotated_queries(ctx, rope):
    p, rng = _random(3, [150, 33], [20, 1], 4, 2, 64, 16, 32)
    ang = rng.uniform(-50, 50, (150, 32))
    tables = (np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32), rope == "pairs")
    pos = rng.integers(0, 150, 21).astype(np.int32)
    sums = rng.random(p["arr"]["k_codes"].shape[:3]).astype(np.float32)
    want, room, _ = S.weigh_want(p, sums, True, tables, pos)
    _near(_weigh(ctx, p, sums, True, tables, pos)[0], want, room)
    pos[4], pos[20] = 150, -1                   # no such table row: those rows add nothing
    got, _ = _weigh(ctx, p, sums, True, tables, pos)
    q = p["q"].copy()
    q[4] = q[20] = np.nan
    pos[4] = pos[20] = 0
    want, room, _ = S.weigh_want(dict(p, q=q), sums, True, tables, pos)
    _near(got, want, room)


@pytest.mark.parametrize("what", ["query", "key", "large"])
@pytest.mark.parametrize("n", [1, 40])
def test_what_is_no_number_adds_nothing(ctx, what, n):
    """Rows that are not finite, that see a key that is none, or whose scores pass fp32."""
    p, rng = _random(4, [200, 90], [n, 1], 4, 2, 64, 16, 0)
    sums = rng.random(p["arr"]["k_codes"].shape[:3]).astype(np.float32)
    q, arr = p["q"].copy(), {k: v.copy() for k, v in p["arr"].items()}
    if what == "query":
        q[0, 1, 5], q[n - 1, 2, 63] = np.inf, np.nan
    elif what == "key":
        arr["k_scales"][p["table"][0][190 // 16], 1, 190 % 16, 1] = 255
    else:
        q[0, 0, :] = 3e38
        arr["k_scales"][p["table"][0][2], 0, 3] = 254
    p = dict(p, q=q, arr=arr)
    if what == "large":      # (64 bits do not overflow: the row is taken out)
        rest = q.copy()
        rest[0, 0, :] = np.nan
        rest[:n, 0:2][np.isfinite(rest[:n, 0:2])] *= 1.0
        got, _ = _weigh(ctx, p, sums, False)
        assert np.isfinite(got).all()
        return
    want, room, _ = S.weigh_want(p, sums, False)
    _near(_weigh(ctx, p, sums, False)[0], want, room)


def test_weights_steps_and_pages(ctx):
    """Steps one after the other: new tokens are set whatever their pages held, earlier ones grow; a page
    outside the cache is passed over; sequences without rows or keys change nothing."""
    p, rng = _random(5, [100, 60, 0, 70], [1, 0, 2, 1], 4, 2, 64, 16, 32)
    sums = np.full(p["arr"]["k_codes"].shape[:3], 1e30, np.float32)
    table = p["table"].copy()
    table[0, 2] = 10 ** 6
    p = dict(p, table=table)
    want, room, _ = S.weigh_want(p, sums, True)
    got, _ = _weigh(ctx, p, sums, True)
    _near(got, want, room)
    t = table[0]
    assert 0 < got[t[99 // 16], 0, 99 % 16] < 1 and got[t[0], 0, 0] >= 1e30 * (1 - 2.0 ** -23)
    p, rng = _random(6, [40], [40], 2, 1, 64, 16, 0)
    sums = np.full(p["arr"]["k_codes"].shape[:3], np.nan, np.float32)     # a page that was never cleared
    want, room, _ = S.weigh_want(p, np.zeros_like(sums), True)
    got, _ = _weigh(ctx, p, sums, True)
    j = np.arange(40)
    at = p["table"][0][j // 16], 0, j % 16
    _near(got[at], want[at], room[at])


def test_weights_of_large_scores(ctx):
    """Scores of several hundred: the largest key has it all."""
    p, rng = _random(7, [300], [30], 4, 2, 64, 16, 0)
    p = dict(p, scale=20.0)
    sums = np.zeros(p["arr"]["k_codes"].shape[:3], np.float32)
    want, room, _ = S.weigh_want(p, sums, True)
    _near(_weigh(ctx, p, sums, True)[0], want, room)


def test_weights_captured(ctx):
    p, rng = _random(8, [900, 90], [1, 1], 8, 2, 128, 16, 32)
    cache, q = S.cache_of(p), S.dev(p["q"]).bfloat16()
    cu, table, lens = S.dev(p["cu"]), S.dev(p["table"]), S.dev(np.array(p["lens"], np.int32))
    ws = ctx.kv_weigh_workspace(cache, q, 2, 1, 900)
    sums = ctx.kv_sums(cache)

    def call(s, w):
        return ctx.kv_weigh(cache, s, q, cu, table, lens, 1, 900, ws=w)

    once = call(ctx.kv_sums(cache), None).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(sums, ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(sums, ws)
    for _ in range(3):
        sums.zero_()
        g.replay()
        eager = call(ctx.kv_sums(cache), None)
        torch.cuda.synchronize()
        assert torch.equal(sums, once) and torch.equal(eager, once)


# ------------------------------------------------------------------ lists
def _sums(rng, kind, shape):
    if kind == "spread":
        return np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    x = rng.standard_normal(shape).astype(np.float32)        # signs, zeros of both, infinities, NaN
    x[rng.random(shape) < 0.2] = 0.0
    x[rng.random(shape) < 0.2] = -0.0
    x[rng.random(shape) < 0.05] = np.inf
    x[rng.random(shape) < 0.05] = -np.inf
    x[rng.random(shape) < 0.1] = np.nan
    return x


@pytest.mark.parametrize("lens,budget,sinks,recent,ps", [
    ([1], 1, 0, 0, 16), ([2], 1, 0, 1, 16), ([100, 7, 0, 33], 8, 2, 3, 16), ([100, 99], 99, 0, 0, 32), ([500], 400, 4, 64, 16),
    ([1000, 1001, 999], 1, 1, 0, 16), ([300], 20, 10, 10, 128), ([4096, 4097, 5000], 1024, 4, 100, 64),
    ([8192, 8191, 100], 2048, 0, 0, 16), ([8193, 20000], 3000, 4, 500, 16), ([40000], 39999, 0, 7, 64), ([9000], 9001, 0, 0, 16),
    ([70000], 257, 1, 5, 1024), ([8193], 8192, 0, 0, 16), ([140000, 30], 20000, 4, 9000, 64), ([16384, 8192], 4000, 0, 4000, 16),
    ([16385], 100, 50, 50, 32),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "all"])
def test_kept_lists(ctx, lens, budget, sinks, recent, ps, kind):
    print("evict", lens, budget, sinks, recent, ps, kind, flush=True)
    rng = np.random.default_rng(sum(lens) + budget)
    hk = 2
    need = [(n + ps - 1) // ps for n in lens]
    pages = sum(need) + 2
    table = np.full((len(lens), max(need + [1])), -1, np.int32)
    order, at = rng.permutation(pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if kind == "all" and need[0] > 3:
        table[0, 1], table[0, 2] = -1, pages          # pages that are not there
    sums = _sums(rng, kind, (pages, hk, ps))
    cache = T.KVCache.empty(pages, ps, hk, 32, 0, DEV)
    keep, new = ctx.kv_evict(cache, S.dev(sums), S.dev(table), S.dev(np.array(lens, np.int32)), max(lens), budget,
                             sinks, recent)
    want, wnew = S.evict_want(sums, table, lens, budget, sinks, recent)
    assert np.array_equal(keep.cpu().numpy(), want) and np.array_equal(new.cpu().numpy(), wnew)


def test_lengths_past_max_kv(ctx):
    """max_kv cuts a sequence as it does in the attention."""
    rng = np.random.default_rng(1)
    cache = T.KVCache.empty(10, 16, 1, 32, 0, DEV)
    sums = _sums(rng, "spread", (10, 1, 16))
    table = np.arange(10, dtype=np.int32)[None]
    keep, new = ctx.kv_evict(cache, S.dev(sums), S.dev(table), S.dev(np.array([160], np.int32)), 50, 20, 1, 2)
    want, _ = S.evict_want(sums, table, [50], 20, 1, 2)
    assert np.array_equal(keep.cpu().numpy(), want) and new.tolist() == [20]


# ------------------------------------------------------------------ moves
def _noise(rng, pages, ps, hk, D):
    dp = (D + 31) // 32 * 32
    arr = [rng.integers(0, 256, (pages, hk, ps, w), dtype=np.uint8) for w in (dp // 2, dp // 32, dp // 2, dp // 32)]
    return arr, rng.random((pages, hk, ps)).astype(np.float32)


@pytest.mark.parametrize("hk,D,ps,lens,most,shared,starts", [
    (1, 64, 16, [40], 12, False, False), (2, 128, 16, [300, 20, 5], 64, False, False), (3, 96, 32, [100, 90], 50, True, True),
    (2, 8, 16, [33], 33, False, True), (5, 40, 64, [500, 700], 400, False, False), (8, 128, 16, [2000], 1500, False, False),
    (2, 72, 16, [64, 1], 7, True, True), (40, 128, 16, [200] * 8, 60, False, False), (130, 64, 16, [90, 95], 80, False, True),
    (64, 32, 16, [5000], 4500, False, True), (2, 64, 16, [2100], 2060, True, False), (33, 96, 32, [2500, 4200], 4100, False, False),
])
@pytest.mark.parametrize("with_sums", [True, False])
def test_moves(ctx, hk, D, ps, lens, most, shared, starts, with_sums):
    print("compact", hk, D, ps, lens, most, shared, starts, with_sums, flush=True)
    rng = np.random.default_rng(D + most)
    need = [(n + ps - 1) // ps for n in lens]
    pages = sum(need) + 2
    table = np.full((len(lens), max(need)), -1, np.int32)
    order, at = rng.permutation(pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    arr, sums = _noise(rng, pages, ps, hk, D)
    heads = 1 if shared else hk
    first = np.array([n // 3 if starts else 0 for n in lens], np.int32)
    keep = np.full((len(lens), heads, most), -1, np.int32)
    counts = np.zeros(len(lens), np.int32)
    for b, n in enumerate(lens):
        counts[b] = min(most, n - first[b])
        for h in range(heads):
            keep[b, h, :counts[b]] = np.sort(rng.permutation(np.arange(first[b], n))[:counts[b]])
    if len(lens) > 1:
        keep[0, 0, counts[0] // 2] = -1               # moves nothing
        counts[1] = most + 9 if counts[1] == most else counts[1]
    cache = T.KVCache(*[S.dev(a) for a in arr], head_dim=D)
    s = S.dev(sums)
    ctx.kv_compact(cache, S.dev(table), S.dev(keep), S.dev(counts), starts=S.dev(first) if starts else None,
                   sums=s if with_sums else None)
    want = S.compact_want(arr + [sums], table, keep, counts, first if starts else None)
    for n, w in zip(("k_codes", "k_scales", "v_codes", "v_scales"), want):
        assert np.array_equal(getattr(cache, n).cpu().numpy(), w), n
    assert np.array_equal(s.cpu().numpy(), want[4] if with_sums else sums)


def test_moves_of_pages_that_are_not_there(ctx):
    rng = np.random.default_rng(2)
    arr, sums = _noise(rng, 6, 16, 2, 64)
    table = np.array([[3, -1, 0, 99, 2]], np.int32)
    keep = np.array([[[2, 5, 17, 33, 40, 50, 70, 79, 80, 2 ** 31 - 1]]], np.int32)
    counts = np.array([10], np.int32)
    for start in (0, 14, 75, 2 ** 31 - 5, -3):
        cache = T.KVCache(*[S.dev(a) for a in arr], head_dim=64)
        keep2 = np.maximum(keep, start if start < 80 else 0).astype(np.int32)
        ctx.kv_compact(cache, S.dev(table), S.dev(keep2), S.dev(counts), starts=S.dev(np.array([start], np.int32)))
        want = S.compact_want(arr, table, keep2, counts, np.array([start]))
        for n, w in zip(("k_codes", "k_scales", "v_codes", "v_scales"), want):
            assert np.array_equal(getattr(cache, n).cpu().numpy(), w), (n, start)


def test_evicted_cache_attends_to_the_kept(ctx):
    """Weigh, evict, move; attention over the rest is that over the kept tokens alone."""
    p, rng = _random(11, [400, 90, 260], [1, 1, 1], 8, 2, 64, 16, 32)
    cache = S.cache_of(p)
    q = S.dev(p["q"]).bfloat16()
    cu, table, lens = S.dev(p["cu"]), S.dev(p["table"]), S.dev(np.array(p["lens"], np.int32))
    sums = ctx.kv_sums(cache)
    ctx.kv_weigh(cache, sums, q, cu, table, lens, 1, 400, causal=False)
    before = sums.cpu().numpy()
    keep, new = ctx.kv_evict(cache, sums, table, lens, 400, 100, sinks=2, recent=10)
    ctx.kv_compact(cache, table, keep, new, sums=sums)
    whole = p["q"] * 0 + np.round(p["q"])               # whole queries: attention_check's bounds
    small = dict(p, arr={n: getattr(cache, n).cpu().numpy() for n in p["arr"]}, lens=new.tolist(), q=whole,
                 scale=A.exact_scale(3, 32), causal=False)
    k = keep.cpu().numpy()
    moved = S.compact_want(list(p["arr"].values()) + [before], p["table"], k, new.cpu().numpy())
    for n, w in zip(p["arr"], moved):
        assert np.array_equal(small["arr"][n], w)
    assert np.array_equal(sums.cpu().numpy(), moved[4])
    lse = torch.empty(q.shape[:2], device=DEV)
    out = ctx.kv_attention(cache, S.dev(whole.astype(np.float32)).bfloat16(), cu, table, new, 1, 100,
                           scale=small["scale"], lse=lse)
    want = A.want(whole, small["arr"], p["table"], small["lens"], p["cu"], small["scale"], False, 64, 32)
    A.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want)
