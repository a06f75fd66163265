"""Accumulated attention weights in every form that a call may take, against 64 bits.

Up to eight rows a key head go by one kernel (up to 1024 keys, 256 pairs of sequence and key head) or by two, with
room for four rows or for eight; more rows by several, in one range of keys and rows or in more.
"""
import numpy as np
import pytest
import torch

from tests import attention_check as A
from tests import serve_check as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# lengths, rows, query heads, key heads, head_dim: a short second sequence, one without keys, one without rows
FORMS = {
    "one kernel, 4 rows": ([300, 90, 0, 40], [1, 1, 1, 0], 8, 2, 64),
    "one kernel, 8 rows": ([700, 90, 0, 40], [2, 1, 1, 0], 16, 4, 128),
    "two kernels, 4 rows": ([1500, 90, 0, 40], [2, 1, 1, 0], 4, 2, 96),
    "two kernels, 8 rows": ([2100, 90, 0, 40], [1, 1, 1, 0], 16, 2, 64),
    "one range": ([200, 90, 0, 40], [40, 20, 1, 0], 4, 2, 64),
    "ranges of keys": ([900, 90, 0, 40], [40, 20, 1, 0], 4, 2, 128),
    "ranges of rows": ([300, 90, 0, 40], [260, 20, 1, 0], 4, 2, 32),
}


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


def _problem(seed, lens, qs, hq, hk, D, ps=16, had=32):
    """Keys of a normal distribution and bf16 queries of one."""
    p = A.problem(seed, lens, qs, hq, hk, D, ps, had)
    rng = np.random.default_rng(seed + 1)
    q = torch.from_numpy(rng.standard_normal(p["q"].shape).astype(np.float32)).bfloat16().float().numpy()
    return dict(p, q=q, scale=float(np.float32(D ** -0.5))), rng


def _call(ctx, p, sums, causal, max_q=None, rope=None, positions=None):
    q = S.dev(np.asarray(p["q"], np.float32)).bfloat16()
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    got = S.dev(np.asarray(sums, np.float32))
    kw = {}
    if rope is not None:
        kw = dict(rope=T.Rope(S.dev(rope[0]), S.dev(rope[1]), rope[2]), positions=S.dev(positions))
    ctx.kv_weigh(S.cache_of(p), got, q, S.dev(np.asarray(p["cu"], np.int32)), S.dev(p["table"]),
                 S.dev(np.asarray(p["lens"], np.int32)), max_q or int(np.diff(p["cu"]).max()), max(p["lens"]),
                 scale=p["scale"], causal=causal, lse=lse, **kw)
    return got.double().cpu().numpy(), lse.double().cpu().numpy()


def _check(got, want):
    """Sums to their room, and the logarithms: a score errs by 2^-18 of its row's spread (serve_check), which is
    below 48 in these problems, and the sum and its logarithm by less than 2^-15: 2^-12 in all."""
    (sums, lse), (wsums, room, wlse) = got, want
    assert np.isfinite(sums).all()
    off = np.abs(sums - wsums)
    assert (off <= room).all(), (off.max(), np.argwhere(off > room)[:5])
    counted = np.isfinite(wlse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(wlse))
    assert np.abs(lse[counted] - wlse[counted]).max(initial=0) < 2.0 ** -12


@pytest.mark.parametrize("lens,qs,hq,hk,D,ps", [
    ([300, 77], [1, 1], 8, 1, 64, 16), ([1000], [1], 12, 2, 128, 16), ([700, 5], [2, 2], 8, 2, 96, 32), ([3, 200], [8, 5], 1, 1, 32, 16),
    ([1024, 60, 2], [2, 1, 2], 8, 2, 128, 64), ([8], [8], 1, 1, 40, 16), ([65, 64, 1], [1, 4, 2], 2, 1, 72, 16),
    ([1500, 40], [1, 1], 8, 1, 64, 16), ([1025], [2], 12, 3, 128, 16), ([3000, 7, 900], [8, 3, 8], 2, 2, 72, 16),
    ([5000], [1], 6, 1, 112, 64), ([4100, 4096, 2], [2, 2, 2], 4, 1, 8, 16), ([1100, 3], [5, 8], 1, 1, 128, 128),
])
@pytest.mark.parametrize("had", [0, 32])
@pytest.mark.parametrize("causal", [True, False])
def test_five_to_eight_rows(ctx, lens, qs, hq, hk, D, ps, had, causal):
    print("weigh", lens, qs, hq, hk, D, ps, had, causal, flush=True)
    p, rng = _problem(sum(lens) + D, lens, qs, hq, hk, D, ps, had)
    sums = rng.random(p["arr"]["k_codes"].shape[:3]).astype(np.float32)
    _check(_call(ctx, p, sums, causal), S.weigh_want(p, sums, causal))


@pytest.mark.parametrize("seqs,hq,hk,most", [(32, 32, 8, 200), (33, 32, 8, 200), (33, 8, 8, 1024), (65, 32, 4, 90)])
@pytest.mark.parametrize("causal", [True, False])
def test_up_to_two_rows_about_256_pairs(ctx, seqs, hq, hk, most, causal):
    rng = np.random.default_rng(seqs)
    lens, qs = [most, 0, 1] + list(rng.integers(1, 60, seqs - 3)), [2] + list(rng.integers(0, 3, seqs - 1))
    p, rng = _problem(seqs, lens, qs, hq, hk, 32)
    sums = rng.random(p["arr"]["k_codes"].shape[:3]).astype(np.float32)
    _check(_call(ctx, p, sums, causal), S.weigh_want(p, sums, causal))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("causal", [True, False])
def test_stale_sums_and_pages_that_are_not_there(ctx, form, causal):
    """What a page held counts for nothing where a token is new; pages outside the cache are passed over."""
    lens, qs, hq, hk, D = FORMS[form]
    p, rng = _problem(sum(lens), lens, qs, hq, hk, D)
    pages = p["arr"]["k_codes"].shape[0]
    table = p["table"].copy()
    table[0, 2], table[0, (lens[0] - 1) // 16], table[1, 0] = -1, pages, 1 << 30
    p = dict(p, table=table)
    sums = np.full(p["arr"]["k_codes"].shape[:3], 1e30 if causal else 3.0, np.float32)
    _check(_call(ctx, p, sums, causal), S.weigh_want(p, sums, causal))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("what", ["query", "key", "row that overflows", "key that overflows"])
@pytest.mark.parametrize("causal", [True, False])
def test_what_is_no_number(ctx, form, what, causal):
    """Rows that are not finite, that see a key that is none, or whose scores pass fp32 add nothing; every other row
    adds what it does without them."""
    lens, qs, hq, hk, D = FORMS[form]
    group = hq // hk
    p, rng = _problem(sum(lens) + 1, lens, qs, hq, hk, D, had=0)
    q, arr = p["q"].copy(), {k: v.copy() for k, v in p["arr"].items()}
    sums = rng.random(arr["k_codes"].shape[:3]).astype(np.float32)
    out = q.copy()                       # the rows that are to add nothing: 64 bits would not overflow
    if what == "query":
        q[0, 1, 5], q[qs[0] - 1, group, D - 1], q[qs[0], 0, 0] = np.inf, np.nan, -np.inf
        out = q
    elif what == "key":                  # with the causal mask the rows before it do not see it
        j = lens[0] - max(qs[0] // 2, 1)
        arr["k_scales"][p["table"][0][j // 16], 1, j % 16, 0] = 255
        arr["k_scales"][p["table"][1][1], 0, 3, 0] = 255
        out = q
    else:                                # every product with one key is positive, and so large that any sum passes fp32
        page = p["table"][0][1]
        arr["k_codes"][page, :, 4] = 0x77
        if what == "row that overflows":
            q[0, 0] = 3e38
            out[0, 0] = np.nan
        else:
            arr["k_scales"][page, 0, 4] = 254
            q[:qs[0], :group] = np.abs(q[:qs[0], :group]) + 0.5
            out[:qs[0], :group] = np.nan
    want = S.weigh_want(dict(p, q=out, arr=arr), sums, causal)
    got, lse = _call(ctx, dict(p, q=q, arr=arr), sums, causal)
    assert np.isfinite(got).all()
    off = np.abs(got - want[0])
    assert (off <= want[1]).all(), (off.max(), np.argwhere(off > want[1])[:5])
    counted = np.isfinite(want[2])
    assert np.isfinite(lse[counted]).all() and counted.any()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("pairs", [False, True])
def test_rotated_queries(ctx, form, pairs):
    lens, qs, hq, hk, D = FORMS[form]
    p, rng = _problem(sum(lens) + 2, lens, qs, hq, hk, D)
    ang = rng.uniform(-50, 50, (400, D // 4))                    # half of the elements are turned
    rope = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32), pairs
    pos = rng.integers(0, 400, sum(qs)).astype(np.int32)
    sums = rng.random(p["arr"]["k_codes"].shape[:3]).astype(np.float32)
    _check(_call(ctx, p, sums, True, rope=rope, positions=pos), S.weigh_want(p, sums, True, rope, pos))
    bad = pos.copy()
    bad[0], bad[qs[0]] = 400, -1                                 # no such table row
    q = p["q"].copy()
    q[0] = q[qs[0]] = np.nan
    want = S.weigh_want(dict(p, q=q), sums, True, rope, pos)
    got, _ = _call(ctx, p, sums, True, rope=rope, positions=bad)
    assert (np.abs(got - want[0]) <= want[1]).all()


@pytest.mark.parametrize("form", [f for f in FORMS if max(FORMS[f][1]) > 1])
def test_rows_past_max_q(ctx, form):
    """Only the first max_q rows of a sequence add; what is new goes by all of its rows."""
    lens, qs, hq, hk, D = FORMS[form]
    p, rng = _problem(sum(lens) + 3, lens, qs, hq, hk, D)
    sums = rng.random(p["arr"]["k_codes"].shape[:3]).astype(np.float32)
    most = max(qs) // 2
    q = p["q"].copy()
    in_seq = np.concatenate([np.arange(n) for n in qs])
    q[in_seq >= most] = np.nan                                   # (rows that are no number add nothing)
    want, room, _ = S.weigh_want(dict(p, q=q), sums, True)
    got, lse = _call(ctx, p, sums, True, max_q=most)
    assert (np.abs(got - want) <= room).all() and (lse[in_seq >= most] == 7).all()


@pytest.mark.parametrize("form", FORMS)
def test_captured(ctx, form):
    """Replays on one workspace, with other calls on it in between, give the eager bits."""
    lens, qs, hq, hk, D = FORMS[form]
    p, rng = _problem(sum(lens) + 4, lens, qs, hq, hk, D)
    cache, q = S.cache_of(p), S.dev(p["q"]).bfloat16()
    cu, table, n = S.dev(np.asarray(p["cu"], np.int32)), S.dev(p["table"]), S.dev(np.array(lens, np.int32))
    ws = ctx.kv_weigh_workspace(cache, q, len(lens), max(qs), max(lens))
    sums, lse = ctx.kv_sums(cache), torch.zeros(q.shape[:2], device=DEV)

    def call(s, logs, w):
        return ctx.kv_weigh(cache, s, q, cu, table, n, max(qs), max(lens), causal=False, lse=logs, ws=w)

    logs = torch.zeros_like(lse)
    once = call(ctx.kv_sums(cache), logs, None).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(sums, lse, ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(sums, lse, ws)
    for _ in range(3):
        sums.zero_()
        lse.zero_()
        ws.fill_(255)
        g.replay()
        eager = call(ctx.kv_sums(cache), None, ws)
        torch.cuda.synchronize()
        assert torch.equal(sums, once) and torch.equal(eager, once) and torch.equal(lse, logs)
