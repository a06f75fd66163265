"""Attention over the paged cache where the ordinary problems do not reach: queries that the kernel
holds exactly, so that a result is checked to what the weights' rounding leaves (attention_check)."""
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


def _run(ctx, p, max_q=None, fill=None):
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)       # noqa: E731
    cache = T.KVCache(*[d(p["arr"][x]) for x in ("k_codes", "k_scales", "v_codes", "v_scales")],
                      head_dim=p["D"], had_block=p["had"])
    q = d(p["q"]).bfloat16()
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = None if fill is None else torch.full_like(q, fill)
    out = ctx.kv_attention(cache, q, d(np.asarray(p["cu"], np.int32)), d(p["table"]),
                           d(np.asarray(p["lens"], np.int32)), max_q or int(np.diff(p["cu"]).max()), max(p["lens"]),
                           scale=p["scale"], causal=p["causal"], out=out, lse=lse)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _want(p):
    return A.want(p["q"], p["arr"], p["table"], p["lens"], p["cu"], p["scale"], p["causal"], p["D"], p["had"])


@pytest.mark.parametrize("had", [0, 32])
@pytest.mark.parametrize("hq,hk,D", [(4, 1, 64), (2, 2, 128), (8, 2, 40)])
def test_rows_past_max_q_keep_the_mask(ctx, hq, hk, D, had):
    """Only the first max_q rows of a sequence are computed, and each sees what it sees of the whole
    sequence: the causal limit goes by all of the sequence's queries."""
    p = A.problem(D + hq, [70, 9, 200], [40, 20, 90], hq, hk, D, 16, had, k=3)
    out, lse, room, lroom = _want(p)
    for m in (1, 3, 16, 17, 39, 90):
        print("attention max_q", m, "heads", hq, hk, "D", D, "had", had, flush=True)
        got, glse = _run(ctx, p, m, fill=9.0)
        in_seq = np.concatenate([np.arange(n) for n in np.diff(p["cu"])])
        done = in_seq < m
        A.check(got[done], glse[done], (out[done], lse[done], room[done], lroom[done]))
        assert (got[~done] == 9).all() and (glse[~done] == 7).all()


def _bytes(kind, b):
    """Scale bytes of the values: all b; b in some keys; b in one key; b in the last block alone."""
    def make(rng, shape):
        x = rng.integers(125, 130, shape)
        if kind == "all":
            x[...] = b
        elif kind == "some":
            x[rng.random(shape[:3]) < 0.1] = b
        elif kind == "one":
            x[shape[0] // 2, :, 3] = b
        else:
            x[..., -1] = b
        return x
    return make


@pytest.mark.parametrize("rows,heads,D", [(1, 2, 128), (16, 1, 64), (20, 2, 64), (140, 1, 128), (1, 3, 32),
                                          (33, 1, 96)])
@pytest.mark.parametrize("had", [0, 32])
@pytest.mark.parametrize("kind", ["all", "some", "one", "block"])
def test_values_of_any_finite_size(ctx, rows, heads, D, had, kind):
    """Scores of about +-36 (base 2), where the weights need no reference, with values from 2^-126 to
    2^127: the result is finite and as exact as that of ordinary values."""
    for n in (1, 5, 64, 300, 2000):
        for b in (1, 30, 60, 66, 67, 90, 177, 178, 210, 245, 252):
            print("attention rows", rows, "heads", heads, "D", D, "had", had, kind, b, "keys", n, flush=True)
            p = A.steep_problem(n + b, n, rows, heads, D, had, _bytes(kind, b))
            w = _want(p)
            A.check(*_run(ctx, p), w)
            some = w[0] != 0
            assert A.outside(0.0, w[0][some], w[2][some]) > 0.6          # zeros would not pass


@pytest.mark.parametrize("D", [64, 128])
def test_far_values_do_not_reach_rows_that_do_not_see_them(ctx, D):
    """Causal rows before a key of a far value are the same bits as with an ordinary one."""
    for rows, n in ((40, 60), (8, 30), (150, 400)):
        for b in (20, 240):
            p = A.steep_problem(rows, n, rows, 2, D, 32, _bytes("all", 127), causal=True)
            a = _run(ctx, p)
            j = n - rows // 2                       # seen by rows // 2 rows
            p["arr"]["v_scales"][p["table"][0, j // 16], :, j % 16, 1] = b
            c = _run(ctx, p)
            w = _want(p)
            A.check(*c, w)
            before = rows - rows // 2
            assert np.array_equal(a[0][:before], c[0][:before]) and np.array_equal(a[1][:before], c[1][:before])


def test_far_values_same_bits_every_time(ctx):
    for rows in (1, 70):
        p = A.steep_problem(3, 3000, rows, 2, 64, 32, _bytes("some", 230))
        a = _run(ctx, p)
        for _ in range(5):
            b = _run(ctx, p)
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("rows", [1, 16, 40])
@pytest.mark.parametrize("D", [32, 128])
def test_queries_are_held_to_13_bits(ctx, rows, D):
    """One key of one code and a score in the hundreds, which lse gives to fp32: an element of the
    query, times the scale, with a mantissa anywhere, just below a power of two among them, is held
    to 2^-13 of the largest of its block (and the score to 2^-21 of its absolute sum)."""
    rng = np.random.default_rng(rows + D)
    kc = np.zeros((1, 1, 16, D // 2), np.uint8)
    kc[..., 0], kc[..., -1] = 7, 0x50                     # a code of 6, and one of 3 in the last block
    ks = np.full((1, 1, 16, D // 32), 127 + 4, np.uint8)
    arr = dict(k_codes=kc, k_scales=ks, v_codes=kc.copy(), v_scales=np.full_like(ks, 127))
    mantissas = [1.0, 1.3, 1.87, 1.876, 1.93, 1.938, 1.99, 1.998, 1.9996, 1.99997, 1.9999995]
    for m in mantissas + list(rng.uniform(1, 2, 8)):
        scale = float(np.float32(m / float(A.LOG2E)))
        q = np.zeros((rows, 1, D), np.float32)
        q[:, 0, 0] = rng.choice([-1.0, 1.0], rows)        # times the scale and log2(e): the mantissa
        q[:, 0, -1] = rng.choice([-1.0, 1.0, 0.5, 0.375], rows)
        p = dict(arr=arr, table=np.zeros((1, 1), np.int32), lens=[1], cu=np.array([0, rows], np.int32), q=q,
                 scale=scale, causal=False, D=D, had=0)
        _, lse = _run(ctx, p)
        k, _, _ = A.gathered(arr, [0], 1)
        s, spread = A.scores(q[:, 0], k[0], scale, 0)
        top = np.abs(q[:, 0]).reshape(rows, -1, 32).max(2)
        kmag = np.abs(k[0, 0]).reshape(-1, 32).sum(1)
        slip = (top * kmag).sum(1) * scale * 2.0 ** -13 + spread[:, 0] * 2.0 ** -21
        off = np.abs(lse[:, 0] - s[:, 0])
        # a score within 40 (base 2) has a weight that is rounded to bf16
        small = np.abs(s[:, 0]) <= 40.5 * np.log(2)
        assert (off <= slip + np.abs(s[:, 0]) * 2.0 ** -22 + np.where(small, 2.0 ** -8, 0)).all(), (m, off, slip)
        assert small.mean() < 0.7


@pytest.mark.parametrize("kind", A.CLIMBS)
@pytest.mark.parametrize("rows,copies,D,n", [
    (1, 1, 64, 1300), (1, 1, 128, 9000), (7, 256, 64, 1300), (16, 128, 128, 1300), (1, 256, 32, 1300),
    (20, 1, 64, 1300), (20, 1, 128, 9000), (20, 256, 64, 1300), (150, 64, 96, 1300), (33, 256, 32, 1300),
])
def test_references_that_move(ctx, kind, rows, copies, D, n):
    """Scores that climb, fall or jump by tens while earlier sums still count, in ranges, in waves and
    in one pass; test_attention_bounds shows which mistakes these rooms reject."""
    for had in (0, 32):
        print("attention", kind, "rows", rows, "heads", 2 * copies, "D", D, "keys", n, "had", had, flush=True)
        p = A.climb_problem(n + D, kind, n, rows, 2, D, had, copies)
        out, lse = _run(ctx, p)
        w = _want(A.only_heads(p, 2))
        A.check(out[:, :2], lse[:, :2], w)
        assert A.outside(0.0, w[0], w[2]) > 0.4                       # zeros would not pass
        assert np.array_equal(out, np.tile(out[:, :2], (1, copies, 1)))
        assert np.array_equal(lse, np.tile(lse[:, :2], (1, copies)))


ORDINARY = [
    # lens, qs, hq, hk, D, page, had, causal
    ([1], [1], 1, 1, 64, 16, 0, True), ([17], [1], 8, 1, 128, 16, 32, True),
    ([64, 65, 63], [1, 1, 1], 8, 2, 128, 16, 32, True), ([1000, 1, 0, 333], [1, 1, 1, 1], 32, 8, 128, 16, 32, True),
    ([129], [1], 16, 1, 96, 32, 0, True), ([200], [1], 20, 1, 112, 64, 32, True),
    ([70, 300], [5, 1], 6, 2, 72, 16, 32, False), ([150, 40], [33, 40], 4, 4, 64, 64, 32, True),
    ([10, 100], [30, 7], 4, 2, 64, 16, 32, True), ([257], [130], 3, 3, 40, 128, 0, True),
    ([31, 300, 128], [64, 129, 1], 2, 2, 80, 16, 32, False), ([48], [17], 2, 1, 32, 16, 32, False),
    ([48], [3], 2, 1, 8, 16, 32, True), ([700], [200], 4, 1, 128, 32, 32, True),
    ([2100], [2], 4, 2, 64, 16, 0, False), ([3000, 5], [1, 1], 4, 1, 96, 16, 0, True),
    ([640], [100], 5, 5, 24, 16, 0, False),
]


@pytest.mark.parametrize("lens,qs,hq,hk,D,ps,had,causal", ORDINARY)
def test_ordinary_problems_closely(ctx, lens, qs, hq, hk, D, ps, had, causal):
    """Masks, ragged lengths, groups and pages with queries held exactly: what is left is the weights'
    rounding, so that most zeros would not pass."""
    print("attention lens", lens, "qs", qs, "heads", hq, hk, "D", D, "page", ps, "had", had, flush=True)
    for k in (3, 1):                                  # scores of a few units, and of tens
        p = A.problem(sum(lens) + D + k, lens, qs, hq, hk, D, ps, had, k=k + (4 if had else 0), causal=causal)
        w = _want(p)
        A.check(*_run(ctx, p), w)
        seen = np.isfinite(w[1])
        assert A.outside(0.0, w[0][seen], w[2][seen]) > 0.75


def test_counts_past_32_bits_are_refused(ctx):
    """A bound of 2^32 was cut to 0 on its way into the library, and every row answered zeros."""
    p = A.problem(1, [20], [2], 4, 2, 64, 16, 0)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)       # noqa: E731
    cache = T.KVCache(*[d(p["arr"][x]) for x in ("k_codes", "k_scales", "v_codes", "v_scales")], head_dim=64)
    q, cu, lens = d(p["q"]).bfloat16(), d(p["cu"]), d(np.asarray(p["lens"], np.int32))
    for max_q, max_kv in ((2, 1 << 32), (1 << 32, 20), (2, (1 << 32) + 20), (2, 1 << 31)):
        with pytest.raises(ValueError):
            ctx.kv_attention(cache, q, cu, d(p["table"]), lens, max_q, max_kv)
        with pytest.raises(ValueError):
            ctx.kv_attention_workspace(cache, q, 1, max_q, max_kv)
    with pytest.raises(T.TabitError) as e:
        ctx.kv_attention(cache, q, cu, d(p["table"]), lens, 2, -1)
    assert e.value.status == T.ESHAPE
    assert torch.isfinite(ctx.kv_attention(cache, q, cu, d(p["table"]), lens, 2, 20)).all()


@pytest.mark.parametrize("rows,n", [(1, 1), (16, 1), (17, 1), (140, 1), (1, 3000), (1, 400), (20, 3000)])
@pytest.mark.parametrize("had", [0, 32])
def test_one_visible_key_answers_its_value(ctx, rows, n, had):
    """One key alone, or one with all the weight of fp32 (the others 200 below, base 2): its value,
    rounded to bf16 (at a tie either way), and zero exactly where the value is zero."""
    for D in (64, 128):
        print("attention one key, rows", rows, "keys", n, "D", D, "had", had, flush=True)
        p = A.climb_problem(rows + n, "late", n, rows, 2, D, had)
        rng = np.random.default_rng(n + D)
        # every score -100 times the factor but one key's, +100
        codes = np.array([A._codes_of(-96), A._codes_of(96)], np.uint8)
        codes = codes[:, 0::2] | codes[:, 1::2] << 4
        kc = p["arr"]["k_codes"]
        kc[:, :, :, :8] = codes[0]
        at = n // 3
        kc[at // 16, :, at % 16, :8] = codes[1]
        if n > 1:
            p["q"] = np.repeat(A.climb_problem(1, "late", 64, rows, 2, D, had)["q"][:1], rows, 0)
        else:                                      # scores between -40 and 40, weights of any mantissa
            p["q"] = 0.3 * rng.standard_normal(p["q"].shape).astype(np.float32) / (5 if had else 1)
        for nib in range(3):                       # zeros among the values
            p["arr"]["v_codes"][:, :, :, nib::5] = 0
        out, _ = _run(ctx, p)
        _, v, _ = A.gathered(p["arr"], p["table"][0], n)
        want = A.joined(np.eye(n)[at:at + 1], v[0], had, D)[0], A.joined(np.eye(n)[at:at + 1], v[1], had, D)[0]
        for h in range(2):
            x = want[h]
            step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 1e-300))) - 7)
            tie = np.abs(np.abs(x / step - np.floor(x / step)) - 0.5) < 1e-9
            assert np.all(out[:, h][:, ~tie] == (np.rint(x / step) * step)[~tie])
            assert np.all(np.abs(out[:, h] - x) <= step / 2 * (1 + 1e-9))
            assert tie.mean() < 0.5
