"""Attention of trees of drafted tokens over the paged cache, and the masks from parents, against
64 bits: queries that the kernel holds exactly (attention_check's bounds)."""
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


def _see(p, rng, kind="tree"):
    see = []
    for n in np.diff(p["cu"]):
        if kind == "tree":
            see.append(S.ancestors(S.random_parents(rng, int(n)))[0])
        elif kind == "chain":
            see.append(np.tril(np.ones((n, n), bool)))
        elif kind == "any":              # any mask at all, rows without a node among them
            m = rng.random((n, n)) < 0.4
            m[rng.random(n) < 0.3] = False
            see.append(m)
        else:                            # nothing of the tree
            see.append(np.zeros((n, n), bool))
    return see


def _mask(p, see, words=None):
    words = words or max((int(np.diff(p["cu"]).max()) + 63) // 64, 1)
    return np.concatenate([S.packed(m, words) for m in see]) if len(see) else np.zeros((0, words), np.int64)


def _run(ctx, p, mask, max_q=None, fill=None):
    cache = S.cache_of(p)
    q = S.dev(p["q"]).bfloat16()
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = None if fill is None else torch.full_like(q, fill)
    out = ctx.kv_tree_attention(cache, q, S.dev(mask), S.dev(np.asarray(p["cu"], np.int32)), S.dev(p["table"]),
                                S.dev(np.asarray(p["lens"], np.int32)), max_q or int(np.diff(p["cu"]).max()),
                                max(p["lens"]), scale=p["scale"], out=out, lse=lse)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("lens,qs,hq,hk,D,ps", [
    ([1], [1], 1, 1, 64, 16), ([9], [8], 4, 1, 128, 16), ([300, 77], [8, 5], 8, 2, 64, 16),
    ([64, 65, 63, 128], [16, 1, 7, 64], 4, 2, 40, 16), ([130], [65], 2, 1, 72, 32), ([1000], [26], 32, 8, 128, 16),
    ([700, 200, 90], [63, 64, 33], 8, 4, 96, 64), ([513], [130], 4, 4, 32, 128), ([2500, 40], [12, 40], 12, 2, 112, 16),
    ([5000], [4], 4, 1, 128, 64), ([4100], [3], 2, 2, 8, 16), ([260], [200], 3, 3, 80, 16),
])
@pytest.mark.parametrize("had", [0, 32])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_against_64_bits(ctx, lens, qs, hq, hk, D, ps, had, kind):
    print("tree", lens, qs, hq, hk, D, ps, had, kind, flush=True)
    p = A.problem(sum(lens) + D, lens, qs, hq, hk, D, ps, had, k=3)
    see = _see(p, np.random.default_rng(D + had), kind)
    A.check(*_run(ctx, p, _mask(p, see)), S.tree_want(p, see))


@pytest.mark.parametrize("lens,qs,hq,hk,D,ps", [
    ([1000, 300, 20], [8, 3, 6], 16, 4, 128, 16), ([90], [32], 2, 2, 96, 32), ([513, 70], [10, 1], 6, 2, 72, 16),
    ([4000, 17], [17, 17], 1, 1, 128, 64), ([200, 90], [33, 5], 1, 1, 128, 16),
])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_about_32_rows(ctx, lens, qs, hq, hk, D, ps, kind):
    """Rows of two tiles of 16, where there are no more (33: one of 128)."""
    p = A.problem(sum(lens) + 7 * D, lens, qs, hq, hk, D, ps, 32, k=3)
    see = _see(p, np.random.default_rng(D), kind)
    A.check(*_run(ctx, p, _mask(p, see)), S.tree_want(p, see))


@pytest.mark.parametrize("n", [3, 40])
def test_rows_that_see_nothing_answer_zeros(ctx, n):
    """A cache that holds the tree alone, and a mask without a node: zeros and -infinity."""
    p = A.problem(n, [n], [n], 4, 2, 64, 16, 32)
    see = _see(p, np.random.default_rng(0), "none")
    out, lse = _run(ctx, p, _mask(p, see))
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("D,hq,hk,n", [(64, 4, 1, 20), (128, 2, 2, 90), (128, 8, 2, 4)])
def test_a_chain_is_causal(ctx, D, hq, hk, n):
    """A chain's mask gives what kv_attention's causal rows give, within both bounds."""
    p = A.problem(D, [333, n], [n, n], hq, hk, D, 16, 32, k=3)
    see = _see(p, np.random.default_rng(0), "chain")
    w = A.want(p["q"], p["arr"], p["table"], p["lens"], p["cu"], p["scale"], True, D, 32)
    A.check(*_run(ctx, p, _mask(p, see)), w)


def test_more_rows_than_keys(ctx):
    """Nodes whose keys would lie before the first token do not exist."""
    p = A.problem(3, [5, 0], [12, 6], 4, 2, 64, 16, 0)
    see = _see(p, np.random.default_rng(1), "tree")
    A.check(*_run(ctx, p, _mask(p, see)), S.tree_want(p, see))


@pytest.mark.parametrize("m", [1, 7, 30])
def test_rows_past_max_q(ctx, m):
    """Only max_q rows of a sequence are computed; the tree stays as large as it is.  Words past the
    needed ones are read as they are."""
    p = A.problem(5, [120, 60], [40, 9], 4, 2, 64, 16, 32)
    see = _see(p, np.random.default_rng(2), "any")
    out, lse, room, lroom = S.tree_want(p, see)
    got, glse = _run(ctx, p, _mask(p, see, 3), m, fill=9.0)
    done = np.concatenate([np.arange(n) for n in np.diff(p["cu"])]) < m
    A.check(got[done], glse[done], (out[done], lse[done], room[done], lroom[done]))
    assert (got[~done] == 9).all() and (glse[~done] == 7).all()


def test_rows_of_no_sequence_are_left(ctx):
    p = A.problem(6, [80, 50], [10, 6], 4, 2, 64, 16, 32)
    see = _see(p, np.random.default_rng(3))
    want = S.tree_want(p, see)
    q = np.concatenate([p["q"], p["q"][:3]])
    mask = np.concatenate([_mask(p, see), np.full((3, 1), -1, np.int64)])
    got, lse = _run(ctx, dict(p, q=q), mask, fill=5.0)
    A.check(got[:16], lse[:16], want)
    assert (got[16:] == 5).all() and (lse[16:] == 7).all()


@pytest.mark.parametrize("rows,hq,hk", [(9, 1, 1), (30, 4, 1), (70, 2, 1)])
def test_nodes_that_are_no_number(ctx, rows, hq, hk):
    """A poisoned node makes NaN of the rows that see it and leaves every other row its bits; so does
    a page that is not in the cache, whose keys nobody sees."""
    p = A.problem(7, [200], [rows], hq, hk, 64, 16, 32)
    see = _see(p, np.random.default_rng(4))
    mask = _mask(p, see)
    clean, _ = _run(ctx, p, mask)
    bad = {k: v.copy() for k, v in p["arr"].items()}
    node = rows // 2
    j = 200 - rows + node
    bad["k_scales"][p["table"][0][j // 16], :, j % 16] = 255
    got, _ = _run(ctx, dict(p, arr=bad), mask)
    touched = see[0][:, node]
    assert np.isnan(got[touched]).all() and (got[~touched] == clean[~touched]).all()
    table = p["table"].copy()
    table[0, 3] = -1
    q = dict(p, table=table)
    A.check(*_run(ctx, q, mask), S.tree_want(q, see))


@pytest.mark.parametrize("rope", ["half", "pairs"])
def test_rotated_queries(ctx, rope):
    """Rows turned to the depth of their node: the same as rows turned beforehand in 64 bits and held
    in bf16 to 2^-8 (what a score moves by, a few hundredths, moves a weight; bound 2^-4 of the
    largest value)."""
    rng = np.random.default_rng(8)
    p = A.problem(8, [150], [20], 4, 2, 64, 16, 0)
    parents = S.random_parents(rng, 20)
    see, depth = S.ancestors(parents)
    half = 32
    ang = rng.uniform(-3, 3, (150, half))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = (130 + depth).astype(np.int32)
    from oracle import block_oracle as B
    turned = B.rotate_f64(p["q"], cos, sin, pos, rope == "pairs")
    want = S.tree_want(dict(p, q=turned), [see])[0]
    cache = S.cache_of(p)
    out = ctx.kv_tree_attention(cache, S.dev(p["q"]).bfloat16(), S.dev(_mask(p, [see])), S.dev(p["cu"]),
                                S.dev(p["table"]), S.dev(np.array([150], np.int32)), 20, 150, scale=p["scale"],
                                rope=T.Rope(S.dev(cos), S.dev(sin), rope == "pairs"), positions=S.dev(pos))
    off = np.abs(out.double().cpu().numpy() - want)
    assert off.max() <= 2.0 ** -4 * np.abs(want).max() and off.mean() < 2.0 ** -8


@pytest.mark.parametrize("sizes", [[1], [5, 0, 17], [64, 65, 3], [300], [1000, 2]])
def test_tree_mask(ctx, sizes):
    rng = np.random.default_rng(sum(sizes))
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    parents = [S.random_parents(rng, n) for n in sizes]
    if sizes[0] > 3:
        parents[0][2] = 2                      # itself, a later one, far outside: no parent
        parents[0][3] = 1 << 30
        parents[0][1] = 4
    mask, depth = ctx.tree_mask(S.dev(np.concatenate(parents)), S.dev(cu), max(sizes))
    see = [S.ancestors(p) for p in parents]
    words = max((max(sizes) + 63) // 64, 1)
    assert np.array_equal(mask.cpu().numpy(), np.concatenate([S.packed(m, words) for m, _ in see]))
    assert np.array_equal(depth.cpu().numpy(), np.concatenate([d for _, d in see]))


def test_tree_mask_long_chain(ctx):
    n = 8192
    mask, depth = ctx.tree_mask(S.dev(np.arange(-1, n - 1, dtype=np.int32)), S.dev(np.array([0, n], np.int32)), n)
    assert np.array_equal(depth.cpu().numpy(), np.arange(n))
    bits = np.unpackbits(mask.cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    assert np.array_equal(bits, np.tril(np.ones((n, n), np.uint8)))


def test_captured_and_on_another_stream(ctx):
    """Replays between eager calls, and a call on a side stream, give the eager bits."""
    p = A.problem(9, [700, 90], [20, 8], 8, 2, 128, 16, 32)
    see = _see(p, np.random.default_rng(5))
    cache, q, mask = S.cache_of(p), S.dev(p["q"]).bfloat16(), S.dev(_mask(p, see))
    cu, table, lens = S.dev(p["cu"]), S.dev(p["table"]), S.dev(np.array(p["lens"], np.int32))
    ws = ctx.kv_tree_attention_workspace(cache, q, 2, 20, 700)
    out = torch.empty_like(q)

    def call(o, w):
        return ctx.kv_tree_attention(cache, q, mask, cu, table, lens, 20, 700, scale=p["scale"], out=o, ws=w)

    want = call(torch.empty_like(q), None).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(torch.empty_like(q), None)
        g = torch.cuda.CUDAGraph()
        call(out, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    with torch.cuda.graph(g):
        call(out, ws)
    for _ in range(3):
        out.fill_(3.0)
        g.replay()
        eager = call(torch.empty_like(q), None)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)
