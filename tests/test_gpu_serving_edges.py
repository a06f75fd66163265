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
