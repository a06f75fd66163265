"""Low-rank adapters of many requests beside a projection, against 64 bits.

Bounds: products are fp32 sums of K (rank) terms, off by at most K 2^-24 (rank 2^-23, two terms each) of
their absolute sum; x A^T in two bf16 terms by 2^-17 of itself and of what it was summed from; out is
rounded once, by half a step of bf16: 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import tabit_oracle as O
from tests import serve_check as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()


def _want(x, y, a, b, scale, cu, which):
    out, room = y.copy(), np.zeros_like(y)
    K, R = a.shape[2], a.shape[1]
    for i, w in enumerate(which):
        rows = slice(max(cu[i], 0), max(cu[i + 1], 0))
        if not 0 <= w < len(a):
            continue
        h, ha = x[rows] @ a[w].T * scale[w], np.abs(x[rows]) @ np.abs(a[w]).T * abs(scale[w])
        out[rows] += h @ b[w].T
        room[rows] = (ha * (K + 8) * 2.0 ** -24 + np.abs(h) * 2.0 ** -17) @ np.abs(b[w]).T
        room[rows] += (np.abs(h) @ np.abs(b[w]).T + np.abs(y[rows])) * (R + 2) * 2.0 ** -23
    return out, room + np.abs(out) * 2.0 ** -8 + 2.0 ** -134


def _segments(rng, rows, count):
    cuts = np.sort(rng.integers(0, rows + 1, count - 1)) if count > 1 else np.zeros(0, int)
    return np.concatenate([[0], cuts, [rows]]).astype(np.int32)


def _rows(rng, fmt, T_, K):
    """Device rows, their scales, and the fp64 values they stand for."""
    x = _bf(rng, T_, K)
    if fmt == "bf16":
        return x.to(DEV), None, x.double().numpy()
    if fmt == "int8":
        q = rng.integers(-127, 128, (T_, K)).astype(np.int8)
        s = rng.uniform(0.001, 0.1, T_).astype(np.float32)
        return S.dev(q), S.dev(s), q * s.astype(np.float64)[:, None]
    codes, e8 = O.mx_quantize_rows(x.float().numpy(), 0)
    return S.dev(codes), S.dev(e8), B.mx_values(codes, e8)


@pytest.mark.parametrize("rows,segments,adapters,rank,K,N", [
    (1, 1, 1, 16, 32, 32), (4, 4, 4, 16, 2240, 96), (3, 1, 2, 16, 96, 2240), (64, 64, 9, 64, 512, 640), (17, 5, 3, 32, 160, 224),
    (200, 3, 2, 16, 320, 288), (333, 2, 2, 32, 1152, 352), (129, 1, 1, 64, 256, 64), (500, 7, 3, 128, 192, 160), (65, 65, 65, 128, 64, 1056),
    (70, 100, 4, 32, 96, 96), (1000, 130, 5, 16, 64, 32),
])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "mxfp4"])
def test_against_64_bits(ctx, rows, segments, adapters, rank, K, N, fmt):
    print("adapter", rows, segments, adapters, rank, K, N, fmt, flush=True)
    rng = np.random.default_rng(rows + K)
    x, xs, xv = _rows(rng, fmt, rows, K)
    y = _bf(rng, rows, N)
    a, b = _bf(rng, adapters, rank, K, scale=K ** -0.5), _bf(rng, adapters, N, rank, scale=rank ** -0.5)
    scale = rng.uniform(-2, 2, adapters).astype(np.float32)
    cu = _segments(rng, rows, segments) if segments != rows else np.arange(rows + 1, dtype=np.int32)
    which = rng.integers(0, adapters, segments).astype(np.int32)
    if segments > 2:
        which[1], which[2] = -1, adapters            # no adapter: out = y
    bank = T.Adapters(a.to(DEV), b.to(DEV), S.dev(scale))
    yd = y.to(DEV)
    out = ctx.adapter_linear(bank, x, yd, S.dev(cu), S.dev(which), x_scale=xs)
    want, room = _want(xv, y.double().numpy(), a.double().numpy(), b.double().numpy(), scale.astype(np.float64), cu, which)
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= room).all(), (off.max(), np.argwhere(off > room)[:4])
    assert torch.equal(yd.cpu(), y)
    again = ctx.adapter_linear(bank, x, yd, S.dev(cu), S.dev(which), x_scale=xs, out=yd)     # in place
    assert again is yd and torch.equal(yd, out)


@pytest.mark.parametrize("few", [True, False])
def test_slices_and_rows_of_no_segment(ctx, few):
    """x, y and out as slices of wider rows; rows before the first and behind the last segment, and what
    lies beside the slices, are left; no scale is a scale of one."""
    rng = np.random.default_rng(3)
    rows, K, N = (12, 64, 96) if few else (150, 64, 96)
    x, y, out = _bf(rng, rows, K + 24).to(DEV), _bf(rng, rows, N + 40).to(DEV), torch.full((rows, N + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    a, b = _bf(rng, 2, 32, K, scale=0.1), _bf(rng, 2, N, 32, scale=0.1)
    cu, which = np.array([2, rows - 5, rows - 3], np.int32), np.array([1, 0], np.int32)
    if few:
        cu = np.array([2, 5, 8], np.int32)
    bank = T.Adapters(a.to(DEV), b.to(DEV))
    ctx.adapter_linear(bank, x[:, 8:8 + K], y[:, 16:16 + N], S.dev(cu), S.dev(which), out=out[:, 8:8 + N])
    want, room = _want(x[:, 8:8 + K].double().cpu().numpy(), y[:, 16:16 + N].double().cpu().numpy(), a.double().numpy(),
                       b.double().numpy(), np.ones(2), cu, which)
    got = out.double().cpu().numpy()
    mine = slice(cu[0], cu[-1])
    assert (np.abs(got[:, 8:8 + N] - want)[mine] <= room[mine]).all()
    got[mine, 8:8 + N] = 7
    assert (got == 7).all()


def test_ranks_are_filled_up(ctx):
    """Adapters of other ranks than the kernels take."""
    rng = np.random.default_rng(4)
    pairs = [(_bf(rng, r, 64), _bf(rng, 32, r)) for r in (1, 8, 20)]
    bank = T.Adapters.of([(a.to(DEV), b.to(DEV)) for a, b in pairs])
    assert bank.rank == 32
    x, y = _bf(rng, 9, 64), _bf(rng, 9, 32)
    cu, which = np.array([0, 3, 6, 9], np.int32), np.array([2, 0, 1], np.int32)
    out = ctx.adapter_linear(bank, x.to(DEV), y.to(DEV), S.dev(cu), S.dev(which))
    a, b = bank.a.double().cpu().numpy(), bank.b.double().cpu().numpy()
    want, room = _want(x.double().numpy(), y.double().numpy(), a, b, np.ones(3), cu, which)
    assert (np.abs(out.double().cpu().numpy() - want) <= room).all()
    for i, (p, q) in enumerate(pairs):
        r = p.shape[0]
        assert np.array_equal(a[i, :r], p.double().numpy()) and (a[i, r:] == 0).all()
        assert np.array_equal(b[i, :, :r], q.double().numpy()) and (b[i, :, r:] == 0).all()


@pytest.mark.parametrize("had", [32, 64, 128])
def test_transformed_rows(ctx, had):
    """Rows quantized after the block transform, with A turned to match, give x A^T: of INT8 codes to a
    half step of theirs and of A's bf16 (2^-8), which add up as independent errors."""
    rng = np.random.default_rng(had)
    M, K, N, R = 40, 256, 64, 16
    x, y = _bf(rng, M, K), torch.zeros(M, N, dtype=torch.bfloat16)
    a, b = _bf(rng, 1, R, K, scale=K ** -0.5), _bf(rng, 1, N, R)
    turned = ctx.adapter_rotate(a.to(DEV), had)
    H = O.sylvester_hadamard(had).astype(np.float64)
    want = (a.double().numpy().reshape(R, -1, had) @ H / had).reshape(1, R, K)
    # fp32 butterflies: log2(b) roundings of at most the block's absolute sum
    room = np.abs(want) * 2.0 ** -8 + np.repeat(np.abs(a.double().numpy()).reshape(1, R, -1, had).sum(3) / had, had, 2) * 8 * 2.0 ** -24
    assert (np.abs(turned.double().cpu().numpy() - want) <= room).all()
    q, s = ctx.hadamard_quant_act(x.to(DEV), had)
    out = ctx.adapter_linear(T.Adapters(turned, b.to(DEV)), q, y.to(DEV), S.dev(np.array([0, M], np.int32)),
                             S.dev(np.array([0], np.int32)), x_scale=s)
    ref = x.double().numpy() @ a[0].double().numpy().T @ b[0].double().numpy().T
    d = np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    # a code is off by a half step at most (rms 1 / sqrt(12)), the row's largest 127 of them being about
    # 3.3 of its rms: 0.0075; A's rounding 2^-8 / sqrt(3) at most; out's as much: 0.0085 together
    assert d < 0.012, d
    same = turned.clone()
    assert torch.equal(ctx.adapter_rotate(a.to(DEV), had, out=same), turned)


def test_beside_the_projection(ctx):
    """A projection of INT8 codes and adapters on the same codes: the sum of both products."""
    rng = np.random.default_rng(9)
    M, K, N, R, had = 37, 256, 96, 16, 64
    x, w = _bf(rng, M, K), _bf(rng, N, K, scale=K ** -0.5)
    a, b = _bf(rng, 2, R, K, scale=K ** -0.5), _bf(rng, 2, N, R, scale=0.3)
    weights = ctx.quantize_weights(w.to(DEV), had)
    q, s = ctx.hadamard_quant_act(x.to(DEV), had)
    y, _ = ctx.masked_qgemm(q, s, weights["w_q"], weights["w_scale"], 0)
    cu, which = np.array([0, 20, M], np.int32), np.array([1, 0], np.int32)
    turned = ctx.adapter_rotate(a.to(DEV), had)
    out = ctx.adapter_linear(T.Adapters(turned, b.to(DEV)), q, y, S.dev(cu), S.dev(which), x_scale=s, out=y.clone())
    want, room = _want(q.double().cpu().numpy() * s.double().cpu().numpy()[:, None], y.double().cpu().numpy(),
                       turned.double().cpu().numpy(), b.double().numpy(), np.ones(2), cu, which)
    assert (np.abs(out.double().cpu().numpy() - want) <= room).all()


def test_not_finite(ctx):
    """A row that is not finite makes NaN of itself alone."""
    rng = np.random.default_rng(10)
    x, y = _bf(rng, 20, 64), _bf(rng, 20, 32)
    a, b = _bf(rng, 1, 16, 64), _bf(rng, 1, 32, 16)
    bank = T.Adapters(a.to(DEV), b.to(DEV))
    cu, which = S.dev(np.array([0, 20], np.int32)), S.dev(np.array([0], np.int32))
    clean = ctx.adapter_linear(bank, x.to(DEV), y.to(DEV), cu, which)
    x[3, 5] = float("nan")
    out = ctx.adapter_linear(bank, x.to(DEV), y.to(DEV), cu, which)
    keep = torch.arange(20) != 3
    assert out[3].isnan().all() and torch.equal(out[keep.to(DEV)], clean[keep.to(DEV)])


def test_captured(ctx):
    rng = np.random.default_rng(11)
    x, y = _bf(rng, 64, 512).to(DEV), _bf(rng, 64, 320).to(DEV)
    bank = T.Adapters(_bf(rng, 5, 64, 512).to(DEV), _bf(rng, 5, 320, 64).to(DEV))
    cu, which = S.dev(np.arange(65, dtype=np.int32)), S.dev(rng.integers(0, 5, 64).astype(np.int32))
    ws, out = ctx.adapter_workspace(bank, x, 64), torch.empty_like(y)
    want = ctx.adapter_linear(bank, x, y, cu, which).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ctx.adapter_linear(bank, x, y, cu, which, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.adapter_linear(bank, x, y, cu, which, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        eager = ctx.adapter_linear(bank, x, y, cu, which)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)


@pytest.mark.parametrize("rank,fmt", [(16, "bf16"), (32, "int8"), (32, "mxfp4")])
def test_one_kernel_or_two_the_same_bits(ctx, rank, fmt):
    """Segments by themselves (one kernel) as all of them in one call (whose matrices are too many for that)."""
    rng = np.random.default_rng(rank)
    rows, K, N = 96, 2240, 6144
    x, xs, _ = _rows(rng, fmt, rows, K)
    y = _bf(rng, rows, N).to(DEV)
    bank = T.Adapters(_bf(rng, 5, rank, K, scale=K ** -0.5).to(DEV), _bf(rng, 5, N, rank).to(DEV))
    cu = np.array(sorted([0, rows] + list(rng.permutation(np.arange(1, rows))[:79])), np.int32)
    which = rng.integers(-1, 5, 80).astype(np.int32)
    out = ctx.adapter_linear(bank, x, y, S.dev(cu), S.dev(which), x_scale=xs)
    for i in range(0, 80, 8):
        a, b = int(cu[i]), int(cu[i + 8])
        part = ctx.adapter_linear(bank, x[a:b].contiguous(), y[a:b].contiguous(), S.dev(cu[i:i + 9] - a), S.dev(which[i:i + 8]),
                                  x_scale=None if xs is None else xs[a:b].contiguous())
        assert torch.equal(part, out[a:b]), (a, b)
