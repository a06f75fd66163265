"""The fused norms' quantized outputs where h is not finite, very small, or shared by no sample."""
import numpy as np
import pytest
import torch

from oracle import tabit_oracle as O
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


def _inputs(M, H, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(M, H, generator=g).bfloat16().to(DEV) for _ in range(2)]


@pytest.mark.parametrize("H", [64, 640, 1536, 4096, 16384])
@pytest.mark.parametrize("pre", [T.NORM_NONE, T.NORM_LAYER, T.NORM_RMS])
def test_what_is_not_finite_stays_so_in_int8(ctx, H, pre):
    """A NaN or infinity in x or y: the row's scale is NaN and its codes are 0; other rows are the
    same bits as without it; a product with the row answers NaN."""
    for had in (0, 32, 64):
        print("block_norm int8", H, pre, had, flush=True)
        x, y = _inputs(14, H, H)
        use = dict(pre=pre, fmt=T.FMT_INT8, had_block=had)
        _, h, s = ctx.block_norm(x, y, **use)
        assert torch.isfinite(s).all()
        bad = {5: ("x", 3, "nan"), 7: ("y", H - 1, "inf"), 9: ("x", H // 2, "-inf"), 13: ("y", 0, "nan")}
        for row, (which, at, v) in bad.items():
            (x if which == "x" else y)[row, at] = float(v)
        _, g, t = ctx.block_norm(x, y, **use)
        rows = sorted(bad)
        good = [i for i in range(14) if i not in bad]
        assert torch.isnan(t[rows]).all() and not g[rows].any()
        assert torch.equal(h[good], g[good]) and torch.equal(s[good], t[good])
    w = ctx.quantize_weights(torch.randn(64, H, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV), 64)
    out = ctx.masked_qgemm(g, t, w["w_q"], w["w_scale"], 0)[0]
    assert torch.isnan(out[rows]).all() and torch.isfinite(out[good]).all()


@pytest.mark.parametrize("H", [64, 640, 4096, 16384])
@pytest.mark.parametrize("pre", [T.NORM_NONE, T.NORM_LAYER, T.NORM_RMS])
def test_what_is_not_finite_stays_so_in_mxfp4(ctx, H, pre):
    """The same in MXFP4, block by block: without a norm only the element's block is marked."""
    for had in (0, 32):
        print("block_norm mxfp4", H, pre, had, flush=True)
        x, y = _inputs(14, H, H + 1)
        use = dict(pre=pre, fmt=T.FMT_MXFP4, had_block=had)
        _, h, s = ctx.block_norm(x, y, **use)
        assert not (s == 255).any()
        bad = {5: ("x", 3, "nan"), 7: ("y", H - 1, "inf"), 9: ("x", H // 2, "-inf"), 13: ("y", 0, "nan")}
        for row, (which, at, v) in bad.items():
            (x if which == "x" else y)[row, at] = float(v)
        _, g, t = ctx.block_norm(x, y, **use)
        marked = torch.zeros_like(s, dtype=torch.bool)
        for row, (_, at, _v) in bad.items():
            # an infinity makes an RMS of infinity: what is finite becomes 0, and itself NaN
            one_block = pre == T.NORM_NONE or (pre == T.NORM_RMS and "inf" in _v)
            marked[row, at // 32 if one_block else slice(None)] = True
        assert torch.equal(t == 255, marked)
        assert not g.view(14, H // 32, 16)[marked].any()
        good = [i for i in range(14) if i not in bad]
        assert torch.equal(h[good], g[good]) and torch.equal(s[good], t[good])


@pytest.mark.parametrize("had", [0, 32, 128])
@pytest.mark.parametrize("e", [80, 93, 94, 115, 120, 121, 126, 130])
def test_int8_codes_of_very_small_rows(ctx, had, e):
    """Whole numbers times 2^-e, whose transform is exact: codes are rint(127 y / max|y|) (two fp32
    roundings of 2^-24 beside a tie) also where 127 / max|y| is past fp32, and nowhere clamped; scales
    are max|y| / 127 to fp32, whose smallest step is 2^-149."""
    for H in (128, 1536, 8192, 16384):
        rng = np.random.default_rng(H + e)
        c = rng.integers(-50, 51, (5, H)).astype(np.float64)
        c[1, 1:] = 0
        c[2] = 0
        x = torch.from_numpy(np.ldexp(c, -e)).bfloat16().to(DEV)
        assert np.array_equal(x.double().cpu().numpy(), np.ldexp(c, -e))
        _, h, s = ctx.block_norm(x, fmt=T.FMT_INT8, had_block=had, want_x=False)
        y = c
        if had:
            y = (c.reshape(5, -1, had) @ O.sylvester_hadamard(had).astype(np.float64)).reshape(5, H)
        a = np.abs(y).max(1, keepdims=True)
        v = np.divide(y * 127, a, out=np.zeros_like(y), where=a > 0)
        code = h.cpu().numpy().astype(np.float64)
        room = 127 * 2.0 ** -23
        assert np.all(np.abs(code - v) <= 0.5 + room)
        sure = np.abs(np.abs(v - np.floor(v)) - 0.5) > room
        assert np.array_equal(code[sure], np.rint(v)[sure]) and sure.mean() > 0.9
        want = np.ldexp(a[:, 0] / 127, -e)
        assert np.all(np.abs(s.double().cpu().numpy() - want) <= want * 2.0 ** -24 + 2.0 ** -150)
