"""The fused norms' quantized outputs where h is not finite, very small, or shared by no sample."""
import numpy as np
import pytest
import torch

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
