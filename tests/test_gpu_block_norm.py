"""Norms before and after a block, fused: bf16 results against fp64, quantized results
against the codes of the fp64 h wherever that is farther from a rounding boundary than
the kernel's fp32 arithmetic can err.

Error of the kernel's fp32 h: each mean or mean square of H terms errs by at most about
(log2(64) + 8 S) 2^-24 of the mean of absolute values in a sum over lanes of S slots of
eight; with the division, root, weight, scale, shift and gate products (about ten
rounded operations, relative 2^-24 of the terms they join) 64 * 2^-24 of the sum of the
absolute terms bounds it for every width used here."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import tabit_oracle as O
import tabit_synth as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


def _f64(t):
    return O.bf16_to_f32(S.bf16_bits(t)).astype(np.float64)


def _inputs(M, H, samples, seed, mean=0.2):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
    wide = 1.0 + 19.0 * (torch.rand(1, H, generator=g) < 0.02).float()
    t = dict(x=(2 * r(M, H) * wide + mean).bfloat16(), y=(r(M, H) * wide).bfloat16(),
             post_weight=(1 + 0.1 * r(H)).bfloat16(), pre_weight=(1 + 0.1 * r(H)).bfloat16())
    mod = (0.3 * r(max(samples, 1), 3, H)).bfloat16()
    t.update(gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2], mod=mod)
    return t


def _terms(x, y, post, gate, t, pre, want, ref):
    """Sum of the absolute terms of h and of x', per element."""
    rep = lambda a: np.repeat(a, x.shape[0] // a.shape[0], 0)      # noqa: E731
    ax = np.abs(t["res"] * x)
    if y is not None:
        ny = np.abs(B.norm(y, post, t["pw"], EPS))
        if post == B.LAYER:
            ny = ny + np.abs(y.mean(1, keepdims=True)) / np.sqrt(y.var(1, keepdims=True) + EPS) * (
                1 if t["pw"] is None else np.abs(t["pw"]))
        ax = ax + ny * (1 if gate is None else np.abs(rep(gate)))
    return ax


def _h_room(xr, ax, pre, prw, scale, shift):
    """Bound of the fp32 error of h, given x' (fp64), its absolute terms, and the norm."""
    rep = lambda a: np.repeat(a, xr.shape[0] // a.shape[0], 0)     # noqa: E731
    room = ax.copy()
    if pre == B.LAYER:
        room = room + np.abs(ax).mean(1, keepdims=True)
        rms = np.sqrt(xr.var(1, keepdims=True) + EPS)
    elif pre == B.RMS:
        rms = np.sqrt((xr * xr).mean(1, keepdims=True) + EPS)
    if pre != B.NONE:
        # an error of the statistic itself moves h in proportion
        rel = (room * np.abs(xr)).mean(1, keepdims=True) / (rms * rms) + 1
        room = (room + np.abs(B.norm(xr, pre, None, EPS)) * rms * rel) / rms
        room = room * (1 if prw is None else np.abs(prw))
    if scale is not None:
        room = room * np.abs(1 + rep(scale))
    if shift is not None:
        room = room + np.abs(rep(shift))
    return 64 * U * room


CASES = [
    # M, H, samples, post, pre, gate, scale/shift, weights, y, res
    (1, 32, 1, "rms", "rms", True, True, True, True, 1.0),
    (3, 64, 0, "none", "layer", False, False, False, True, 1.0),
    (5, 1152, 1, "none", "layer", True, True, False, True, 1.0),
    (6, 1152, 2, "rms", "layer", True, True, True, True, 0.9375),
    (4, 2240, 4, "rms", "rms", True, True, True, True, 1.0),
    (7, 1920, 1, "layer", "layer", True, True, True, True, 0.5),
    (2, 640, 0, "none", "rms", False, False, True, False, 1.0),
    (3, 96, 1, "layer", "none", True, True, True, True, -1.25),
    (2, 2560, 1, "none", "layer", True, True, False, True, 1.0),
    (3, 5120, 1, "rms", "layer", True, True, True, True, 1.0),
    (2, 7680, 2, "rms", "rms", True, True, True, True, 1.0),
    (2, 32768, 1, "layer", "layer", True, True, True, True, 1.0),
]
KIND = {"none": T.NORM_NONE, "layer": T.NORM_LAYER, "rms": T.NORM_RMS}


def _setup(case, seed=0, mean=0.2):
    M, H, samples, post, pre, gate, mod, weights, y, res = case
    t = _inputs(M, H, samples, M * 7 + H + seed, mean)
    use = dict(post=KIND[post], pre=KIND[pre], res_scale=res, eps=EPS)
    d = t["mod"].to(DEV)
    if y and post != "none" and weights:
        use["post_weight"] = t["post_weight"].to(DEV)
    if pre != "none" and weights:
        use["pre_weight"] = t["pre_weight"].to(DEV)
    if gate:
        use["gate"] = d[:, 0]
    if mod:
        use["scale"], use["shift"] = d[:, 1], d[:, 2]
    f = {n: _f64(t[n]) for n in ("x", "y", "post_weight", "pre_weight")}
    m = _f64(t["mod"].reshape(-1, H)).reshape(-1, 3, H)
    pw = f["post_weight"] if "post_weight" in use else None
    prw = f["pre_weight"] if "pre_weight" in use else None
    g, s, b = (m[:, 0] if gate else None), (m[:, 1] if mod else None), (m[:, 2] if mod else None)
    yy = f["y"] if y else None
    xr, hr = B.block_norm(f["x"], yy, KIND[post], pw, g, res, KIND[pre], prw, s, b, EPS)
    ax = _terms(f["x"], yy, KIND[post], g, {"res": res, "pw": pw}, KIND[pre], xr, hr)
    room_x = 64 * U * ax
    room_h = _h_room(xr, ax, KIND[pre], prw, s, b)
    args = (t["x"].to(DEV), t["y"].to(DEV) if y else None)
    return args, use, xr, hr, room_x, room_h


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("case", CASES)
def test_bf16(ctx, case):
    print("block_norm", case, flush=True)
    args, use, xr, hr, rx, rh = _setup(case)
    x, h, s = ctx.block_norm(*args, **use)
    assert s is None
    assert np.all(np.abs(_host(x) - xr) <= rx + np.abs(xr) * 2.0 ** -8 + 1e-38)
    assert np.all(np.abs(_host(h) - hr) <= rh * 1.01 + np.abs(hr) * 2.0 ** -8 + 1e-38)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("b", [0, 32, 64, 128])
def test_int8(ctx, case, b):
    M, H = case[:2]
    if b and H % b:
        pytest.skip("width is not a multiple of the block")
    print("block_norm int8", case, b, flush=True)
    args, use, xr, hr, rx, rh = _setup(case)
    x, h, top = ctx.block_norm(*args, fmt=T.FMT_INT8, had_block=b, **use)
    y, room = hr, rh
    if b:
        n = int(np.log2(b))
        had = O.sylvester_hadamard(b).astype(np.float64)
        y = (hr.reshape(M, -1, b) @ had).reshape(M, H)
        room = np.repeat((rh + n * U * np.abs(hr)).reshape(M, -1, b).sum(2), b, 1)
    a = np.abs(y).max(1, keepdims=True)
    ra = room.max(1, keepdims=True)                     # error of the largest magnitude
    assert np.all(np.abs(top.cpu().numpy().astype(np.float64)[:, None] - a / 127) <= (ra + 4 * U * a) / 127)
    v = y * 127 / a
    slip = (room + np.abs(y) * (ra / a + 4 * U)) * 127 / a
    code = h.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(code - v) <= 0.5 + slip) and np.abs(code).max() <= 127
    # away from a tie the code is the nearest whole number
    sure = np.abs(np.abs(v - np.floor(v)) - 0.5) > slip
    assert sure.mean() > 0.9
    assert np.array_equal(code[sure], np.clip(np.rint(v), -127, 127)[sure])
    assert np.all(np.abs(_host(x) - xr) <= rx + np.abs(xr) * 2.0 ** -8 + 1e-38)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("b", [0, 32])
def test_mxfp4(ctx, case, b):
    M, H = case[:2]
    print("block_norm mxfp4", case, b, flush=True)
    args, use, xr, hr, rx, rh = _setup(case)
    x, h, e8 = ctx.block_norm(*args, fmt=T.FMT_MXFP4, had_block=b, want_x=False, **use)
    assert x is None
    y, room = hr, rh
    if b:
        y = B.hadamard_blocks(hr)
        room = np.repeat((rh + 5 * U * np.abs(hr)).reshape(M, -1, 32).sum(2), 32, 1)
    e = e8.cpu().numpy().astype(np.int64)
    a, ra = np.abs(y).reshape(M, -1, 32).max(2), room.reshape(M, -1, 32).max(2)
    X = lambda v: np.floor(np.log2(v)).astype(np.int64) - 2 + 127     # noqa: E731
    assert np.all((e >= X(a - ra)) & (e <= X(a + ra)))
    val = O.mx_unpack(h.cpu().numpy(), e8.cpu().numpy()).astype(np.float64)
    unit = np.repeat(2.0 ** (e - 127.0), 32, 1)
    lo, hi = np.abs(y) - room, np.abs(y) + room
    near = lambda v: O.e2m1_decode(O.e2m1_encode((v / unit).astype(np.float64))) * unit   # noqa: E731
    assert np.all((np.abs(val) >= near(np.maximum(lo, 0))) & (np.abs(val) <= near(hi)))
    sure = np.abs(y) > room
    assert np.all((np.sign(val) == np.sign(y))[sure & (val != 0)])


def test_large_common_mean(ctx):
    """Values whose spread is a thousandth of their mean: centred before they are squared."""
    args, use, xr, hr, rx, rh = _setup((4, 1152, 1, "none", "layer", False, False, False, False, 1.0), mean=300.0)
    x, h, _ = ctx.block_norm(*args, **use)
    assert np.all(np.abs(_host(h) - hr) <= rh * 1.01 + np.abs(hr) * 2.0 ** -8)


def test_zero_rows_and_extremes(ctx):
    H = 1152
    x = torch.zeros(3, H, dtype=torch.bfloat16, device=DEV)
    x[1] = 1e-30
    x[2] = 1e15
    for pre in (T.NORM_LAYER, T.NORM_RMS):
        for fmt in (T.FMT_BF16, T.FMT_INT8, T.FMT_MXFP4):
            _, h, s = ctx.block_norm(x, pre=pre, fmt=fmt)
            assert not h[0].any()
            if fmt == T.FMT_INT8:
                assert s[0] == 0 and torch.isfinite(s).all()
            if fmt == T.FMT_BF16:
                assert torch.isfinite(h).all()
    _, h, _ = ctx.block_norm(x, pre=T.NORM_RMS)
    assert torch.allclose(h[2].float(), torch.ones(H, device=DEV), atol=2 ** -8)


def test_equals_the_chain_of_quantizer(ctx):
    """Without norms the INT8 and MXFP4 outputs are tabit_hadamard_quant_act's of a bf16 x."""
    x = S.gen_activation(33, 1920, seed=4).to(DEV)
    for fmt, b in ((T.FMT_INT8, 0), (T.FMT_INT8, 64), (T.FMT_INT8, 128), (T.FMT_MXFP4, 0), (T.FMT_MXFP4, 32)):
        q, s = ctx.hadamard_quant_act(x, b, fmt)
        _, h, hs = ctx.block_norm(x, fmt=fmt, had_block=b, want_x=False)
        assert torch.equal(q, h) and torch.equal(s, hs)


def test_in_place_empty_and_odd_rows(ctx):
    for M in (0, 1, 2, 3, 255, 257):
        t = _inputs(M, 320, 1, M)
        x, y = t["x"].to(DEV), t["y"].to(DEV)
        a, h, _ = ctx.block_norm(x, y, post=T.NORM_RMS, pre=T.NORM_LAYER)
        assert a.shape == (M, 320) and h.shape == (M, 320)
        b, h2, _ = ctx.block_norm(x, y, post=T.NORM_RMS, pre=T.NORM_LAYER, x_out=x)
        assert b.data_ptr() == x.data_ptr() and torch.equal(a, x) and torch.equal(h, h2)
        only, none, _ = ctx.block_norm(x, y, want_h=False)
        assert none is None and only.shape == (M, 320)


@pytest.mark.parametrize("M,H,samples", [
    (9000, 512, 3), (7000, 1024, 7), (5000, 1536, 5), (5000, 2048, 4), (1700, 4096, 17), (1100, 8192, 11),
    (40, 16384, 2), (9, 32768, 3),
])
def test_a_row_does_not_depend_on_the_others(ctx, M, H, samples):
    """Enough rows for runs that end inside a sample: each sample by itself gives the same bits."""
    print("block_norm runs", M, H, samples, flush=True)
    t = _inputs(M, H, samples, H)
    x, y, m = t["x"].to(DEV), t["y"].to(DEV), t["mod"].to(DEV)
    w, n = t["post_weight"].to(DEV), M // samples
    use = dict(post=T.NORM_RMS, post_weight=w, pre=T.NORM_LAYER, fmt=T.FMT_INT8, had_block=32)
    a, h, s = ctx.block_norm(x, y, gate=m[:, 0], scale=m[:, 1], shift=m[:, 2], **use)
    for i in range(samples):
        for r in (slice(i * n, i * n + n // 2), slice(i * n + n // 2, i * n + n)):
            a1, h1, s1 = ctx.block_norm(x[r], y[r], gate=m[i:i + 1, 0], scale=m[i:i + 1, 1],
                                        shift=m[i:i + 1, 2], **use)
            assert torch.equal(a[r], a1) and torch.equal(h[r], h1) and torch.equal(s[r], s1), (i, r)


@pytest.mark.parametrize("H", [64, 1536, 4096, 16384])
def test_not_a_number_stays_in_its_row(ctx, H):
    t = _inputs(12, H, 1, 3)
    x, y = t["x"].to(DEV), t["y"].to(DEV)
    use = dict(post=T.NORM_RMS, pre=T.NORM_LAYER)
    a, h, _ = ctx.block_norm(x, y, **use)
    x[5, 3], y[7, H - 1] = float("nan"), float("inf")
    b, g, _ = ctx.block_norm(x, y, **use)
    good = [i for i in range(12) if i not in (5, 7)]
    assert torch.equal(a[good], b[good]) and torch.equal(h[good], g[good])
    assert torch.isnan(g[5]).all() and torch.isnan(g[7]).all()
    assert torch.isnan(b[5]).sum() == 1 and torch.isnan(b[7]).any()


def test_binding_refusals(ctx):
    x = torch.zeros(6, 64, dtype=torch.bfloat16, device=DEV)
    m = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        ctx.block_norm(x.float())
    with pytest.raises(TypeError):
        ctx.block_norm(x, scale=m.float(), pre=T.NORM_RMS)
    with pytest.raises(ValueError):
        ctx.block_norm(x, x[:3])
    with pytest.raises(ValueError):
        ctx.block_norm(x, scale=m.repeat(2, 1), pre=T.NORM_RMS)       # 6 rows, 4 samples
    with pytest.raises(ValueError):
        ctx.block_norm(x, scale=m, shift=m[:1], pre=T.NORM_RMS)
    with pytest.raises(T.TabitError) as e:
        ctx.block_norm(x, gate=m)                                     # a gate without y
    assert e.value.status == T.EINVAL
