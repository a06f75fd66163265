"""The example block against the same block with its formats: INT8 codes of activations and weights,
MXFP4 keys and values, bf16 between the operators, sums and norms in fp64.

What differs: the attention's weights are rounded to bf16 (its output by 2^-8 of itself at most, about
2^-9 in the mean) and every value that lies near a rounding boundary may fall on its other side.  An
INT8 step is about 2^-5 of the mean element, so a difference d of a mean element changes a code with
chance 2^5 d, and codes that change by chance c differ by sqrt(c) steps: 2^-9 before a linear becomes
sqrt(2^-4) 2^-5 = 2^-7 behind it.  The attention's branch and the MLP's, whose input the first moves by a
gate of 0.2, are each off by about 2^-7 of themselves, so the change of the stream by less than 2^-5 of
itself (a wrong head, page, mask, gate or scale by its own size; the formats themselves by 0.1 to 0.2)."""
import numpy as np
import pytest
import torch

from examples import cached_block as E
from oracle import block_oracle as B
from oracle import tabit_oracle as O
import tabit_synth as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu


def _bf16(x):
    return O.bf16_to_f32(O.f64_to_bf16_bits(np.asarray(x, np.float64))).astype(np.float64)


def _codes(h, had):
    """INT8 codes and scales of fp64 rows after the block transform."""
    y = (h.reshape(len(h), -1, had) @ O.sylvester_hadamard(had).astype(np.float64)).reshape(h.shape)
    a = np.abs(y).max(1, keepdims=True)
    return np.clip(np.rint(y * 127 / a), -127, 127), a / 127


def _linear(codes, scale, w):
    return _bf16(codes @ w["w_q"].cpu().double().numpy().T * scale * w["w_scale"].cpu().double().numpy())


@pytest.mark.parametrize("q_heads,kv_heads,D,width,hidden,n", [
    (4, 2, 64, 256, 512, 100), (5, 1, 64, 320, 640, 45), (2, 2, 128, 256, 512, 33)])
def test_block_with_its_formats(q_heads, kv_heads, D, width, hidden, n):
    print("cached block", q_heads, kv_heads, D, width, n, flush=True)
    ctx = T.Context()
    b = E.Block(ctx, width, q_heads, kv_heads, D, hidden, 128)
    x16 = torch.randn(n, width, generator=torch.Generator().manual_seed(n)).bfloat16()
    half = n // 2                            # a chunk, then another behind it
    got = torch.cat([b.forward(x16[:half].to(E.DEV)), b.forward(x16[half:].to(E.DEV))]).double().cpu().numpy()
    x = O.bf16_to_f32(S.bf16_bits(x16)).astype(np.float64)
    m, nw = b.mod[0].double().cpu().numpy(), b.norm.double().cpu().numpy()
    _, h = B.block_norm(x, None, pre=B.LAYER, pre_w=nw[0], scale=m[1:2], shift=m[2:3])
    qkv = _linear(*_codes(h, E.HAD), b.qkv).reshape(n, q_heads + 2 * kv_heads, D)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
    cos, sin = b.rope.cos.cpu().numpy(), b.rope.sin.cpu().numpy()
    pos = np.arange(n)
    k = B.rotate_f32(k.astype(np.float32), cos, sin, pos, False)
    pages = (n + 15) // 16
    cache = {}
    for name, y in (("k", k), ("v", v.astype(np.float32))):
        for part, z in zip(("codes", "scales"), B.mx_rows(y, E.HAD)):
            full = np.zeros((pages * 16,) + z.shape[1:], np.uint8)
            full[:n] = z
            cache[f"{name}_{part}"] = full.reshape(pages, 16, kv_heads, -1).transpose(0, 2, 1, 3)
    a, _, _, _ = B.attention(q, cache, np.arange(pages)[None], [n], [0, n], D ** -0.5, True, D, E.HAD,
                             (cos, sin, pos, False))
    y = _linear(*_codes(_bf16(a).reshape(n, -1), E.HAD), b.out)
    x1, h = B.block_norm(x, y, B.RMS, nw[1], m[0:1], 1.0, B.LAYER, nw[2], m[4:5], m[5:6])
    x1 = _bf16(x1)
    up = _linear(*_codes(h, E.HAD), b.up)
    y = _linear(*_codes(_bf16(O.gelu_tanh_f64(up)), E.HAD), b.down)
    want, _ = B.block_norm(x1, y, B.RMS, nw[3], m[3:4], 1.0)
    err = np.linalg.norm(got - want) / np.linalg.norm(want - x)
    print("error of the change", err, flush=True)
    assert err <= 2.0 ** -5, err
    ctx.close()
