"""The example block: norms, quantized products, cache and attention used together.

Token by token against one chunk: every operator works row by row, so the two differ by the
attention's rounding (weights and outputs to bf16, 2^-9 of an output at most, half that in the
mean) and by INT8 codes that this moves over a rounding boundary: a step is 1/127 of the row's
largest element, about 2^-5 of the mean element, and an element that moves by a part d of a step
changes its code with chance d, so codes move by d of a step in the mean and the relative error
sqrt(d / 12) of a step at worst: under 2^-7 of the stream a block, with two blocks under 2^-5.

Against fp64: the same block with exact products and attention.  The 4-bit keys and values err
by about 0.1 of an element (E2M1 steps of 1/2 to 2 over values up to 6), so scores of order one
by 0.1, weights by 0.1 of themselves, and the attention's output by about 0.15 of itself; the
MLP's input, a stream that the attention moves by a gate of 0.2, by 0.03; the 8-bit codes of five
products add about 2^-7 each.  That is under 0.25 of the stream's change; a wrong rotation, mask,
page or modulation errs by the change's own size.
"""
import numpy as np
import pytest
import torch

from examples import cached_block as E
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [
    dict(width=256, q_heads=4, kv_heads=2, head_dim=64, hidden=512, prompt=70, tokens=6),
    dict(width=320, q_heads=5, kv_heads=1, head_dim=64, hidden=640, prompt=33, tokens=3),
])
def test_token_by_token_is_the_chunk(shape):
    print("cached block", shape, flush=True)
    whole, step, _ = E.run(**shape)
    assert torch.isfinite(whole.float()).all()
    p = shape["prompt"]
    d = (whole.double() - step.double()).norm() / whole.double().norm()
    assert d <= 2.0 ** -5, d
    assert step.shape == whole.shape and not torch.equal(whole[:p], whole[1:p + 1])


def _values(w):
    """The weights that int8 codes stand for (their block rotation undone)."""
    c = w["w_q"].cpu().double() * w["w_scale"].cpu().double()[:, None]
    h = torch.ones(1, 1, dtype=torch.float64)
    while h.shape[0] < E.HAD:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return (c.reshape(c.shape[0], -1, E.HAD) @ h).reshape(c.shape)


def test_block_against_fp64():
    ctx = T.Context()
    b = E.Block(ctx, 256, 4, 2, 64, 512, 100)
    x = torch.randn(100, 256, generator=torch.Generator().manual_seed(2)).bfloat16()
    got = b.forward(x.to(E.DEV)).cpu().double()
    m, nw = b.mod[0].cpu().double(), b.norm.cpu().double()
    ln = lambda t: (t - t.mean(1, keepdim=True)) / (t.var(1, unbiased=False, keepdim=True) + 1e-6).sqrt()   # noqa: E731
    rms = lambda t: t / ((t * t).mean(1, keepdim=True) + 1e-6).sqrt()      # noqa: E731
    x = x.double()
    qkv = (ln(x) * nw[0] * (1 + m[1]) + m[2]) @ _values(b.qkv).T
    q, k, v = qkv.unflatten(1, (8, 64)).split([4, 2, 2], 1)
    c, s = (t.cpu().double()[:100, None] for t in (b.rope.cos, b.rope.sin))

    def turn(t):
        lo, hi = t[..., :32], t[..., 32:]
        return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)

    q, k = turn(q), turn(k).repeat_interleave(2, 1)
    sc = torch.einsum("ihd,jhd->hij", q, k) / 8.0
    sc = sc.masked_fill(~torch.ones(100, 100).tril().bool(), -np.inf)
    a = torch.einsum("hij,jhd->ihd", sc.softmax(-1), v.repeat_interleave(2, 1)).flatten(1)
    x1 = x + m[0] * rms(a @ _values(b.out).T) * nw[1]
    h = (ln(x1) * nw[2] * (1 + m[4]) + m[5]) @ _values(b.up).T
    want = x1 + m[3] * rms(torch.nn.functional.gelu(h, approximate="tanh") @ _values(b.down).T) * nw[3]
    err = (got - want).norm() / (want - x).norm()
    assert err <= 0.25, err
    with pytest.raises(ValueError):
        b.forward(torch.zeros(1, 256, dtype=torch.bfloat16, device=E.DEV))     # the cache is full
    ctx.close()
