"""The paged cache with the largest and smallest values it holds."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import tabit_oracle as O
import tabit_synth as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("size", [3e38, 1e38, 2e37, 1e-37, 1e-38])
def test_one_large_element_is_read_back(ctx, D, size):
    """A single element of nearly the largest bf16: its transform is 32 times it before the division.
    The read is that of the stored codes, bit for bit but for fp32 sums (5 * 2^-24 of the block's
    absolute sum over 32) and the rounding to bf16 (2^-8; 2^-134 for the smallest)."""
    rng = np.random.default_rng(D)
    for at in (0, 5, D - 1):
        x = torch.zeros(3, 2, D)
        x[:, :, at] = torch.from_numpy(rng.choice([-1.0, 1.0, 0.75], (3, 2)) * size).float()
        x = x.bfloat16()
        cache = T.KVCache.empty(1, 16, 2, D, 32, DEV)
        slots = torch.tensor([3, 0, 9], device=DEV)
        ctx.kv_append(cache, x.to(DEV), x.flip(0).to(DEV), slots)
        rk, rv = ctx.kv_read(cache, slots)
        f = O.bf16_to_f32(S.bf16_bits(x))
        codes, e8 = B.mx_rows(f, 32)
        vals = B.mx_values(codes, e8)
        want = B.unrotated(vals, 32)[..., :D]
        total = np.repeat(np.abs(vals).reshape(3, 2, -1, 32).sum(3) / 32, 32, 2)[..., :D]
        room = np.abs(want) * 2.0 ** -8 + 5 * 2.0 ** -24 * total + 2.0 ** -134
        for r, w, m in ((rk, want, room), (rv, want[::-1], room[::-1])):
            r = r.double().cpu().numpy()
            assert np.isfinite(r).all() and np.all(np.abs(r - w) <= m), (at, r[0, 0, :4], w[0, 0, :4])
