"""Paged MXFP4 cache: appended codes and scales bit for bit against the CPU oracle
(fp32 rotation, transform and quantization in the stated order), reads against
their values, everything else in the cache untouched."""
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


def _tables(P, half, seed):
    a = np.random.default_rng(seed).uniform(-50, 50, (P, half))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _arrays(cache):
    return {n: getattr(cache, n).cpu().numpy() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}


def _filled(pages, ps, heads, D, had):
    """A cache full of one byte, so that untouched bytes show."""
    c = T.KVCache.empty(pages, ps, heads, D, had, DEV)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(0x5A)
    return c


def _put(want, slot, ps, rows):
    for name, r in rows.items():
        want[name][slot // ps, :, slot % ps] = r


@pytest.mark.parametrize("tokens,heads,D,ps,had,rope,slack", [
    (1, 1, 64, 16, 32, "half", 0), (3, 2, 128, 16, 0, "pairs", 0), (37, 5, 72, 32, 32, "none", 0),
    (50, 3, 112, 64, 32, "half", 8), (17, 7, 40, 16, 0, "half", 16), (64, 4, 96, 128, 32, "pairs", 24),
    (5, 2, 8, 16, 32, "none", 0), (33, 3, 32, 16, 32, "pairs", 0), (129, 30, 64, 64, 32, "pairs", 0),
    (9, 2, 80, 16, 32, "part", 0),
])
def test_append_bit_exact(ctx, tokens, heads, D, ps, had, rope, slack):
    print(f"append {tokens}x{heads}x{D} ps {ps} had {had} rope {rope}", flush=True)
    rng = np.random.default_rng(tokens * 1000 + D)
    # k and v as slices of wider rows
    wide = torch.from_numpy(rng.standard_normal((tokens, 2 * heads * D + slack)).astype(np.float32))
    wide[0, :D] *= 1e-30                      # a block of tiny values
    wide[-1, heads * D:heads * D + D] = 0.0   # a zero block
    wide[tokens // 2, 0] = 3e30               # one large among small
    wide = wide.bfloat16()
    dev = wide.to(DEV)
    k, v = (dev[:, i * heads * D:(i + 1) * heads * D].unflatten(1, (heads, D)) for i in (0, 1))
    pages = (tokens + ps - 1) // ps + 2
    slots = rng.permutation(pages * ps)[:tokens].astype(np.int64)
    if tokens > 4:
        slots[1], slots[3] = -1, pages * ps   # padding and one past the end write nothing
    cache = _filled(pages, ps, heads, D, had)
    want = _arrays(cache)
    R = {"none": 0, "part": 16}.get(rope, D // 16 * 16)
    bits = S.bf16_bits(wide)
    kf = O.bf16_to_f32(bits[:, :heads * D]).reshape(tokens, heads, D)
    vf = O.bf16_to_f32(bits[:, heads * D:2 * heads * D]).reshape(tokens, heads, D)
    kw = {}
    if R:
        cos, sin = _tables(11, R // 2, D)
        pos = rng.integers(0, 11, tokens).astype(np.int32)
        inter = rope == "pairs"
        kf = B.rotate_f32(kf, cos, sin, pos, inter)
        kw = dict(rope=T.Rope(torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV), inter),
                  positions=torch.from_numpy(pos).to(DEV))
    ctx.kv_append(cache, k, v, torch.from_numpy(slots).to(DEV), **kw)
    kc, ks = B.mx_rows(kf, had)
    vc, vs = B.mx_rows(vf, had)
    for t in range(tokens):
        if 0 <= slots[t] < pages * ps:
            _put(want, slots[t], ps, {"k_codes": kc[t], "k_scales": ks[t], "v_codes": vc[t],
                                      "v_scales": vs[t]})
    got = _arrays(cache)
    for n in want:
        assert np.array_equal(got[n], want[n]), n
    # the read: values of the stored rows, turned back, rounded to bf16 once
    rk, rv = ctx.kv_read(cache, torch.from_numpy(slots).to(DEV))
    for r, c, e in ((rk, kc, ks), (rv, vc, vs)):
        val = B.unrotated(B.mx_values(c, e), had)[..., :D]
        val[(slots < 0) | (slots >= pages * ps)] = 0.0
        r = r.float().cpu().numpy().astype(np.float64)
        # 32 summands of at most 9 significant bits each, within one block: the fp32
        # butterflies err by at most 5 * 2^-24 of the block's absolute sum
        room = np.abs(val) * 2.0 ** -8
        if had:
            room = room + 5 * 2.0 ** -24 * _block_sum(c, e)[..., :D] / 32
        assert np.all(np.abs(r - val) <= room + 1e-38)


def _block_sum(codes, e8):
    a = np.abs(B.mx_values(codes, e8)).reshape(e8.shape + (32,)).sum(-1, keepdims=True)
    return np.broadcast_to(a, e8.shape + (32,)).reshape(codes.shape[:-1] + (-1,))


@pytest.mark.parametrize("heads", [1, 2, 3, 4, 6, 8, 12])
@pytest.mark.parametrize("D", [64, 96])
def test_head_tiles(ctx, heads, D):
    """Head counts of every kind of tile, tokens that end inside one; all ranges of exponents."""
    rng = np.random.default_rng(heads * 100 + D)
    tokens = 67
    bits = rng.integers(0, 1 << 16, (tokens, 2, heads, D), dtype=np.uint16)
    top = rng.integers(0, 255, (tokens, 2, heads, 1), dtype=np.uint16)      # a vector's exponents
    ex = np.maximum(top.astype(np.int64) - rng.integers(0, 9, bits.shape), 0).astype(np.uint16)
    ex = np.minimum(ex, 240)                                                # room for the sums of 32
    bits = (bits & 0x807F) | (ex << 7)
    t = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    f = O.bf16_to_f32(bits)
    for had in (0, 32):
        cache = _filled(6, 16, heads, D, had)
        slots = rng.permutation(96)[:tokens].astype(np.int64)
        want = _arrays(cache)
        ctx.kv_append(cache, t[:, 0].contiguous().to(DEV), t[:, 1].contiguous().to(DEV),
                      torch.from_numpy(slots).to(DEV))
        kc, ks = B.mx_rows(f[:, 0], had)
        vc, vs = B.mx_rows(f[:, 1], had)
        for i in range(tokens):
            _put(want, slots[i], 16, {"k_codes": kc[i], "k_scales": ks[i], "v_codes": vc[i], "v_scales": vs[i]})
        got = _arrays(cache)
        for n in want:
            assert np.array_equal(got[n], want[n]), (n, had)
        rk, rv = ctx.kv_read(cache, torch.from_numpy(slots).to(DEV))
        for r, c, e in ((rk, kc, ks), (rv, vc, vs)):
            val = B.unrotated(B.mx_values(c, e), had)[..., :D]
            room = np.abs(val) * 2.0 ** -8
            if had:
                room = room + 5 * 2.0 ** -24 * _block_sum(c, e)[..., :D] / 32
            r = r.float().cpu().numpy().astype(np.float64)
            assert np.all(np.abs(r - val) <= room + 1e-38)


def test_append_marks_what_is_not_finite(ctx):
    heads, D, ps = 2, 64, 16
    g = torch.Generator().manual_seed(3)
    k = torch.randn(6, heads, D, generator=g).bfloat16().to(DEV)
    v = torch.randn(6, heads, D, generator=g).bfloat16().to(DEV)
    k[1, 0, 5] = float("nan")
    v[2, 1, 63] = float("inf")
    k[3, 1] = 3e38            # finite, but its transform is not
    cache = T.KVCache.empty(1, ps, heads, D, 32, DEV)
    cos = torch.ones(4, 16, device=DEV)
    rope = T.Rope(cos, torch.zeros_like(cos))
    pos = torch.tensor([0, 1, 2, 3, 4, -1], dtype=torch.int32, device=DEV)   # rows 4 and 5: no such position
    slots = torch.arange(6, device=DEV)
    ctx.kv_append(cache, k, v, slots, rope=rope, positions=pos)
    bad = {(1, 0), (2, 1), (3, 1), (4, 0), (4, 1), (5, 0), (5, 1)}
    a = _arrays(cache)
    rk, rv = ctx.kv_read(cache, slots)
    for t in range(6):
        for h in range(heads):
            marked = (t, h) in bad
            assert np.all((a["k_scales"][0, h, t] == 255) == marked), (t, h)
            assert not np.any(a["v_scales"][0, h, t] == 255)
            assert bool(torch.isnan(rk[t, h]).all()) == marked
            if marked:
                assert not a["v_codes"][0, h, t].any() and not rv[t, h].any()


def test_append_past_4_gib(ctx):
    """Rows whose byte offset passes 32 bits."""
    heads, D, ps = 8, 128, 64
    pages = (5 << 30) // (heads * ps * (D // 2))
    cache = T.KVCache(*[torch.empty((pages, heads, ps, w), dtype=torch.uint8, device=DEV)
                        for w in (D // 2, D // 32, D // 2, D // 32)], head_dim=D, had_block=0)
    x = torch.randn(4, heads, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    slots = torch.tensor([pages * ps - 1, pages * ps - 17, 0, (1 << 32) // (heads * D // 2) + 3])
    ctx.kv_append(cache, x.to(DEV), x.flip(0).to(DEV), slots.to(DEV))
    rk, rv = ctx.kv_read(cache, slots.to(DEV))
    f = O.bf16_to_f32(S.bf16_bits(x))
    want = B.mx_values(*B.mx_rows(f, 0))
    assert np.array_equal(rk.float().cpu().numpy(), want)
    assert np.array_equal(rv.float().cpu().numpy(), want[::-1])


def test_append_of_nothing_and_streams(ctx):
    cache = _filled(2, 16, 2, 64, 32)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    ctx.kv_append(cache, e, e, torch.empty(0, dtype=torch.int64, device=DEV))
    assert ctx.kv_read(cache, torch.empty(0, dtype=torch.int64, device=DEV))[0].shape == (0, 2, 64)
    x = torch.randn(20, 2, 64, device=DEV).bfloat16()
    slots = torch.arange(20, device=DEV)
    ctx.kv_append(cache, x, x, slots)
    a = ctx.kv_read(cache, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _filled(2, 16, 2, 64, 32)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ctx.kv_append(other, x, x, slots)
        b = ctx.kv_read(other, slots)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_binding_refusals(ctx):
    cache = T.KVCache.empty(2, 16, 2, 64, 0, DEV)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    s = torch.arange(4, device=DEV)
    with pytest.raises(TypeError):
        ctx.kv_append(cache, x.float(), x, s)
    with pytest.raises(TypeError):
        ctx.kv_append(cache, x, x, s.int())
    with pytest.raises(ValueError):
        ctx.kv_append(cache, x, x[:3], s)
    with pytest.raises(ValueError):
        ctx.kv_append(cache, x.transpose(1, 2), x, s)
    with pytest.raises(ValueError):
        ctx.kv_append(cache, x, x, s[:2])
    with pytest.raises(T.TabitError) as e:      # token stride not a multiple of 8
        ctx.kv_append(cache, torch.zeros(4, 132, dtype=torch.bfloat16, device=DEV)[:, :128].unflatten(1, (2, 64)), x, s)
    assert e.value.status == T.ESHAPE
