"""Argument checks of the cache, attention and block-norm entry points: every refusal
comes before the first HIP call, so these run without a GPU."""
import ctypes

import pytest

import timestep_adaptive_bit_amd as T
from timestep_adaptive_bit_amd import _lib as L

FAKE = 0x10000        # 16-byte aligned, never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def lib():
    return T.load()


@pytest.fixture
def ctx():
    c = T.Context()
    yield c
    c.close()


def _cache(**kw):
    a = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, num_pages=4, page_size=16,
             num_kv_heads=2, head_dim=64, had_block=32)
    a.update(kw)
    return L._KvCache(*[a[n] for n, _ in L._KvCache._fields_])


def _rope(**kw):
    a = dict(cos=FAKE, sin=FAKE, num_positions=8, rope_dim=64, interleaved=0)
    a.update(kw)
    return L._Rope(*[a[n] for n, _ in L._Rope._fields_])


CACHE_REFUSALS = [
    (dict(head_dim=0), T.ESHAPE), (dict(head_dim=60), T.ESHAPE), (dict(head_dim=136), T.ESHAPE),
    (dict(num_kv_heads=0), T.ESHAPE), (dict(num_kv_heads=65536), T.ESHAPE),
    (dict(page_size=8), T.ESHAPE), (dict(page_size=48), T.ESHAPE), (dict(page_size=1 << 21), T.ESHAPE),
    (dict(num_pages=-1), T.ESHAPE), (dict(had_block=64), T.ERANGE), (dict(k_codes=None), T.EINVAL),
    (dict(v_scales=None), T.EINVAL), (dict(v_codes=FAKE + 8), T.EALIGN), (dict(k_scales=FAKE + 2), T.EALIGN),
]


def _append(lib, ctx, cache=None, k=FAKE, ks=128, v=FAKE, vs=128, n=3, slots=FAKE, rope=None, pos=None):
    c = cache if cache is not None else _cache()
    return lib.tabit_kv_append(ctx.handle, ctypes.addressof(c), k, ks, v, vs, n, slots,
                               ctypes.addressof(rope) if rope is not None else None, pos, None)


@pytest.mark.parametrize("kw,want", CACHE_REFUSALS)
def test_cache_refusals(lib, ctx, kw, want):
    c = _cache(**kw)
    assert _append(lib, ctx, cache=c) == want
    assert lib.tabit_kv_read(ctx.handle, ctypes.addressof(c), FAKE, 3, FAKE, FAKE, None) == want
    a = L._KvAttentionArgs()
    assert lib.tabit_kv_attention(ctx.handle, ctypes.addressof(c), ctypes.addressof(a), None) == want
    assert ctx.last_error() != ""


def test_append_refusals(lib, ctx):
    assert lib.tabit_kv_append(None, None, FAKE, 128, FAKE, 128, 1, FAKE, None, None, None) == T.EINVAL
    assert lib.tabit_kv_append(ctx.handle, None, FAKE, 128, FAKE, 128, 1, FAKE, None, None, None) == T.EINVAL
    cases = [
        (dict(n=-1), T.ESHAPE), (dict(k=None), T.EINVAL), (dict(v=None), T.EINVAL),
        (dict(slots=None), T.EINVAL), (dict(ks=120), T.ESHAPE), (dict(vs=132), T.ESHAPE),
        (dict(k=FAKE + 8), T.EALIGN), (dict(slots=FAKE + 4), T.EALIGN),
        (dict(rope=_rope(), pos=None), T.EINVAL), (dict(rope=_rope(cos=None), pos=FAKE), T.EINVAL),
        (dict(rope=_rope(rope_dim=24), pos=FAKE), T.ESHAPE),
        (dict(rope=_rope(rope_dim=80), pos=FAKE), T.ESHAPE),
        (dict(rope=_rope(num_positions=0), pos=FAKE), T.ESHAPE),
        (dict(rope=_rope(sin=FAKE + 4), pos=FAKE), T.EALIGN),
        (dict(n=0), T.OK), (dict(cache=_cache(num_pages=0)), T.OK),
    ]
    for kw, want in cases:
        assert _append(lib, ctx, **kw) == want, (kw, ctx.last_error())


def test_read_refusals(lib, ctx):
    c = _cache()

    def r(slots=FAKE, n=2, k=FAKE, v=FAKE):
        return lib.tabit_kv_read(ctx.handle, ctypes.addressof(c), slots, n, k, v, None)
    assert r(slots=None) == T.EINVAL
    assert r(k=None) == T.EINVAL
    assert r(n=-1) == T.ESHAPE
    assert r(v=FAKE + 8) == T.EALIGN
    assert r(n=0) == T.OK


def _attention(lib, ctx, rope=None, cache=None, **kw):
    a = dict(q=FAKE, q_stride=512, num_tokens=5, num_q_heads=8, cu_q=FAKE, num_seqs=2, max_q=3,
             block_table=FAKE, table_stride=4, kv_lens=FAKE, max_kv=64, scale=0.125, causal=1,
             rope=None if rope is None else ctypes.addressof(rope), positions=FAKE, out=FAKE, lse=None,
             ws=FAKE, ws_bytes=0)
    a.update(kw)
    c = cache or _cache()
    s = L._KvAttentionArgs(*[a[n] for n, _ in L._KvAttentionArgs._fields_])
    return lib.tabit_kv_attention(ctx.handle, ctypes.addressof(c), ctypes.addressof(s), None)


def test_attention_refusals(lib, ctx):
    cases = [
        (dict(num_tokens=-1), T.ESHAPE), (dict(num_seqs=-1), T.ESHAPE), (dict(max_q=-1), T.ESHAPE),
        (dict(max_kv=-1), T.ESHAPE), (dict(num_q_heads=7), T.ESHAPE), (dict(num_q_heads=0), T.ESHAPE),
        (dict(num_seqs=65536), T.ESHAPE), (dict(q=None), T.EINVAL), (dict(out=None), T.EINVAL),
        (dict(cu_q=None), T.EINVAL), (dict(kv_lens=None), T.EINVAL), (dict(block_table=None), T.EINVAL),
        (dict(max_kv=65), T.ESHAPE), (dict(table_stride=0), T.ESHAPE), (dict(q_stride=504), T.ESHAPE),
        (dict(q_stride=516), T.ESHAPE), (dict(scale=float("nan")), T.EINVAL),
        (dict(scale=float("inf")), T.EINVAL), (dict(q=FAKE + 8), T.EALIGN), (dict(out=FAKE + 2), T.EALIGN),
        (dict(lse=FAKE + 2), T.EALIGN), (dict(ws=FAKE + 4), T.EALIGN),
        (dict(rope=_rope(), positions=None), T.EINVAL),
        (dict(max_q=1 << 30), T.ESHAPE),
        (dict(num_tokens=0), T.OK), (dict(num_seqs=0), T.OK), (dict(max_q=0), T.OK),
    ]
    for kw, want in cases:
        assert _attention(lib, ctx, **kw) == want, (kw, ctx.last_error())
    # a long cache read by one row is split and needs its workspace
    need = lib.tabit_kv_attention_workspace_bytes(1, 8, 2, 64, 1, 1, 4096)
    assert need > 0
    long = dict(num_tokens=1, num_seqs=1, max_q=1, max_kv=4096, table_stride=256)
    assert _attention(lib, ctx, ws=None, **long) == T.EINVAL
    assert _attention(lib, ctx, ws_bytes=need - 1, **long) == T.ESHAPE
    assert lib.tabit_kv_attention(ctx.handle, ctypes.addressof(_cache()), None, None) == T.EINVAL


def test_attention_workspace_bytes(lib):
    ws = lib.tabit_kv_attention_workspace_bytes
    for bad in ((0, 8, 2, 64, 1, 1, 64), (1, 7, 2, 64, 1, 1, 64), (1, 8, 2, 64, 0, 1, 64),
                (1, 8, 2, 64, 1, 1, 0)):
        assert ws(*bad) == 0
    # rows of Dp sums and two statistics for each split
    n = ws(1, 32, 8, 72, 1, 1, 131072)
    assert n % (32 * (96 + 2) * 4) == 0 and 2 <= n // (32 * (96 + 2) * 4) <= 128


def _norm(lib, ctx, **kw):
    a = dict(x=FAKE, y=FAKE, rows=4, width=64, post_kind=T.NORM_RMS, pre_kind=T.NORM_LAYER,
             post_weight=FAKE, pre_weight=FAKE, gate=FAKE, scale=FAKE, shift=FAKE, mod_stride=64,
             num_samples=2, rows_per_sample=2, res_scale=1.0, eps=1e-6, x_out=FAKE, h=FAKE,
             h_scale=FAKE, fmt=T.FMT_INT8, had_block=32)
    a.update(kw)
    s = L._BlockNormArgs(*[a[n] for n, _ in L._BlockNormArgs._fields_])
    return lib.tabit_block_norm(ctx.handle, ctypes.addressof(s), None)


def test_block_norm_refusals(lib, ctx):
    none = dict(post_kind=T.NORM_NONE, post_weight=None, gate=None)
    cases = [
        (dict(x=None), T.EINVAL), (dict(rows=-1), T.ESHAPE), (dict(width=48), T.ESHAPE),
        (dict(width=0), T.ESHAPE), (dict(width=32800), T.ESHAPE), (dict(post_kind=3), T.EINVAL),
        (dict(pre_kind=-1), T.EINVAL), (dict(y=None), T.EINVAL),
        (dict(y=None, **{**none, "gate": FAKE}), T.EINVAL),
        (dict(post_kind=T.NORM_NONE), T.EINVAL), (dict(pre_kind=T.NORM_NONE), T.EINVAL),
        (dict(x_out=None, h=None), T.EINVAL), (dict(h=None), T.EINVAL),
        (dict(res_scale=float("nan")), T.EINVAL), (dict(eps=-1.0), T.EINVAL),
        (dict(eps=float("nan")), T.EINVAL), (dict(fmt=3), T.EINVAL), (dict(had_block=16), T.ERANGE),
        (dict(fmt=T.FMT_BF16), T.ERANGE), (dict(fmt=T.FMT_MXFP4, had_block=64), T.ERANGE),
        (dict(had_block=128), T.ESHAPE), (dict(h_scale=None), T.EINVAL),
        (dict(rows_per_sample=0), T.ESHAPE), (dict(num_samples=1), T.ESHAPE),
        (dict(mod_stride=56), T.ESHAPE), (dict(mod_stride=68), T.ESHAPE),
        (dict(gate=FAKE + 8), T.EALIGN), (dict(h=FAKE + 8), T.EALIGN), (dict(x_out=FAKE + 2), T.EALIGN),
        (dict(h_scale=FAKE + 2), T.EALIGN), (dict(rows=0), T.OK),
    ]
    for kw, want in cases:
        assert _norm(lib, ctx, **kw) == want, (kw, ctx.last_error())
    assert lib.tabit_block_norm(ctx.handle, None, None) == T.EINVAL


def test_binding_takes_gpu_tensors_only():
    import torch
    z = torch.zeros(1, 1, 16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        T.KVCache(z, z, z, z, head_dim=64)
    with pytest.raises(ValueError):
        T.Rope(torch.zeros(2, 8), torch.zeros(2, 8))
