"""Argument checks of the entry points for serving many requests: every refusal comes before the first HIP
call, so these run without a GPU."""
import ctypes

import pytest
import torch

import timestep_adaptive_bit_amd as T
from timestep_adaptive_bit_amd import _lib as L

FAKE = 0x10000        # 16-byte aligned, never dereferenced (validation fails first)
BIG = 1 << 62         # bytes of a workspace that is large enough


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


CACHE_REFUSALS = [
    (dict(head_dim=60), T.ESHAPE), (dict(num_kv_heads=0), T.ESHAPE), (dict(page_size=48), T.ESHAPE),
    (dict(num_pages=-1), T.ESHAPE), (dict(had_block=64), T.ERANGE), (dict(k_codes=None), T.EINVAL),
    (dict(v_codes=FAKE + 8), T.EALIGN), (dict(k_scales=FAKE + 2), T.EALIGN),
]


def _args(**kw):
    a = dict(q=FAKE, q_stride=512, num_tokens=5, num_q_heads=8, cu_q=FAKE, num_seqs=2, max_q=3,
             block_table=FAKE, table_stride=4, kv_lens=FAKE, max_kv=64, scale=0.125, causal=0, rope=None,
             positions=FAKE, out=FAKE, lse=None, ws=None, ws_bytes=0)
    a.update(kw)
    return L._KvAttentionArgs(*[a[n] for n, _ in L._KvAttentionArgs._fields_])


def _tree(lib, ctx, cache=None, mask=FAKE, words=1, **kw):
    c, a = cache or _cache(), _args(**kw)
    return lib.tabit_kv_tree_attention(ctx.handle, ctypes.addressof(c), ctypes.addressof(a), mask, words, None)


def _weigh(lib, ctx, cache=None, sums=FAKE, **kw):
    c, a = cache or _cache(), _args(**{"out": None, **kw})
    return lib.tabit_kv_weigh(ctx.handle, ctypes.addressof(c), ctypes.addressof(a), sums, None)


def _evict(lib, ctx, cache=None, **kw):
    a = dict(sums=FAKE, table=FAKE, stride=4, lens=FAKE, seqs=2, max_kv=64, budget=8, sinks=1, recent=2, keep=FAKE,
             new=FAKE, ws=None, ws_bytes=0)
    a.update(kw)
    c = cache or _cache()
    return lib.tabit_kv_evict(ctx.handle, ctypes.addressof(c), *a.values(), None)


def _compact(lib, ctx, cache=None, **kw):
    a = dict(table=FAKE, stride=4, seqs=2, keep=FAKE, heads=2, most=8, counts=FAKE, starts=None, sums=None, ws=None,
             ws_bytes=0)
    a.update(kw)
    c = cache or _cache()
    return lib.tabit_kv_compact(ctx.handle, ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("kw,want", CACHE_REFUSALS)
def test_cache_refusals(lib, ctx, kw, want):
    for call in (_tree, _weigh, _evict, _compact):
        assert call(lib, ctx, cache=_cache(**kw)) == want, call
        assert ctx.last_error() != ""


ROWS = [
    (dict(num_tokens=-1), T.ESHAPE), (dict(num_seqs=-1), T.ESHAPE), (dict(max_q=-1), T.ESHAPE),
    (dict(max_kv=-1), T.ESHAPE), (dict(num_q_heads=7), T.ESHAPE), (dict(num_seqs=65536), T.ESHAPE),
    (dict(q=None), T.EINVAL), (dict(cu_q=None), T.EINVAL), (dict(kv_lens=None), T.EINVAL),
    (dict(block_table=None), T.EINVAL), (dict(max_kv=65), T.ESHAPE), (dict(q_stride=504), T.ESHAPE),
    (dict(q_stride=516), T.ESHAPE), (dict(scale=float("nan")), T.EINVAL), (dict(q=FAKE + 8), T.EALIGN),
    (dict(lse=FAKE + 2), T.EALIGN), (dict(ws=FAKE + 4), T.EALIGN),
    (dict(num_tokens=0), T.OK), (dict(num_seqs=0), T.OK), (dict(max_q=0), T.OK),
]


@pytest.mark.parametrize("kw,want", ROWS)
def test_row_refusals(lib, ctx, kw, want):
    assert _tree(lib, ctx, **kw) == want
    assert _weigh(lib, ctx, **kw) == want


def test_tree_refusals(lib, ctx):
    cases = [(dict(out=None), T.EINVAL), (dict(causal=1), T.EINVAL), (dict(mask=None), T.EINVAL), (dict(words=0), T.ESHAPE),
             (dict(max_q=65), T.ESHAPE), (dict(max_q=8193, words=200), T.ESHAPE), (dict(mask=FAKE + 4), T.EALIGN),
             (dict(out=FAKE + 2), T.EALIGN), (dict(max_q=8192, words=128, num_seqs=60000), T.ESHAPE)]
    for kw, want in cases:
        assert _tree(lib, ctx, **kw) == want, (kw, ctx.last_error())
    assert lib.tabit_kv_tree_attention(None, None, None, FAKE, 1, None) == T.EINVAL
    assert lib.tabit_kv_tree_attention(ctx.handle, ctypes.addressof(_cache()), None, FAKE, 1, None) == T.EINVAL
    # a long cache is split and needs its workspace
    n = lib.tabit_kv_tree_attention_workspace_bytes(5, 8, 2, 64, 2, 3, 64000)
    assert n > 0
    kw = dict(max_kv=64000, table_stride=4000)
    assert _tree(lib, ctx, **kw) == T.EINVAL
    assert _tree(lib, ctx, ws=FAKE, ws_bytes=n - 1, **kw) == T.ESHAPE


def test_tree_mask_refusals(lib, ctx):
    def call(parents=FAKE, n=4, cu=FAKE, seqs=1, max_q=4, mask=FAKE, words=1, depth=FAKE):
        return lib.tabit_tree_mask(ctx.handle, parents, n, cu, seqs, max_q, mask, words, depth, None)
    assert call(parents=None) == T.EINVAL and call(cu=None) == T.EINVAL and call(mask=None) == T.EINVAL
    assert call(n=-1) == T.ESHAPE and call(seqs=-1) == T.ESHAPE and call(max_q=-1) == T.ESHAPE
    assert call(max_q=65) == T.ESHAPE and call(max_q=8193, words=1000) == T.ESHAPE and call(words=0) == T.ESHAPE
    assert call(mask=FAKE + 4) == T.EALIGN and call(depth=FAKE + 2) == T.EALIGN
    assert call(n=0) == T.OK and call(seqs=0) == T.OK and call(max_q=0) == T.OK
    assert lib.tabit_tree_mask(None, FAKE, 4, FAKE, 1, 4, FAKE, 1, None, None) == T.EINVAL


def test_weigh_refusals(lib, ctx):
    cases = [(dict(out=FAKE), T.EINVAL), (dict(sums=None), T.EINVAL), (dict(sums=FAKE + 8), T.EALIGN),
             (dict(), T.EINVAL), (dict(ws=FAKE, ws_bytes=16), T.ESHAPE),
             (dict(max_kv=1 << 30, table_stride=1 << 26, num_seqs=65535, max_q=1), T.ESHAPE),
             (dict(max_kv=0, block_table=None), T.OK)]
    for kw, want in cases:
        assert _weigh(lib, ctx, **kw) == want, (kw, ctx.last_error())
    assert lib.tabit_kv_weigh(None, None, None, FAKE, None) == T.EINVAL
    for rows in (1, 2, 4, 5):      # (both forms have a workspace)
        assert lib.tabit_kv_weigh_workspace_bytes(5, 8, 2, 64, 2, rows, 64) > 0
    assert lib.tabit_kv_weigh_workspace_bytes(5, 7, 2, 64, 2, 1, 64) == 0


def test_evict_refusals(lib, ctx):
    cases = [(dict(seqs=-1), T.ESHAPE), (dict(seqs=65536), T.ESHAPE), (dict(table=None), T.EINVAL), (dict(stride=0), T.ESHAPE),
             (dict(max_kv=-1), T.ESHAPE), (dict(max_kv=65), T.ESHAPE), (dict(max_kv=(1 << 30) + 1, stride=1 << 28), T.ESHAPE),
             (dict(budget=0), T.ESHAPE), (dict(sinks=-1), T.ESHAPE), (dict(recent=-1), T.ESHAPE), (dict(sinks=4, recent=5), T.ESHAPE),
             (dict(lens=None), T.EINVAL), (dict(keep=None), T.EINVAL), (dict(new=None), T.EINVAL), (dict(sums=None), T.EINVAL),
             (dict(sums=FAKE + 4), T.EALIGN), (dict(keep=FAKE + 2), T.EALIGN), (dict(ws=FAKE + 8), T.EALIGN), (dict(seqs=0), T.OK),
             (dict(max_kv=8193, stride=1000), T.EINVAL), (dict(max_kv=8193, stride=1000, ws=FAKE, ws_bytes=64), T.ESHAPE)]
    for kw, want in cases:
        assert _evict(lib, ctx, **kw) == want, (kw, ctx.last_error())
    assert lib.tabit_kv_evict_workspace_bytes(2, 2, 8192) == 0 < lib.tabit_kv_evict_workspace_bytes(2, 2, 8193)


@pytest.mark.parametrize("budget", [(1 << 30) + 1, (1 << 31) - 1])
def test_evict_budget_limit(lib, ctx, budget):
    """Indexes of a list are whole numbers of 32 bits that the kernel steps by thousands."""
    assert _evict(lib, ctx, budget=budget) == T.ESHAPE


def test_compact_refusals(lib, ctx):
    cases = [(dict(seqs=-1), T.ESHAPE), (dict(table=None), T.EINVAL), (dict(stride=0), T.ESHAPE), (dict(heads=3), T.ESHAPE),
             (dict(heads=0), T.ESHAPE), (dict(most=-1), T.ESHAPE), (dict(most=(1 << 26) + 1), T.ESHAPE), (dict(keep=None), T.EINVAL),
             (dict(counts=None), T.EINVAL), (dict(sums=FAKE + 2), T.EALIGN), (dict(ws=FAKE + 8), T.EALIGN), (dict(starts=FAKE + 1), T.EALIGN),
             (dict(most=5000), T.EINVAL), (dict(most=5000, ws=FAKE, ws_bytes=8), T.ESHAPE),
             (dict(seqs=0), T.OK), (dict(most=0), T.OK), (dict(cache=_cache(num_pages=0)), T.OK)]
    for kw, want in cases:
        assert _compact(lib, ctx, **kw) == want, (kw, ctx.last_error())
    assert lib.tabit_kv_compact_workspace_bytes(2, 8, 128, 2048) == 0 < lib.tabit_kv_compact_workspace_bytes(2, 8, 128, 2049)


def test_adapter_refusals(lib, ctx):
    def call(**kw):
        a = dict(x=FAKE, x_scale=None, x_fmt=T.FMT_BF16, rows=4, K=64, N=96, x_stride=64, a=FAKE, b=FAKE, scale=None,
                 num_adapters=2, rank=16, cu_rows=FAKE, adapter=FAKE, num_segments=2, y=FAKE, y_stride=96, out=FAKE,
                 out_stride=96, ws=FAKE, ws_bytes=BIG)
        a.update(kw)
        s = L._AdapterArgs(*[a[n] for n, _ in L._AdapterArgs._fields_])
        return lib.tabit_adapter_linear(ctx.handle, ctypes.addressof(s), None)
    cases = [(dict(x_fmt=9), T.EINVAL), (dict(rows=-1), T.ESHAPE), (dict(num_segments=-1), T.ESHAPE), (dict(num_adapters=-1), T.ESHAPE),
             (dict(K=48), T.ESHAPE), (dict(K=0), T.ESHAPE), (dict(K=32800), T.ESHAPE), (dict(N=100), T.ESHAPE), (dict(rank=8), T.ESHAPE),
             (dict(rank=48), T.ESHAPE), (dict(x=None), T.EINVAL), (dict(cu_rows=None), T.EINVAL), (dict(adapter=None), T.EINVAL),
             (dict(y=None), T.EINVAL), (dict(out=None), T.EINVAL), (dict(a=None), T.EINVAL), (dict(b=None), T.EINVAL),
             (dict(x_fmt=T.FMT_INT8), T.EINVAL), (dict(x_fmt=T.FMT_MXFP4), T.EINVAL), (dict(x_stride=56), T.ESHAPE), (dict(x_stride=68), T.ESHAPE),
             (dict(y_stride=88), T.ESHAPE), (dict(out_stride=100), T.ESHAPE), (dict(out_stride=104), T.ESHAPE),
             (dict(x=FAKE + 8), T.EALIGN), (dict(out=FAKE + 8), T.EALIGN), (dict(ws=FAKE + 8), T.EALIGN), (dict(scale=FAKE + 2), T.EALIGN),
             (dict(x_fmt=T.FMT_INT8, x_scale=FAKE + 2), T.EALIGN), (dict(rows=1 << 30, N=32768, y_stride=32768, out_stride=32768), T.ESHAPE),
             (dict(ws=None, ws_bytes=0), T.EINVAL), (dict(ws_bytes=64), T.ESHAPE), (dict(rows=0), T.OK), (dict(num_segments=0), T.OK)]
    for kw, want in cases:
        assert call(**kw) == want, (kw, ctx.last_error())
    assert lib.tabit_adapter_linear(None, None, None) == T.EINVAL
    assert lib.tabit_adapter_linear(ctx.handle, None, None) == T.EINVAL
    assert lib.tabit_adapter_workspace_bytes(4, 16, 2) > 0 == lib.tabit_adapter_workspace_bytes(0, 16, 2)


def test_rotate_refusals(lib, ctx):
    def call(a=FAKE, rows=4, K=128, had=32, out=FAKE):
        return lib.tabit_adapter_rotate(ctx.handle, a, rows, K, had, out, None)
    assert call(had=0) == T.ERANGE and call(had=16) == T.ERANGE
    assert call(rows=-1) == T.ESHAPE and call(K=96, had=64) == T.ESHAPE and call(K=65536, had=64) == T.ESHAPE
    assert call(rows=1 << 30, K=32768) == T.ESHAPE
    assert call(a=None) == T.EINVAL and call(out=None) == T.EINVAL and call(a=FAKE + 8) == T.EALIGN
    assert call(rows=0) == T.OK


def test_binding_refusals(ctx):
    """Types, shapes and devices are refused before any call."""
    z = torch.zeros
    with pytest.raises(ValueError):
        T.Adapters(z(2, 16, 64, dtype=torch.bfloat16), z(2, 32, 16, dtype=torch.bfloat16))    # not on a GPU
    with pytest.raises(TypeError):
        T.Adapters([1], [2])
    with pytest.raises(ValueError):
        T.Adapters.of([(z(200, 64), z(32, 200))])
    with pytest.raises(ValueError):
        ctx.tree_mask(z(4, 4, dtype=torch.int32), z(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        ctx.adapter_rotate(z(4, 64, dtype=torch.bfloat16), 32)


@pytest.mark.parametrize("a,b", [((8, 64), (32, 16)), ((16, 64), (32, 8)), ((8, 64), (32, 200)), ((64,), (32, 8))])
def test_pairs_of_unequal_ranks(a, b):
    """Filling up to a common rank must not hide that a pair's matrices do not belong together."""
    with pytest.raises(ValueError, match="pair"):
        T.Adapters.of([(torch.zeros(a, dtype=torch.bfloat16), torch.zeros(b, dtype=torch.bfloat16))])
