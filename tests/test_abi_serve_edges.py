"""Calls of the entry points for serving many requests that must be refused before the first HIP call."""
import ctypes

import pytest

import timestep_adaptive_bit_amd as T
from timestep_adaptive_bit_amd import _lib as L

BASE = 1 << 32        # never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def lib():
    return T.load()


@pytest.fixture
def ctx():
    c = T.Context()
    yield c
    c.close()


def _at(i):
    """Places a GB apart."""
    return BASE + (i << 30)


def _cache(pages=4):
    return L._KvCache(_at(10), _at(11), _at(12), _at(13), pages, 16, 2, 64, 32)


def _evict(lib, ctx, **kw):
    a = dict(sums=_at(0), table=_at(1), stride=4, lens=_at(2), seqs=2, max_kv=64, budget=8, sinks=1, recent=2, keep=_at(3),
             new=_at(4), ws=None, ws_bytes=0)
    a.update(kw)
    c = _cache()
    return lib.tabit_kv_evict(ctx.handle, ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(new=_at(2)), dict(new=_at(2) + 4), dict(new=_at(2) - 4), dict(new=_at(1)), dict(new=_at(1) + 28), dict(new=_at(0) + 508),
    dict(keep=_at(2)), dict(keep=_at(2) - 124), dict(keep=_at(1)), dict(keep=_at(0)), dict(keep=_at(4)), dict(keep=_at(4) - 124),
    dict(new=_at(3) + 124),
])
def test_lists_over_what_is_read(lib, ctx, kw):
    """Other workgroups still read lengths, tables and sums when one writes its list or length."""
    assert _evict(lib, ctx, **kw) == T.EINVAL
    assert "overlap" in ctx.last_error()


def _adapter(lib, ctx, **kw):
    a = dict(x=_at(0), x_scale=_at(1), x_fmt=T.FMT_BF16, rows=100, K=64, N=96, x_stride=64, a=_at(2), b=_at(3), scale=None,
             num_adapters=2, rank=16, cu_rows=_at(4), adapter=_at(5), num_segments=2, y=_at(6), y_stride=96, out=_at(7),
             out_stride=96, ws=_at(8), ws_bytes=1 << 20)
    a.update(kw)
    s = L._AdapterArgs(*[a[n] for n, _ in L._AdapterArgs._fields_])
    return lib.tabit_adapter_linear(ctx.handle, ctypes.addressof(s), None)


@pytest.mark.parametrize("kw", [
    dict(out=_at(0)), dict(out=_at(0) + 64 * 2 * 100 - 16), dict(out=_at(0) - 96 * 2 * 100 + 16),
    dict(out=_at(0), x_fmt=T.FMT_INT8), dict(out=_at(0) + 64 * 100 - 16, x_fmt=T.FMT_INT8),
    dict(out=_at(0) + 32 * 100 - 16, x_fmt=T.FMT_MXFP4),
    dict(out=_at(6) + 16), dict(out=_at(6) - 16), dict(out=_at(6) + 192 * 99), dict(out=_at(6) - 192 * 100 + 16),
    dict(out=_at(0) + 112, x_stride=160, out_stride=160), dict(out=_at(0) - 176, x_stride=160, out_stride=160),
    dict(out=_at(0) + 320 * 99 + 112, x_stride=160, out_stride=160), dict(out=_at(0) - 320 * 99 - 176, x_stride=160, out_stride=160),
    dict(out=_at(6) + 176, y_stride=192, out_stride=192), dict(out=_at(6) - 176, y_stride=192, out_stride=192),
    dict(out=_at(0) + 128, x_stride=160, out_stride=168),
])
def test_products_over_what_is_read(lib, ctx, kw):
    """Other workgroups still read a row of x, or of y, when one writes its part of out."""
    assert _adapter(lib, ctx, **kw) == T.EINVAL
    assert "overlap" in ctx.last_error()


def _weigh(lib, ctx, max_kv, heads=1, max_q=1, tokens=16):
    a = dict(q=_at(0), q_stride=8192, num_tokens=tokens, num_q_heads=heads, cu_q=_at(1), num_seqs=1, max_q=max_q, block_table=_at(2),
             table_stride=1 << 27, kv_lens=_at(3), max_kv=max_kv, scale=0.125, causal=1, rope=None, positions=None, out=None,
             lse=None, ws=_at(4), ws_bytes=1 << 62)
    args = L._KvAttentionArgs(*[a[n] for n, _ in L._KvAttentionArgs._fields_])
    c = L._KvCache(_at(10), _at(11), _at(12), _at(13), 4, 16, 1, 64, 32)
    return lib.tabit_kv_weigh(ctx.handle, ctypes.addressof(c), ctypes.addressof(args), _at(5), None)


@pytest.mark.parametrize("max_kv", [(1 << 30) + 1, (1 << 31) - 300, (1 << 31) - 1])
@pytest.mark.parametrize("heads,max_q", [(1, 1), (8, 1), (16, 1), (4, 16)])
def test_weights_of_too_many_keys(lib, ctx, max_kv, heads, max_q):
    """Places of keys are whole numbers of 32 bits that the kernels step by hundreds past the last one."""
    assert _weigh(lib, ctx, max_kv, heads, max_q) == T.ESHAPE
    assert "max_kv" in ctx.last_error()
    assert lib.tabit_kv_weigh_workspace_bytes(16, heads, 1, 64, 1, max_q, max_kv) == 0


@pytest.mark.parametrize("heads,max_q", [(1, 1), (8, 1), (16, 1), (4, 16)])
def test_workspace_of_the_most_keys(lib, heads, max_q):
    """Scores of 4 or 8 rows a key; of more rows the tiles' terms and sums of up to 16 ranges."""
    n = lib.tabit_kv_weigh_workspace_bytes(16, heads, 1, 64, 1, max_q, 1 << 30)
    rows = heads * max_q
    assert (1 << 30) * (16 if rows <= 4 else 32) <= n < 1 << 36 if rows <= 8 else 0 < n < 1 << 37


@pytest.mark.parametrize("heads,tokens", [(33, (1 << 31) - 1), (64, (1 << 31) - 1), (64, 1 << 30), (96, (1 << 31) - 64)])
def test_weights_of_too_many_rows(lib, ctx, heads, tokens):
    """Tile places of a head are whole numbers of 32 bits."""
    assert _weigh(lib, ctx, 64, heads, 1, tokens) == T.ESHAPE
    assert "too many rows" in ctx.last_error()
    assert lib.tabit_kv_weigh_workspace_bytes(tokens, heads, 1, 64, 1, 1, 64) == 0
