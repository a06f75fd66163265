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
