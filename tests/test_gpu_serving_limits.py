"""What the operators for serving many requests must hold to beyond their results: places past 2^32 bytes,
graphs that share a workspace or move a cache in place."""
import numpy as np
import pytest
import torch

from tests import attention_check as A
from tests import serve_check as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ARRAYS = ("k_codes", "k_scales", "v_codes", "v_scales")


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


def _captured(call):
    """A graph of call, after one run of it on a side stream."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_pages_past_32_bits(ctx):
    """The same pages at the start and at the end of a cache of 17 GB: the same bits by either table."""
    p = A.problem(21, [2500, 90], [20, 8], 16, 8, 128, 64, 32)
    small = S.cache_of(p)
    held = small.num_pages
    pages = (1 << 18) + held                              # 2^18 pages of 8 heads x 64 tokens: 2^33 bytes of codes
    cache = T.KVCache.empty(pages, 64, 8, 128, 32, DEV)
    far = pages - held
    for n in ARRAYS:
        getattr(cache, n)[:held] = getattr(small, n)
        getattr(cache, n)[far:] = getattr(small, n)
    wide = torch.full((2, 130), -1, dtype=torch.int32, device=DEV)
    wide[:, :p["table"].shape[1]] = S.dev(p["table"])
    tables = [wide, torch.where(wide >= 0, wide + far, wide)]
    cu, lens = S.dev(np.asarray(p["cu"], np.int32)), S.dev(np.array(p["lens"], np.int32))
    q = S.dev(np.asarray(p["q"], np.float32)).bfloat16()
    rng = np.random.default_rng(3)
    parents = np.concatenate([S.random_parents(rng, n) for n in (20, 8)])
    mask, _ = ctx.tree_mask(S.dev(parents), cu, 20)
    one = S.dev(np.array([0, 1, 2], np.int32))
    sums = ctx.kv_sums(cache)
    seen = []
    for table in tables:
        print("tables from", int(table.max()), flush=True)
        out = [ctx.kv_tree_attention(cache, q, mask, cu, table, lens, 20, 2500)]
        out.append(ctx.kv_tree_attention(cache, q[:2].contiguous(), mask[:2].contiguous(), one, table, lens, 1, 2500))
        ctx.kv_weigh(cache, sums, q, cu, table, lens, 20, 2500)
        ctx.kv_weigh(cache, sums, q[:2].contiguous(), one, table, lens, 1, 2500, causal=False)
        for max_kv in (2500, 8193):                       # in one workgroup, in chunks
            out += ctx.kv_evict(cache, sums, table, lens, max_kv, 2100, sinks=4, recent=16)
        keep, new = out[-2:]
        assert ctx.kv_compact_workspace(cache, 2, 2100) is not None
        ctx.kv_compact(cache, table, keep, new, sums=sums)                                       # through the workspace
        ctx.kv_compact(cache, table, keep[:, :, 50:1000].contiguous(), torch.full_like(new, 700))    # in place
        seen.append(out)
    for x, y in zip(*seen):
        assert torch.equal(x, y)
    assert torch.equal(sums[:held], sums[far:]) and sums[:held].any()
    for n in ARRAYS:
        x = getattr(cache, n)
        assert torch.equal(x[:held], x[far:]) and not torch.equal(x[:held], getattr(small, n)), n
        assert not x[held:far].any(), n


def test_adapter_rows_past_32_bits(ctx):
    """y and out of 4.6 GB: the last rows as by themselves."""
    rows, last, N = 70000, 200, 32768
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(rows, 32, generator=g, device=DEV, dtype=torch.bfloat16)
    y = torch.zeros(rows, N, device=DEV, dtype=torch.bfloat16)
    y[-last:] = torch.randn(last, N, generator=g, device=DEV, dtype=torch.bfloat16)
    bank = T.Adapters(torch.randn(2, 16, 32, generator=g, device=DEV, dtype=torch.bfloat16),
                      torch.randn(2, N, 16, generator=g, device=DEV, dtype=torch.bfloat16))
    which = S.dev(np.array([0, 1], np.int32))
    tail = y[-last:].clone()
    ctx.adapter_linear(bank, x, y, S.dev(np.array([0, rows - last, rows], np.int32)), which, out=y)
    want = ctx.adapter_linear(bank, x[-last:].contiguous(), tail, S.dev(np.array([0, 0, last], np.int32)), which)
    assert torch.equal(y[-last:], want)
    head = ctx.adapter_linear(bank, x[:last].contiguous(), torch.zeros_like(tail), S.dev(np.array([0, last, last], np.int32)), which)
    assert torch.equal(y[:last], head)


@pytest.mark.parametrize("budget", [40, 2100])
def test_eviction_captured(ctx, budget):
    """A graph that lists, moves and counts in place, replayed on caches put back in between."""
    n = [2600, 2200, 30]
    p = A.problem(22, n, [1, 1, 1], 8, 2, 64, 16, 32)
    cache, table, lens = S.cache_of(p), S.dev(p["table"]), S.dev(np.array(n, np.int32))
    start = [getattr(cache, x).clone() for x in ARRAYS]
    ws = ctx.kv_compact_workspace(cache, 3, budget)
    sums = ctx.kv_sums(cache)
    got = {}

    def put_back(seed):
        for x, v in zip(ARRAYS, start):
            getattr(cache, x).copy_(v)
        sums.copy_(torch.rand(sums.shape, generator=torch.Generator().manual_seed(seed)))

    def call():
        got["keep"], got["lens"] = ctx.kv_evict(cache, sums, table, lens, max(n), budget, sinks=2, recent=8)
        ctx.kv_compact(cache, table, got["keep"], got["lens"], sums=sums, ws=ws)

    def state():
        return [t.clone() for t in [got["keep"], got["lens"], sums] + [getattr(cache, x) for x in ARRAYS]]

    put_back(0)
    g = _captured(call)
    held = dict(got)
    for seed in range(3):
        put_back(seed)
        call()
        want = state()
        put_back(seed)
        got.update(held)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(state(), want)), seed


def test_graphs_that_share_a_workspace(ctx):
    """Weights of two batches by two graphs on one workspace, in turn: each as by itself."""
    runs = []
    for seed, lens, qs in ((23, [900, 400], [30, 64]), (24, [300, 1500], [64, 5])):
        p = A.problem(seed, lens, qs, 8, 2, 128, 16, 32)
        cache, q = S.cache_of(p), S.dev(np.asarray(p["q"], np.float32)).bfloat16()
        runs.append((cache, q, S.dev(np.asarray(p["cu"], np.int32)), S.dev(p["table"]), S.dev(np.array(lens, np.int32)),
                     max(qs), max(lens), ctx.kv_sums(cache)))
    need = [ctx.kv_weigh_workspace(r[0], r[1], 2, r[5], r[6]).numel() for r in runs]
    ws = torch.empty(max(need), dtype=torch.uint8, device=DEV)
    want, graphs = [], []
    for cache, q, cu, table, lens, most_q, most, sums in runs:
        want.append(ctx.kv_weigh(cache, ctx.kv_sums(cache), q, cu, table, lens, most_q, most).clone())
        graphs.append(_captured(lambda: ctx.kv_weigh(cache, sums, q, cu, table, lens, most_q, most, ws=ws)))    # noqa: B023
    for turn in (0, 1, 0, 0, 1, 1):
        runs[turn][-1].zero_()
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert torch.equal(runs[turn][-1], want[turn]), turn
