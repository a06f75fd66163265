"""The operators for serving many requests together, as a server uses them: one attention layer for three
requests with an adapter each over one cache, its projections quantized and shared; prompts, eviction, a
drafted tree for each, and the accepted path kept."""
import numpy as np
import pytest
import torch

from tests import serve_check as S
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HK, D, W, PAGE, HAD = 8, 2, 64, 512, 16, 32
PROMPTS, NODES, BUDGET = [70, 33, 120], [7, 12, 5], 40


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


class Layer:
    """Weights, adapters and a cache with room for all."""

    def __init__(self, ctx, seed=0):
        self.ctx = ctx
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)            # noqa: E731
        n = (HQ + 2 * HK) * D
        self.qkv = ctx.quantize_weights((r(n, W) * W ** -0.5).bfloat16().to(DEV), HAD)
        a = (r(3, 16, W) * W ** -0.5).bfloat16().to(DEV)
        self.bank = T.Adapters(ctx.adapter_rotate(a, HAD), (r(3, n, 16) * 0.25).bfloat16().to(DEV))
        pages = sum((p + 40 + PAGE - 1) // PAGE for p in PROMPTS)
        self.cache = T.KVCache.empty(pages, PAGE, HK, D, HAD, DEV)
        self.sums = ctx.kv_sums(self.cache)
        order, at = torch.randperm(pages, generator=g).int(), 0
        self.table = torch.full((3, 10), -1, dtype=torch.int32)
        for b, p in enumerate(PROMPTS):
            n = (p + 40 + PAGE - 1) // PAGE
            self.table[b, :n] = order[at:at + n]
            at += n
        self.table = self.table.to(DEV)
        angle = torch.arange(256)[:, None] / 10000.0 ** (torch.arange(D // 2) / (D // 2))
        self.rope = T.Rope(angle.cos().to(DEV), angle.sin().to(DEV))
        self.which = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)

    def project(self, x, cu):
        """q, k, v of rows x of the requests, whose adapters add to the shared projection."""
        codes, scales = self.ctx.hadamard_quant_act(x, HAD)
        y, _ = self.ctx.masked_qgemm(codes, scales, self.qkv["w_q"], self.qkv["w_scale"], 0)
        self.ctx.adapter_linear(self.bank, codes, y, cu, self.which, x_scale=scales, out=y)
        return y.unflatten(1, (HQ + 2 * HK, D)).split([HQ, HK, HK], dim=1)

    def slots(self, b, index):
        index = torch.as_tensor(index, device=DEV)
        return self.table[b].long()[index // PAGE] * PAGE + index % PAGE


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _run(ctx):
    """Everything that a server would see of one such run, in order."""
    layer, seen = Layer(ctx), []
    g = torch.Generator().manual_seed(1)
    cu = np.concatenate([[0], np.cumsum(PROMPTS)])
    x = torch.randn(int(cu[-1]), W, generator=g).bfloat16().to(DEV)
    q, k, v = layer.project(x, _i32(cu))
    pos = torch.cat([torch.arange(p) for p in PROMPTS]).int().to(DEV)
    slots = torch.cat([layer.slots(b, torch.arange(p)) for b, p in enumerate(PROMPTS)])
    ctx.kv_append(layer.cache, k, v, slots, rope=layer.rope, positions=pos)
    lens = _i32(PROMPTS)
    args = (_i32(cu), layer.table, lens, max(PROMPTS), max(PROMPTS))
    seen.append(ctx.kv_attention(layer.cache, q, *args, causal=True, rope=layer.rope, positions=pos))
    ctx.kv_weigh(layer.cache, layer.sums, q, *args, rope=layer.rope, positions=pos)
    seen.append(layer.sums.clone())
    # cut to the budget: two first, ten last and the most looked at
    keep, lens = ctx.kv_evict(layer.cache, layer.sums, layer.table, lens, max(PROMPTS), BUDGET, sinks=2, recent=10)
    ctx.kv_compact(layer.cache, layer.table, keep, lens, sums=layer.sums)
    seen += [keep, lens]
    # a tree of drafted tokens for each: appended, looked from, and one path of it kept
    rng = np.random.default_rng(2)
    parents = [S.random_parents(rng, n, roots=0.0) for n in NODES]
    held = lens.tolist()
    tcu = _i32(np.concatenate([[0], np.cumsum(NODES)]))
    mask, depth = ctx.tree_mask(_i32(np.concatenate(parents)), tcu, max(NODES))
    x = torch.randn(sum(NODES), W, generator=g).bfloat16().to(DEV)
    q, k, v = layer.project(x, tcu)
    first = torch.repeat_interleave(_i32(PROMPTS), torch.tensor(NODES, device=DEV))
    pos = (first + depth).int()
    slots = torch.cat([layer.slots(b, torch.arange(held[b], held[b] + n)) for b, n in enumerate(NODES)])
    ctx.kv_append(layer.cache, k, v, slots, rope=layer.rope, positions=pos)
    lens = _i32([m + n for m, n in zip(held, NODES)])
    seen.append(ctx.kv_tree_attention(layer.cache, q, mask, tcu, layer.table, lens, max(NODES), int(lens.max()),
                                      rope=layer.rope, positions=pos))
    paths = []
    for p in parents:                                   # the path to the last node
        path, i = [], len(p) - 1
        while i >= 0:
            path.append(i)
            i = int(p[i])
        paths.append(path[::-1])
    most = max(len(p) for p in paths)
    lists = np.full((3, 1, most), -1, np.int32)
    for b, p in enumerate(paths):
        lists[b, 0, :len(p)] = np.array(p) + held[b]
    twin = T.KVCache(*[t.clone() for t in (layer.cache.k_codes, layer.cache.k_scales, layer.cache.v_codes,
                                           layer.cache.v_scales)], head_dim=D, had_block=HAD)
    ctx.kv_compact(layer.cache, layer.table, _i32(lists), _i32([len(p) for p in paths]), starts=_i32(held))
    # the same path appended by itself
    rows = np.concatenate([np.array(p) + o for p, o in zip(paths, np.concatenate([[0], np.cumsum(NODES)])[:-1])])
    at = torch.as_tensor(rows, device=DEV)
    slots = torch.cat([layer.slots(b, torch.arange(held[b], held[b] + len(p))) for b, p in enumerate(paths)])
    ctx.kv_append(twin, k[at].contiguous(), v[at].contiguous(), slots, rope=layer.rope, positions=pos[at].contiguous())
    lens = _i32([m + len(p) for m, p in zip(held, paths)])
    one = torch.randn(3, W, generator=g).bfloat16().to(DEV)
    q, _, _ = layer.project(one, _i32([0, 1, 2, 3]))
    args = (_i32([0, 1, 2, 3]), layer.table, lens, 1, int(lens.max()))
    seen.append(ctx.kv_attention(layer.cache, q, *args))
    other = ctx.kv_attention(twin, q, *args)
    return layer, twin, seen, other, held, paths, mask, q


def test_served_together(ctx):
    layer, twin, seen, other, held, paths, mask, q = _run(ctx)
    # the accepted path kept in place is the path appended by itself, byte for byte
    for b, p in enumerate(paths):
        s = layer.slots(b, torch.arange(held[b] + len(p)))
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            x, y = getattr(layer.cache, n), getattr(twin, n)
            assert torch.equal(x[s // PAGE, :, s % PAGE], y[s // PAGE, :, s % PAGE]), (n, b)
    assert torch.equal(seen[-1], other)
    for t in seen:
        assert not t.is_floating_point() or torch.isfinite(t).all()
    # a token's sum is what its own query and later ones gave it: those of a request add up to its
    # rows and heads, each row's weights to one
    sums = seen[1]
    for b, p in enumerate(PROMPTS):
        s = layer.slots(b, torch.arange(p))
        total = sums[s // PAGE, :, s % PAGE].double().sum(0)
        # p rows of HQ / HK heads, each off by 2^-18 at most of its weights' sum
        rows = p * (HQ // HK)
        assert (total - rows).abs().max() < 2.0 ** -16 * rows
    want, new = S.evict_want(sums.cpu().numpy(), layer.table.cpu().numpy(), PROMPTS, BUDGET, 2, 10)
    assert np.array_equal(seen[2].cpu().numpy(), want) and np.array_equal(seen[3].cpu().numpy(), new)


def test_served_twice_alike(ctx):
    """The same run gives the same bits, also beside one on another stream."""
    first = [t.clone() for t in _run(ctx)[2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = T.Context()
    with torch.cuda.stream(side):
        other = _run(second)[2]
    again = _run(ctx)[2]
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, other):
        assert torch.equal(a, b) and torch.equal(a, c)
    second.close()


def test_adapters_reach_their_requests_alone(ctx):
    """Another adapter for one request changes its rows and no other's."""
    layer = Layer(ctx)
    x = torch.randn(30, W, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    cu = _i32([0, 10, 20, 30])
    one = torch.cat(layer.project(x, cu), 1)
    layer.which = _i32([2, 1, 1])
    two = torch.cat(layer.project(x, cu), 1)
    assert torch.equal(one[:10], two[:10]) and torch.equal(one[20:], two[20:]) and not torch.equal(one[10:20], two[10:20])
    layer.which = _i32([-1, -1, -1])
    none = torch.cat(layer.project(x, cu), 1)
    codes, scales = ctx.hadamard_quant_act(x, HAD)
    y, _ = ctx.masked_qgemm(codes, scales, layer.qkv["w_q"], layer.qkv["w_scale"], 0)
    assert torch.equal(none.flatten(1), y)
