"""Cases and plain forms of the operators that serving many requests adds to the cache and the linears.

Four operators, each in the plain form (elementary torch operations, fp32) and through the library:

  tree     softmax attention of trees of drafted tokens over the paged MXFP4 cache: a row sees the
           tokens before its tree and, of the tree, what its mask names
  weigh    the attention weights that a step's queries give to each cached token, added to fp32
           sums kept a page beside the cache; the sums of the queries' own tokens are set
  evict    of each head's tokens the first, the last and those of the largest sums are kept and
           moved together in place; the lists, the moved sums, and the kept rows as the values they
           stand for come back
  adapt    out = y + c (x A^T) B^T with the low-rank adapter of each row's request, on bf16 rows or
           on the INT8 codes that the projection beside it reads

`listed()` and `draw()` give the cases, `prepare()` a case's inputs, `run()` one pass, `work()` its
unavoidable bytes and flops, `exact()` the outputs in 64 bits.
"""
import math

import torch

own = False   # False: the plain forms; True: the library's operators

DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _tree(name, seqs, nodes, kv_len, q_heads, kv_heads, head_dim, page, rope, had):
    return {"name": name, "op": "tree", "seqs": seqs, "q_len": nodes, "kv_len": kv_len,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "rope": rope, "had": had}


def _weigh(name, seqs, q_len, kv_len, q_heads, kv_heads, head_dim, page, causal, rope, had):
    return {"name": name, "op": "weigh", "seqs": seqs, "q_len": q_len, "kv_len": kv_len,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "causal": causal, "rope": rope, "had": had}


def _evict(name, seqs, kv_len, budget, sinks, recent, kv_heads, head_dim, page):
    return {"name": name, "op": "evict", "seqs": seqs, "kv_len": kv_len, "budget": budget,
            "sinks": sinks, "recent": recent, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "had": 32}


def _adapt(name, segments, rows, adapters, rank, k, n, x):
    return {"name": name, "op": "adapt", "segments": segments, "rows": rows, "adapters": adapters,
            "rank": rank, "k": k, "n": n, "x": x}


def listed():
    return [
        # a small tree of drafted tokens of one sequence over a short cache: latency
        _tree("tree_one", 1, 8, 1000, 32, 8, 128, 16, "half", 32),
        # trees of up to 26 nodes of 16 running sequences, ragged lengths
        _tree("tree_batch", 16, 26, 8192, 32, 8, 128, 16, "half", 32),
        # a large tree over a very long cache: the longest axis
        _tree("tree_long", 1, 64, 131072, 32, 8, 128, 64, "half", 0),
        # what one new token of one sequence looks at: latency
        _weigh("weigh_token", 1, 1, 1000, 32, 8, 128, 16, True, "half", 32),
        # one token of each of 64 sequences, ragged lengths
        _weigh("weigh_batch", 64, 1, 8192, 32, 8, 128, 16, True, "half", 32),
        # the prompts of two sequences behind what is cached of them: the most products
        _weigh("weigh_prompt", 2, 2048, 6144, 32, 8, 128, 32, True, "half", 32),
        # one short sequence cut to a quarter: latency
        _evict("evict_one", 1, 2048, 512, 4, 64, 8, 128, 16),
        # 32 running sequences, ragged, cut to 2048 tokens a head
        _evict("evict_batch", 32, 8192, 2048, 4, 256, 8, 128, 16),
        # one very long sequence cut to an eighth
        _evict("evict_long", 1, 131072, 16384, 4, 1024, 8, 128, 64),
        # one token of each of four requests at SANA's width, an adapter each: latency
        _adapt("adapt_tokens", 4, 4, 4, 16, 2240, 2240, "bf16"),
        # one token of each of 64 requests, 40 adapters among them, on a fused QKV projection
        _adapt("adapt_batch", 64, 64, 40, 64, 4096, 6144, "int8"),
        # as many rows as a CogVideoX-shaped video has, of two requests with a style each, on the fused QKV
        _adapt("adapt_video", 2, 17776, 2, 32, 1920, 5760, "int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "weigh", "evict", "adapt"])
    head_dim = rng.choice([40, 64, 72, 80, 96, 112, 128])
    rope = rng.choice(["none", "half", "pairs"])
    page = rng.choice([16, 32, 64, 128])
    had = rng.choice([0, 32])
    kv_heads, group = rng.choice([(8, 4), (4, 8), (2, 6), (16, 1), (20, 1), (30, 1), (1, 16)])
    if op == "tree":
        seqs, nodes = _log(rng, 1, 32), _log(rng, 2, 128)
        most = 64 * 131072 * 32 * 128 // (seqs * nodes * kv_heads * group * head_dim)
        kv_len = max(nodes, min(_log(rng, 16, 131072), 16 * 8192 * 8 // (seqs * kv_heads), most))
        case = _tree("", seqs, nodes, kv_len, kv_heads * group, kv_heads, head_dim, page, rope, had)
    elif op == "weigh":
        if rng.random() < 0.5:      # single tokens
            seqs, q_len, causal = _log(rng, 1, 64), 1, True
            kv_len = min(_log(rng, 1, 131072), 64 * 8192 * 8 // (seqs * kv_heads))
        else:                       # chunks of queries
            seqs, q_len, causal = rng.randint(1, 4), _log(rng, 2, 4096), rng.random() < 0.7
            most = max(1, 2 * 2048 * 6144 * 32 * 128 // (q_len * seqs * kv_heads * group * head_dim))
            kv_len = min(_log(rng, 1, 20000), most)
            kv_len = max(kv_len, q_len) if causal and q_len <= most else kv_len
        case = _weigh("", seqs, q_len, kv_len, kv_heads * group, kv_heads, head_dim, page, causal,
                      rope, had)
    elif op == "evict":
        seqs = _log(rng, 1, 32)
        kv_len = max(16, min(_log(rng, 64, 131072), 32 * 8192 * 8 // (seqs * kv_heads)))
        budget = max(8, min(kv_len * rng.randint(5, 70) // 100, 32 * 2048 * 8 // (seqs * kv_heads)))
        recent = rng.randint(0, budget // 2)
        case = _evict("", seqs, kv_len, budget, min(rng.choice([0, 1, 4]), budget - recent), recent,
                      kv_heads, head_dim, page)
    else:
        rank = rng.choice([16, 16, 32, 64, 128])
        k, n = 32 * rng.randint(4, 192), 32 * rng.randint(4, 192)
        if rng.random() < 0.5:      # single tokens
            segments = rows = _log(rng, 1, 64)
        else:
            segments = rng.randint(1, 8)
            rows = max(segments, min(_log(rng, 8, 17776), 17776 * 7680 // (k + n)))
        case = _adapt("", segments, rows, rng.randint(1, segments), rank, k, n,
                      rng.choice(["bf16", "int8"]))
    del case["name"]
    return case


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _rope_dim(case):
    return 0 if case["rope"] == "none" else case["head_dim"] // 16 * 16


def _tables(case, positions):
    """cos and sin rows of positions 0 .. positions-1, one per rotated pair."""
    r = _rope_dim(case)
    freq = 10000.0 ** (-torch.arange(r // 2, device=DEV, dtype=torch.float64) * 2 / max(r, 1))
    ang = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * freq
    return ang.cos().float().contiguous(), ang.sin().float().contiguous()


def _ragged(case, seed):
    """Lengths of 0.3 to 1 of the longest, which the first sequence has; one sequence alone has it."""
    u = torch.rand(case["seqs"], generator=torch.Generator().manual_seed(int(seed))).tolist()
    lens = [max(1, int(case["kv_len"] * (0.3 + 0.7 * x))) for x in u]
    lens[0] = case["kv_len"]
    return lens


def _pages(case, lens, g):
    """A block table of pages in any order, of a pool that holds all sequences at the longest."""
    page = case["page"]
    need = torch.tensor([(n + page - 1) // page for n in lens], device=DEV)
    pages = case["seqs"] * ((max(case["kv_len"], case.get("q_len", 1)) + page - 1) // page) + 2
    order = torch.randperm(pages, generator=g, device=DEV).int()
    j = torch.arange(int(need.max()), device=DEV)
    at = (need.cumsum(0) - need)[:, None] + j
    return torch.where(j < need[:, None], order[at.clamp(max=pages - 1)], -1).int(), pages


def _fill(case, pages, g):
    """Codes and scales of keys (some channels several times the others) and values."""
    h, D = case["kv_heads"], case["head_dim"]
    chan = 1.0 + 3.0 * (torch.rand(1, h, 1, D, generator=g, device=DEV) < 0.05).float()
    k_codes, k_scales = _mx(_rotated(_randn(g, pages, h, case["page"], D) * chan, case["had"]))
    v_codes, v_scales = _mx(_rotated(_randn(g, pages, h, case["page"], D), case["had"]))
    return [k_codes, k_scales, v_codes, v_scales]


def _grow(rng, n):
    """A tree of n drafted tokens: the parent of each (-1: the last cached token), its depth, and
    its row of the mask (itself and its ancestors) as whole numbers of 64 bits."""
    parents, depth, seen = [], [], []
    for i in range(n):
        p = rng.randint(max(-1, i - 8), i - 1) if i else -1
        parents.append(p)
        depth.append(depth[p] + 1 if p >= 0 else 0)
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    words = [[(m >> 64 * w) & (1 << 64) - 1 for w in range((n + 63) // 64)] for m in seen]
    return parents, depth, [[x - (1 << 64) if x >> 63 else x for x in row] for row in words]


def _prepare_queries(case, seed):
    """What the attention-like operators share: queries behind a ragged cache."""
    g = _gen(seed)
    B, D = case["seqs"], case["head_dim"]
    lens = _ragged(case, seed)
    # fewer queries in some sequences; the same counts in another order for another seed
    qs = [max(1, case["q_len"] * (4 - (b + int(seed)) % B % 3) // 4) for b in range(B)]
    if case.get("causal", True):
        lens = [max(n, min(m, case["kv_len"])) for n, m in zip(lens, qs)]
    cu = [0]
    for n in qs:
        cu.append(cu[-1] + n)
    table, pages = _pages(case, lens, g)
    cache = _fill(case, pages, g)
    cos, sin = _tables(case, max(case["kv_len"], case["q_len"]))
    q = _randn(g, cu[-1], case["q_heads"], D).bfloat16()
    return g, lens, qs, {
        "case": case, "q": q, "cache": cache, "table": table, "pages": pages, "cos": cos, "sin": sin,
        "cu_q": torch.tensor(cu, dtype=torch.int32, device=DEV),
        "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
        "max_q": max(qs), "max_kv": max(lens), "scale": D ** -0.5}


def _prepare_tree(case, seed):
    import random
    _, lens, qs, s = _prepare_queries(case, seed)
    rng = random.Random(int(seed))
    words, positions, mask = (s["max_q"] + 63) // 64, [], []
    for n, m in zip(qs, lens):
        _, depth, rows = _grow(rng, n)
        positions += [m - n + d for d in depth]
        mask += [row + [0] * (words - len(row)) for row in rows]
    s["positions"] = torch.tensor(positions, dtype=torch.int32, device=DEV)
    s["mask"] = torch.tensor(mask, dtype=torch.int64, device=DEV)
    return s


def _prepare_weigh(case, seed):
    g, lens, qs, s = _prepare_queries(case, seed)
    s["positions"] = torch.cat([torch.arange(n, device=DEV) + max(m - n, 0) for n, m in zip(qs, lens)]).int()
    # what earlier steps have left: a few tokens have most of it
    s["sums"] = 0.05 * torch.exp(2.0 * _randn(g, s["pages"], case["kv_heads"], case["page"]))
    return s


def _prepare_evict(case, seed):
    g = _gen(seed)
    B, page, budget = case["seqs"], case["page"], case["budget"]
    lens = _ragged(case, seed)
    table, pages = _pages(case, lens, g)
    cache = _fill(case, pages, g)
    sums = 0.05 * torch.exp(2.0 * _randn(g, pages, case["kv_heads"], page))
    j = torch.arange(budget, device=DEV)
    n = torch.tensor(lens, device=DEV)[:, None]
    first = table[:, (j // page).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(j < n, first * page + j % page, -1)
    return {"case": case, "cache": cache, "table": table, "pages": pages, "sums": sums,
            "moved": torch.empty_like(sums), "slots": slots.flatten(),
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "max_kv": max(lens)}


def _prepare_adapt(case, seed):
    g = _gen(seed)
    S, T, R, K, N = (case[n] for n in ("segments", "rows", "rank", "k", "n"))
    u = torch.rand(S, generator=torch.Generator().manual_seed(int(seed))) + 0.5
    ends = (u.cumsum(0) / u.sum() * (T - S)).round().long() + torch.arange(1, S + 1)   # one row each at least
    ends[-1] = T
    which = torch.randperm(S, generator=torch.Generator().manual_seed(int(seed) + 1)) % case["adapters"]
    s = {"case": case, "cu_rows": torch.cat([torch.zeros(1, dtype=torch.int64), ends]).int().to(DEV),
         "which": which.int().to(DEV), "y": _randn(g, T, N).bfloat16(),
         "a": (_randn(g, case["adapters"], R, K) * K ** -0.5).bfloat16(),
         "b": (_randn(g, case["adapters"], N, R) * R ** -0.5).bfloat16(),
         "c": 0.25 + 0.5 * torch.rand(case["adapters"], generator=g, device=DEV), "x_scale": None}
    x = _randn(g, T, K) * (1.0 + 9.0 * (torch.rand(1, K, generator=g, device=DEV) < 0.01).float())
    if case["x"] == "int8":     # the codes and row scales that the projection reads
        top = x.abs().amax(1, keepdim=True) / 127.0
        s["x"], s["x_scale"] = torch.round(x / top).to(torch.int8), top[:, 0].contiguous()
    else:
        s["x"] = x.bfloat16()
    return s


def prepare(case, seed):
    state = {"tree": _prepare_tree, "weigh": _prepare_weigh, "evict": _prepare_evict,
             "adapt": _prepare_adapt}[case["op"]](case, seed)
    if own:   # the handles that a program makes once: a context, views of cache and adapters, workspaces
        import timestep_adaptive_bit_amd as T
        ctx = state["ctx"] = T.Context()
        if case["op"] == "adapt":
            state["bank"] = T.Adapters(state["a"], state["b"], state["c"])
            state["ws"] = ctx.adapter_workspace(state["bank"], state["x"], case["segments"])
            return state
        state["kv"] = T.KVCache(*state["cache"], head_dim=case["head_dim"], had_block=case["had"])
        if case["op"] == "evict":
            state["ws"] = ctx.kv_compact_workspace(state["kv"], case["seqs"], case["budget"])
            return state
        state["rope"] = None if case["rope"] == "none" else T.Rope(
            state["cos"], state["sin"], interleaved=case["rope"] == "pairs")
        space = ctx.kv_tree_attention_workspace if case["op"] == "tree" else ctx.kv_weigh_workspace
        state["ws"] = space(state["kv"], state["q"], case["seqs"], state["max_q"], state["max_kv"])
    return state


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _stage(x, h):
    v = x.unflatten(-1, (-1, 2, h))
    a, b = v[..., 0, :], v[..., 1, :]
    return torch.stack([a + b, a - b], -2).flatten(-3)


def _fwht32(x):
    """Unnormalized Walsh-Hadamard transform of each 32 consecutive elements."""
    return _stage(_stage(_stage(_stage(_stage(x, 1), 2), 4), 8), 16)


def _rotated(x, had):
    """x padded with zeros to whole blocks of 32, each block transformed if asked."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 32))
    return _fwht32(x) if had else x


def _turned(x, case, cos, sin, positions):
    """The position rotation of the first elements of each head, x [T][heads][D]."""
    r = _rope_dim(case)
    if r == 0:
        return x
    c, s = cos[positions.long()][:, None], sin[positions.long()][:, None]
    if case["rope"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), x[..., r:]], -1)


def _mx(y):
    """MXFP4 of the last axis: packed E2M1 codes (first of a pair low) and E8M0 scales."""
    b = y.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)       # floor(log2 top) - 2
    e = torch.where(top == 0, torch.zeros_like(e), e)
    a = torch.ldexp(b, -e)
    m = a.abs()
    code = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte()
            + (m > 2.5).byte() + (m >= 3.5).byte() + (m > 5.0).byte())
    code = code + 8 * ((a < 0) & (code > 0)).byte()
    code = code.flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).contiguous(), (e[..., 0] + 127).byte().contiguous()


def _unmx(codes, scales):
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (scales.int() - 127)[..., None]).flatten(-2)


def _weights(s):
    """exp(score - largest) [B][hk][rows of (query, head of the group)][keys] and its sums over the keys,
    rows [B][n] of the queries, and the pages of the table."""
    case, B = s["case"], s["case"]["seqs"]
    hk, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    T, n = s["q"].shape[0], s["max_q"]
    q = _rotated(_turned(s["q"].float(), case, s["cos"], s["sin"], s["positions"]), case["had"])
    i = torch.arange(n, device=DEV)
    n_q = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    row = torch.where(i < n_q[:, None], s["cu_q"][:-1].long()[:, None] + i, T)      # [B][n], T: no query
    q = torch.cat([q, q.new_zeros(1, *q.shape[1:])])[row]                           # [B][n][hq][dp]
    q = q.unflatten(2, (hk, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)            # [B][hk][n*group][dp]
    pages = s["table"].clamp(min=0).long()
    k = _unmx(s["cache"][0][pages], s["cache"][1][pages]).transpose(1, 2).flatten(2, 3)
    w = torch.matmul(q, k.transpose(2, 3)) * (s["scale"] / (32 if case["had"] else 1))
    j, lens = torch.arange(k.shape[2], device=DEV), s["lens"].long()
    node = j - (lens - n_q)[:, None]                                                # [B][keys]
    if case["op"] == "tree":
        mask = torch.cat([s["mask"], s["mask"].new_zeros(1, s["mask"].shape[1])])[row]      # [B][n][words]
        at = node.clamp(0, 64 * mask.shape[2] - 1)[:, None].expand(B, n, -1)
        bit = (torch.gather(mask, 2, at // 64) >> (at % 64)) & 1
        seen = ((node < 0)[:, None] | (bit == 1)) & (j < lens[:, None])[:, None]
    elif case["causal"]:
        seen = (node[:, None] <= i[:, None]) & (j < lens[:, None])[:, None]
    else:
        seen = (j < lens[:, None])[:, None].expand(B, n, -1)
    seen = seen & (i < n_q[:, None])[..., None]
    seen = seen[:, None, :, None].expand(B, 1, n, group, -1).flatten(2, 3)
    w = w.masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    return w, w.sum(-1, keepdim=True).clamp(min=1e-30), row, pages, node


def _plain_tree(s):
    case, D = s["case"], s["case"]["head_dim"]
    w, total, row, pages, _ = _weights(s)
    v = _unmx(s["cache"][2][pages], s["cache"][3][pages]).transpose(1, 2).flatten(2, 3)
    o = torch.matmul(w, v) / total
    if case["had"]:
        o = _fwht32(o) * 0.03125
    group = case["q_heads"] // case["kv_heads"]
    o = o[..., :D].unflatten(2, (-1, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B][n][hq][D]
    out = o.new_empty(s["q"].shape[0] + 1, *o.shape[2:])
    out[row] = o
    return out[:-1].bfloat16()


def _plain_weigh(s):
    case, page = s["case"], s["case"]["page"]
    w, total, _, pages, node = _weights(s)
    new = w.div_(total).sum(2)                                                      # [B][hk][keys]
    j = torch.arange(new.shape[2], device=DEV)
    b, at = (j < s["lens"].long()[:, None]).nonzero(as_tuple=True)
    where = pages[b, at // page]
    old = s["sums"][where, :, at % page]
    if case["causal"]:
        old = old * (node[b, at] < 0).float()[:, None]
    s["sums"][where, :, at % page] = old + new[b, :, at]
    return s["sums"]


def _plain_evict(s):
    case, page, budget = s["case"], s["case"]["page"], s["case"]["budget"]
    s["moved"].copy_(s["sums"])
    pages, lens = s["table"].clamp(min=0).long(), s["lens"].long()[:, None]
    w = s["sums"][pages].transpose(1, 2).flatten(2, 3)                              # [B][hk][keys]
    j = torch.arange(w.shape[2], device=DEV)
    held = ((j < case["sinks"]) | (j >= lens - case["recent"])) & (j < lens)
    w = torch.where(held[:, None], math.inf, w).masked_fill((j >= lens)[:, None], -math.inf)
    keep = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :budget]
    count = lens.clamp(max=budget)
    past = (torch.arange(keep.shape[2], device=DEV) >= count)[:, None]
    keep = torch.sort(keep.masked_fill(past, 1 << 40), dim=-1)[0]
    keep = torch.nn.functional.pad(keep, (0, budget - keep.shape[2]), value=1 << 40)
    there = keep < (1 << 40)
    b, h, to = there.nonzero(as_tuple=True)
    src = keep[b, h, to]
    from_page, to_page = pages[b, src // page], pages[b, to // page]
    for t in s["cache"] + [s["moved"]]:
        t[to_page, h, to % page] = t[from_page, h, src % page]
    at = s["slots"].clamp(min=0)
    back = lambda c, e: _unmx(c[at // page, :, at % page], e[at // page, :, at % page])   # noqa: E731
    k, v = back(*s["cache"][:2]), back(*s["cache"][2:])
    if case["had"]:
        k, v = _fwht32(k) * 0.03125, _fwht32(v) * 0.03125
    gone = (s["slots"] < 0)[:, None, None]
    return {"keep": torch.where(there, keep, -1).int(), "lens": count[:, 0].int(), "sums": s["moved"],
            "k": k[..., :case["head_dim"]].masked_fill(gone, 0.0).bfloat16(),
            "v": v[..., :case["head_dim"]].masked_fill(gone, 0.0).bfloat16()}


def _plain_adapt(s):
    x = s["x"].float() if s["x_scale"] is None else s["x"].float() * s["x_scale"][:, None]
    R, A = s["a"].shape[1], s["a"].shape[0]
    seg = torch.bucketize(torch.arange(x.shape[0], device=DEV), s["cu_rows"][1:].long(), right=True)
    mine = s["which"].long()[seg]
    # every adapter's products, and of them each row's own
    h = torch.matmul(x, s["a"].float().flatten(0, 1).t()).unflatten(1, (A, R)) * s["c"][:, None]
    h = h * (torch.arange(A, device=DEV) == mine[:, None]).float()[..., None]
    return (s["y"].float() + torch.matmul(h.flatten(1), s["b"].float().transpose(1, 2).flatten(0, 1))).bfloat16()


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _own(s):
    ctx, case = s["ctx"], s["case"]
    if case["op"] == "tree":
        return ctx.kv_tree_attention(s["kv"], s["q"], s["mask"], s["cu_q"], s["table"], s["lens"],
                                     s["max_q"], s["max_kv"], scale=s["scale"], rope=s["rope"],
                                     positions=s["positions"], ws=s["ws"])
    if case["op"] == "weigh":
        ctx.kv_weigh(s["kv"], s["sums"], s["q"], s["cu_q"], s["table"], s["lens"], s["max_q"],
                     s["max_kv"], scale=s["scale"], causal=case["causal"], rope=s["rope"],
                     positions=s["positions"], ws=s["ws"])
        return s["sums"]
    if case["op"] == "evict":
        s["moved"].copy_(s["sums"])     # every pass starts from the same sums
        keep, lens = ctx.kv_evict(s["kv"], s["moved"], s["table"], s["lens"], s["max_kv"],
                                  case["budget"], sinks=case["sinks"], recent=case["recent"])
        ctx.kv_compact(s["kv"], s["table"], keep, lens, sums=s["moved"], ws=s["ws"])
        k, v = ctx.kv_read(s["kv"], s["slots"])
        return {"keep": keep, "lens": lens, "sums": s["moved"], "k": k, "v": v}
    return ctx.adapter_linear(s["bank"], s["x"], s["y"], s["cu_rows"], s["which"],
                              x_scale=s["x_scale"], ws=s["ws"])


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "weigh": _plain_weigh, "evict": _plain_evict,
            "adapt": _plain_adapt}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "adapt":
        T, R, K, N = (case[n] for n in ("rows", "rank", "k", "n"))
        return {"bytes": T * K * (2 if case["x"] == "bf16" else 1) + 4 * T * N
                + 2 * case["adapters"] * R * (K + N), "flops": 2 * T * R * (K + N)}
    B, hk, D = case["seqs"], case["kv_heads"], case["head_dim"]
    dp = (D + 31) // 32 * 32
    row = dp // 2 + dp // 32                              # bytes of a key or value
    keys = case["kv_len"] * (1 + 0.65 * (B - 1))          # the first is the longest, the mean of the rest 0.65
    if case["op"] == "evict":
        kept = sum(min(case["budget"], case["kv_len"] * (1.0 if b == 0 else 0.65)) for b in range(B))
        # the sums once, the lists, the kept rows and sums from place to place, and the values back
        return {"bytes": keys * hk * 4 + kept * hk * (4 + 2 * (2 * row + 4) + 4 * D),
                "flops": kept * hk * 2 * dp * 8}
    nq = case["q_len"] * (0.75 if B > 1 else 1.0)
    seen = keys * nq
    if case.get("causal"):
        seen -= B * nq * (nq - 1) / 2
    if case["op"] == "weigh":
        return {"bytes": keys * hk * (row + 8) + B * nq * case["q_heads"] * D * 2,
                "flops": 2.0 * max(seen, 1) * case["q_heads"] * D}
    return {"bytes": keys * hk * 2 * row + B * nq * case["q_heads"] * D * 4,
            "flops": 4.0 * max(seen, 1) * case["q_heads"] * D}


# ----------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ----------------------------------------------------------------------------
def _hadamard(n):
    """Sylvester's matrix by the parity of the common bits of row and column."""
    return torch.tensor([[1.0 - 2.0 * (bin(r & c).count("1") & 1) for c in range(n)] for r in range(n)],
                        dtype=torch.float64, device=DEV)


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rows(codes, scales, case):
    """The vectors that rows of the cache hold, [..][D]."""
    lut = torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=torch.float64, device=DEV)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=DEV)
    v[..., 0::2], v[..., 1::2] = lut[(codes % 16).long()], lut[(codes // 16).long()]
    v = v * torch.repeat_interleave(2.0 ** (scales.double() - 127.0), 32, dim=-1)
    if case["had"]:
        v = (v.view(*v.shape[:-1], -1, 32) @ _hadamard(32)).view(v.shape) / 32
    return v[..., :case["head_dim"]]


def _exact_turn(x, case, s):
    """Each pair as a complex number times e^(i angle)."""
    r = _rope_dim(case)
    if r == 0:
        return x
    z = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, None]
    i = torch.arange(r // 2, device=DEV)
    first, second = (i, i + r // 2) if case["rope"] == "half" else (2 * i, 2 * i + 1)
    y = torch.complex(x[..., first], x[..., second]) * z
    x = x.clone()
    x[..., first], x[..., second] = y.real, y.imag
    return x


def _exact_probabilities(case, s):
    """Sequence by sequence and head by head: its rows of q, its table's pages, the softmax's values."""
    q = _exact_turn(s["q"].double(), case, s)
    group = case["q_heads"] // case["kv_heads"]
    cu, lens = s["cu_q"].tolist(), s["lens"].tolist()
    for b in range(case["seqs"]):
        n, length = cu[b + 1] - cu[b], lens[b]
        t = s["table"][b, :(length + case["page"] - 1) // case["page"]].long()
        node = torch.arange(length, device=DEV) - (length - n)
        if case["op"] == "tree":
            words = s["mask"][cu[b]:cu[b + 1]]
            bits = torch.cat([(words[:, w:w + 1] >> torch.arange(64, device=DEV)) & 1
                              for w in range(words.shape[1])], 1) == 1
            hidden = torch.zeros(n, length, dtype=torch.bool, device=DEV)
            hidden[:, node >= 0] = ~bits[:, node[node >= 0]]
        elif case["causal"]:
            hidden = node > torch.arange(n, device=DEV)[:, None]
        else:
            hidden = torch.zeros(n, length, dtype=torch.bool, device=DEV)
        hidden = hidden.repeat_interleave(group, 0)
        for h in range(case["kv_heads"]):
            k = _exact_rows(s["cache"][0][t, h], s["cache"][1][t, h], case).flatten(0, 1)[:length]
            mine = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].reshape(-1, case["head_dim"])
            w = (mine @ k.T * s["scale"]).masked_fill_(hidden, -math.inf)
            p = torch.softmax(w, -1)
            p[w.amax(-1) == -math.inf] = 0      # a query that sees no key
            yield b, h, slice(cu[b], cu[b + 1]), n, length, t, p


def exact(case, seed):
    s = {"tree": _prepare_tree, "weigh": _prepare_weigh, "evict": _prepare_evict,
         "adapt": _prepare_adapt}[case["op"]](case, seed)
    page = case.get("page", 1)
    if case["op"] == "tree":
        group = case["q_heads"] // case["kv_heads"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for _, h, rows, n, length, t, p in _exact_probabilities(case, s):
            v = _exact_rows(s["cache"][2][t, h], s["cache"][3][t, h], case).flatten(0, 1)[:length]
            out[rows, h * group:(h + 1) * group] = (p @ v).view(n, group, -1)
        return out
    if case["op"] == "weigh":
        sums = s["sums"].double()
        for _, h, _, n, length, t, p in _exact_probabilities(case, s):
            mine = torch.zeros(t.numel() * page, dtype=torch.float64, device=DEV)
            mine[:length] = p.sum(0)
            old = sums[t, h].flatten()
            if case["causal"]:
                old[max(length - n, 0):length] = 0
            sums[t, h] = (old + mine).view(-1, page)
        return sums
    if case["op"] == "evict":
        B, H, D, budget = case["seqs"], case["kv_heads"], case["head_dim"], case["budget"]
        rows = {n: torch.zeros(B, budget, H, D, dtype=torch.float64, device=DEV) for n in ("k", "v")}
        sums, old = s["sums"].double(), s["sums"]
        for b, length in enumerate(s["lens"].tolist()):
            t, kept = s["table"][b].clamp(min=0).long(), min(length, budget)
            for h in range(H):
                w = old[t, h].flatten()[:length].clone()
                w[:case["sinks"]] = w[max(length - case["recent"], 0):] = math.inf
                keep = torch.argsort(-w, stable=True)[:kept].sort()[0]
                new = sums[t, h].flatten()
                new[:kept] = sums[t, h].flatten()[keep]
                at = t[keep // page], torch.full_like(keep, h), keep % page
                for n, c, e in (("k", 0, 1), ("v", 2, 3)):
                    rows[n][b, :kept, h] = _exact_rows(s["cache"][c][at], s["cache"][e][at], case)
                real = s["table"][b] >= 0       # the table's rows that there are
                sums[t[real], h] = new.view(-1, page)[real]
        return {"keep": None, "lens": None, "sums": sums, "k": rows["k"].flatten(0, 1), "v": rows["v"].flatten(0, 1)}
    x = s["x"].double() if s["x_scale"] is None else s["x"].double() * s["x_scale"].double()[:, None]
    out = s["y"].double()
    cu, which = s["cu_rows"].tolist(), s["which"].tolist()
    for i, a in enumerate(which):
        rows = slice(cu[i], cu[i + 1])
        out[rows] += s["c"][a].double() * (x[rows] @ s["a"][a].double().T) @ s["b"][a].double().T
    return out
