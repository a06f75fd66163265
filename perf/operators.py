"""Cases and plain forms of the operators between a block's quantized linears.

Three operators, each in the plain form (elementary torch operations, fp32)
and through the library:

  append     keys and values of new tokens, position-rotated, written to a paged
             MXFP4 cache; the written rows come back as the bf16 values they
             stand for
  attention  softmax attention of a ragged batch of queries over such a cache
  norm       x' = r x + gate * N_post(y), h = N_pre(x') (1 + scale) + shift, with h
             in bf16 or quantized to INT8 after a block Hadamard

`listed()` and `draw()` give the cases, `prepare()` a case's inputs, `run()` one
pass, `work()` its unavoidable bytes and flops, `exact()` the outputs in 64 bits.
"""
import math

import torch

own = False   # False: the plain forms; True: the library's operators

DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _append(name, tokens, kv_heads, head_dim, page, rope, had):
    return {"name": name, "op": "append", "tokens": tokens, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "rope": rope, "had": had}


def _attention(name, seqs, q_len, kv_len, q_heads, kv_heads, head_dim, page, causal, rope, had,
               ragged):
    return {"name": name, "op": "attention", "seqs": seqs, "q_len": q_len, "kv_len": kv_len,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "causal": causal, "rope": rope, "had": had, "ragged": ragged}


def _norm(name, rows, samples, width, post, pre, out, had):
    return {"name": name, "op": "norm", "rows": rows, "samples": samples, "width": width,
            "post": post, "pre": pre, "out": out, "had": had}


def listed():
    return [
        # one new token in each of 16 running sequences: latency
        _append("append_tokens", 16, 8, 128, 16, "half", 32),
        # the encoded prompt of a PixArt-shaped cross attention, written once per image
        _append("append_prompt", 300, 16, 72, 16, "none", 0),
        # all tokens of a CogVideoX-shaped video, rotated by a table row per token
        _append("append_video", 17776, 30, 64, 64, "pairs", 32),
        # one token of one sequence over a short cache: latency
        _attention("attend_token", 1, 1, 1000, 32, 8, 128, 16, True, "half", 32, False),
        # one token of each of 64 sequences, ragged lengths
        _attention("attend_batch", 64, 1, 8192, 32, 8, 128, 16, True, "half", 32, True),
        # one token over a very long cache: the longest axis
        _attention("attend_long", 1, 1, 131072, 32, 8, 128, 64, True, "half", 0, False),
        # PixArt-shaped cross attention, guided and unguided: 4096 queries over the prompt
        _attention("attend_prompt", 2, 4096, 300, 16, 16, 72, 16, False, "none", 0, True),
        # two new latent frames of a CogVideoX-shaped video over all frames and the text
        _attention("attend_video", 1, 2700, 17776, 30, 30, 64, 64, False, "pairs", 32, False),
        # new turns of four sequences behind what is cached of them, causal
        _attention("attend_turns", 4, 2048, 6144, 32, 8, 128, 32, True, "half", 32, True),
        # one token at SANA's width: latency
        _norm("norm_token", 1, 1, 2240, "rms", "rms", "bf16", 0),
        # PixArt's block boundary, guided and unguided: adaptive layer norm
        _norm("norm_image", 8192, 2, 1152, "none", "layer", "bf16", 0),
        # CogVideoX's block boundary with norms on both sides, into the INT8 linear
        _norm("norm_video", 17776, 1, 1920, "rms", "layer", "int8", 32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "norm"])
    head_dim = rng.choice([40, 64, 72, 80, 96, 112, 128])
    rope = rng.choice(["none", "half", "pairs"])
    page = rng.choice([16, 32, 64, 128])
    had = rng.choice([0, 32])
    if op == "append":
        kv_heads = rng.randint(1, 32)
        tokens = _log(rng, 1, 17776 * 30 * 64 // max(kv_heads * head_dim, 30 * 64))
        case = _append("", tokens, kv_heads, head_dim, page, rope, had)
    elif op == "attention":
        kv_heads, group = rng.choice([(8, 4), (4, 8), (2, 6), (16, 1), (20, 1), (30, 1), (1, 16)])
        if rng.random() < 0.5:      # single tokens
            seqs = _log(rng, 1, 64)
            kv_len = min(_log(rng, 1, 131072), 64 * 8192 * 8 // (seqs * kv_heads))
            q_len, causal = 1, True
        else:                       # chunks of queries
            seqs = rng.randint(1, 4)
            q_len = _log(rng, 2, 4096)
            causal = rng.random() < 0.5
            most = max(1, 2700 * 17776 * 30 * 64 // (q_len * seqs * kv_heads * group * head_dim))
            kv_len = min(_log(rng, 1, 20000), most)
            kv_len = max(kv_len, q_len) if causal and q_len <= most else kv_len
        case = _attention("", seqs, q_len, kv_len, kv_heads * group, kv_heads, head_dim, page,
                          causal, rope, had, seqs > 1)
    else:
        samples = rng.choice([1, 2, 4])
        width = 32 * rng.randint(2, 128)
        rows = samples * max(1, min(_log(rng, 1, 17776), 34000000 // width) // samples)
        out = rng.choice(["bf16", "int8"])
        case = _norm("", rows, samples, width, rng.choice(["none", "rms", "layer"]),
                     rng.choice(["rms", "layer"]), out, rng.choice([0, 32]) if out == "int8" else 0)
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


def _channels(g, heads, dim):
    """Magnitude of each channel: some key channels are several times the others."""
    return 1.0 + 3.0 * (torch.rand(1, heads, dim, generator=g, device=DEV) < 0.05).float()


def _prepare_append(case, seed):
    g = _gen(seed)
    T, H, D, page = case["tokens"], case["kv_heads"], case["head_dim"], case["page"]
    dp = (D + 31) // 32 * 32
    # k and v as they leave the QKV linear: two thirds of one row-major matrix
    qkv = (_randn(g, T, 3, H, D) * torch.cat([_channels(g, 3 * H, D)]).view(1, 3, H, D)).bfloat16()
    need = (T + page - 1) // page
    pages = need + 4
    order = torch.randperm(pages, generator=g, device=DEV)[:need]
    i = torch.arange(T, device=DEV)
    slots = order[i // page] * page + i % page
    positions = (i + int(seed) % 97).int()
    cos, sin = _tables(case, T + 97)
    return {"case": case, "k": qkv[:, 1], "v": qkv[:, 2], "slots": slots, "positions": positions,
            "cos": cos, "sin": sin, "pages": pages, "dp": dp,
            "cache": [torch.zeros(pages, H, page, w, dtype=torch.uint8, device=DEV)
                      for w in (dp // 2, dp // 32, dp // 2, dp // 32)]}


def _prepare_attention(case, seed):
    g = _gen(seed)
    B, D, page = case["seqs"], case["head_dim"], case["page"]
    hq, hk = case["q_heads"], case["kv_heads"]
    lens = [case["kv_len"]] * B
    qs = [case["q_len"]] * B
    if case["ragged"]:
        u = torch.rand(B, generator=torch.Generator().manual_seed(int(seed))).tolist()
        lens = [max(1, int(n * (0.3 + 0.7 * x))) for n, x in zip(lens, u)]
        lens[0] = case["kv_len"]
        if case["causal"]:      # the same lengths in another order: their sum goes by the case alone
            qs = [max(1, n * (4 - (b + int(seed)) % B % 3) // 4) for b, n in enumerate(qs)]
            lens = [max(n, min(m, case["kv_len"])) for n, m in zip(lens, qs)]
    cu = [0]
    for n in qs:
        cu.append(cu[-1] + n)
    need = [(n + page - 1) // page for n in lens]
    width = max(need)
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    chan = _channels(g, hk, D)[:, :, None]
    k = _randn(g, pages, hk, page, D) * chan
    k_codes, k_scales = _mx(_rotated(k, case["had"]))
    del k
    v_codes, v_scales = _mx(_rotated(_randn(g, pages, hk, page, D), case["had"]))
    q = _randn(g, cu[-1], hq, D).bfloat16()
    ends = torch.tensor(lens, device=DEV) - torch.tensor(qs, device=DEV)
    positions = torch.cat([torch.arange(n, device=DEV) + ends[b].clamp(min=0) for b, n in enumerate(qs)])
    cos, sin = _tables(case, max(case["kv_len"], case["q_len"]))
    return {"case": case, "q": q, "cache": [k_codes, k_scales, v_codes, v_scales],
            "cu_q": torch.tensor(cu, dtype=torch.int32, device=DEV), "table": table,
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "positions": positions.int(), "cos": cos, "sin": sin, "pages": pages,
            "max_q": max(qs), "max_kv": max(lens), "scale": D ** -0.5}


def _prepare_norm(case, seed):
    g = _gen(seed)
    M, H, S = case["rows"], case["width"], case["samples"]
    wide = 1.0 + 9.0 * (torch.rand(1, H, generator=g, device=DEV) < 0.01).float()
    # shift, scale and gate as they leave the conditioning linear: thirds of one row
    mod = (0.3 * _randn(g, S, 3, H)).bfloat16()
    return {"case": case, "x": (2.0 * _randn(g, M, H) * wide + 0.2).bfloat16(),
            "y": (_randn(g, M, H) * wide).bfloat16(), "shift": mod[:, 0], "scale": mod[:, 1],
            "gate": mod[:, 2], "post_w": (1.0 + 0.1 * _randn(g, H)).bfloat16(),
            "pre_w": (1.0 + 0.1 * _randn(g, H)).bfloat16(), "res_scale": 0.9375, "eps": 1e-6}


def prepare(case, seed):
    state = {"append": _prepare_append, "attention": _prepare_attention,
             "norm": _prepare_norm}[case["op"]](case, seed)
    if own:   # the handles that a program makes once: a context, and views of the cache and tables
        import timestep_adaptive_bit_amd as T
        state["ctx"] = T.Context()
        if case["op"] != "norm":
            state["kv"] = T.KVCache(*state["cache"], head_dim=case["head_dim"], had_block=case["had"])
            state["rope"] = None if case["rope"] == "none" else T.Rope(
                state["cos"], state["sin"], interleaved=case["rope"] == "pairs")
        if case["op"] == "attention":
            state["ws"] = state["ctx"].kv_attention_workspace(
                state["kv"], state["q"], case["seqs"], state["max_q"], state["max_kv"])
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


def _plain_append(s):
    case, D = s["case"], s["case"]["head_dim"]
    k = _turned(s["k"].float(), case, s["cos"], s["sin"], s["positions"])
    kc, ks = _mx(_rotated(k, case["had"]))
    vc, vs = _mx(_rotated(s["v"].float(), case["had"]))
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    s["cache"][0][page, :, at], s["cache"][1][page, :, at] = kc, ks
    s["cache"][2][page, :, at], s["cache"][3][page, :, at] = vc, vs
    back = lambda c, e: _unmx(c[page, :, at], e[page, :, at])   # noqa: E731
    k, v = back(*s["cache"][:2]), back(*s["cache"][2:])
    if case["had"]:
        k, v = _fwht32(k) * 0.03125, _fwht32(v) * 0.03125
    return {"k": k[..., :D].bfloat16(), "v": v[..., :D].bfloat16()}


def _plain_attention(s):
    case, D, B = s["case"], s["case"]["head_dim"], s["case"]["seqs"]
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
    v = _unmx(s["cache"][2][pages], s["cache"][3][pages]).transpose(1, 2).flatten(2, 3)
    w = torch.matmul(q, k.transpose(2, 3)) * (s["scale"] / (32 if case["had"] else 1))
    j, lens = torch.arange(k.shape[2], device=DEV), s["lens"].long()[:, None]
    last = (lens - n_q[:, None] + i + 1).clamp(max=lens) if case["causal"] else lens.expand(B, n)
    seen = j < last[..., None]                                                      # [B][n][keys]
    seen = seen[:, None, :, None].expand(B, 1, n, group, -1).flatten(2, 3)
    w = w.masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    o = torch.matmul(w, v) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    if case["had"]:
        o = _fwht32(o) * 0.03125
    o = o[..., :D].unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)    # [B][n][hq][D]
    out = o.new_empty(T + 1, *o.shape[2:])
    out[row] = o
    return out[:T].bfloat16()


def _normed(x, kind, w, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _plain_norm(s):
    case, rep = s["case"], s["case"]["rows"] // s["case"]["samples"]
    gate, scale, shift = (s[n].float()[:, None] for n in ("gate", "scale", "shift"))
    t = _normed(s["y"].float(), case["post"], s["post_w"], s["eps"]).unflatten(0, (-1, rep))
    x = s["res_scale"] * s["x"].float() + (gate * t).flatten(0, 1)
    h = _normed(x, case["pre"], s["pre_w"], s["eps"]).unflatten(0, (-1, rep))
    h = (h * (1.0 + scale) + shift).flatten(0, 1)
    if case["out"] == "int8":
        h = _fwht32(h) if case["had"] else h
        top = h.abs().amax(-1, keepdim=True)
        code = torch.round(h * (127.0 / top)).clamp(-127, 127)
        h = code * (top / 127.0)
    return {"x": x.bfloat16(), "h": h.bfloat16()}


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _own(s):
    ctx, case = s["ctx"], s["case"]
    if case["op"] == "append":
        ctx.kv_append(s["kv"], s["k"], s["v"], s["slots"], rope=s["rope"], positions=s["positions"])
        k, v = ctx.kv_read(s["kv"], s["slots"])
        return {"k": k, "v": v}
    if case["op"] == "attention":
        return ctx.kv_attention(s["kv"], s["q"], s["cu_q"], s["table"], s["lens"], s["max_q"],
                                s["max_kv"], scale=s["scale"], causal=case["causal"],
                                rope=s["rope"], positions=s["positions"], ws=s["ws"])
    import timestep_adaptive_bit_amd as T
    kinds = {"none": T.NORM_NONE, "layer": T.NORM_LAYER, "rms": T.NORM_RMS}
    x, h, top = ctx.block_norm(
        s["x"], s["y"], post=kinds[case["post"]], post_weight=s["post_w"] if case["post"] != "none" else None,
        gate=s["gate"], res_scale=s["res_scale"], pre=kinds[case["pre"]], pre_weight=s["pre_w"],
        scale=s["scale"], shift=s["shift"], eps=s["eps"],
        fmt=T.FMT_INT8 if case["out"] == "int8" else T.FMT_BF16, had_block=case["had"])
    if case["out"] == "int8":   # the codes as the values they stand for
        h = torch.mul(h, top[:, None], out=torch.empty(h.shape, dtype=torch.bfloat16, device=h.device))
    return {"x": x, "h": h}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attention": _plain_attention,
            "norm": _plain_norm}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "append":
        n = case["tokens"] * case["kv_heads"]
        dp = (case["head_dim"] + 31) // 32 * 32
        # k and v in, codes and scales out, the written rows back in bf16; per element a
        # rotation, five butterflies, scaling and the transform back
        return {"bytes": n * 2 * (4 * case["head_dim"] + dp // 2 + dp // 32), "flops": n * 2 * dp * 16}
    if case["op"] == "attention":
        B, dp = case["seqs"], (case["head_dim"] + 31) // 32 * 32
        part = 0.65 if case["ragged"] and B > 1 else 1.0     # mean share of the longest
        keys = B * case["kv_len"] * part
        nq = case["q_len"] * (0.75 if case["ragged"] and case["causal"] and B > 1 else 1.0)
        seen = keys * nq
        if case["causal"]:
            seen -= B * nq * (nq - 1) / 2
        return {"bytes": keys * case["kv_heads"] * 2 * (dp // 2 + dp // 32)
                + B * nq * case["q_heads"] * case["head_dim"] * 4,
                "flops": 4.0 * max(seen, 1) * case["q_heads"] * case["head_dim"]}
    n = case["rows"] * case["width"]
    return {"bytes": n * (6 + (1 if case["out"] == "int8" else 2)), "flops": n * 20}


# ----------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ----------------------------------------------------------------------------
def _hadamard(n):
    """Sylvester's matrix by the parity of the common bits of row and column."""
    return torch.tensor([[1.0 - 2.0 * (bin(r & c).count("1") & 1) for c in range(n)] for r in range(n)],
                        dtype=torch.float64, device=DEV)


def _exact_blocks(x, had, n=32):
    out = torch.zeros(*x.shape[:-1], (x.shape[-1] + n - 1) // n * n, dtype=torch.float64, device=DEV)
    out[..., :x.shape[-1]] = x
    return (out.view(*out.shape[:-1], -1, n) @ _hadamard(n)).view(out.shape) if had else out


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


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_mx(y):
    """The values that MXFP4 holds for y: the nearest grid point, of two the one of even code."""
    b = y.reshape(*y.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    unit = 2.0 ** (torch.floor(torch.log2(top.clamp(min=1e-300))) - 2).clamp(-127, 127)
    a = (b / unit).abs().clamp(max=6.0)
    near, found = torch.zeros_like(a), torch.full_like(a, math.inf)
    for code in (0, 2, 4, 6, 1, 3, 5, 7):       # even codes first: they keep the ties
        off = (a - _GRID[code]).abs()
        near = torch.where(off < found, torch.full_like(a, _GRID[code]), near)
        found = torch.minimum(off, found)
    return (near * unit * torch.sign(b)).reshape(y.shape)


def _exact_unmx(codes, scales):
    lut = torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=torch.float64, device=DEV)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=DEV)
    v[..., 0::2], v[..., 1::2] = lut[(codes % 16).long()], lut[(codes // 16).long()]
    return v * torch.repeat_interleave(2.0 ** (scales.double() - 127.0), 32, dim=-1)


def exact(case, seed):
    s = {"append": _prepare_append, "attention": _prepare_attention,
         "norm": _prepare_norm}[case["op"]](case, seed)
    if case["op"] == "append":
        D = case["head_dim"]
        k = _exact_mx(_exact_blocks(_exact_turn(s["k"].double(), case, s), case["had"]))
        v = _exact_mx(_exact_blocks(s["v"].double(), case["had"]))
        if case["had"]:
            k, v = _exact_blocks(k, True) / 32, _exact_blocks(v, True) / 32
        return {"k": k[..., :D].contiguous(), "v": v[..., :D].contiguous()}
    if case["op"] == "attention":
        D, page = case["head_dim"], case["page"]
        group = case["q_heads"] // case["kv_heads"]
        q = _exact_turn(s["q"].double(), case, s)
        out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        cu, lens = s["cu_q"].tolist(), s["lens"].tolist()
        for b in range(case["seqs"]):
            n, length = cu[b + 1] - cu[b], lens[b]
            t = s["table"][b, :(length + page - 1) // page].long()
            for h in range(case["kv_heads"]):
                k = _exact_unmx(s["cache"][0][t, h], s["cache"][1][t, h]).flatten(0, 1)[:length]
                v = _exact_unmx(s["cache"][2][t, h], s["cache"][3][t, h]).flatten(0, 1)[:length]
                if case["had"]:
                    k, v = _exact_blocks(k, True) / 32, _exact_blocks(v, True) / 32
                k, v = k[:, :D], v[:, :D]
                mine = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].reshape(-1, D)
                w = mine @ k.T * s["scale"]
                if case["causal"]:
                    i = torch.arange(n, device=DEV).repeat_interleave(group)
                    w[torch.arange(length, device=DEV) > (length - n + i)[:, None]] = -math.inf
                p = torch.softmax(w, -1)
                p[w.amax(-1) == -math.inf] = 0      # a query that sees no key answers zero
                out[cu[b]:cu[b + 1], h * group:(h + 1) * group] = (p @ v).view(n, group, D)
        return out
    rep = case["rows"] // case["samples"]

    def norm(x, kind, w):
        if kind == "none":
            return x
        if kind == "layer":
            return (x - x.mean(1, keepdim=True)) / (x.var(1, unbiased=False, keepdim=True) + s["eps"]).sqrt() * w
        return x / (x.square().mean(1, keepdim=True) + s["eps"]).sqrt() * w

    gate, scale, shift = (s[n].double().repeat_interleave(rep, 0) for n in ("gate", "scale", "shift"))
    x = s["res_scale"] * s["x"].double() + gate * norm(s["y"].double(), case["post"], s["post_w"].double())
    h = norm(x, case["pre"], s["pre_w"].double()) * (1 + scale) + shift
    if case["out"] == "int8":
        h = _exact_blocks(h, case["had"])
        unit = h.abs().amax(1, keepdim=True) / 127
        h = torch.round(h / unit).clamp(-127, 127) * unit
    return {"x": x, "h": h}
