"""Bounds of the cached attention's error for queries that it holds exactly (test support).

A query of small whole numbers with a scale of 2^-k / log2(e) (times 32 for a cache that is
transformed) becomes, rotated by nothing and transformed or not, whole numbers of at most seven
bits times 2^-k: the three FP6 terms of the kernel hold them but for the last bit of the scale's
product with log2(e).  Then only this is left of its error:

  scores    fp32: 2^-21 of the absolute sum of a score's products, at most
  weights   2^s by the hardware's exponential (2^-21 relative) and rounded to bf16: 2^-8 at most.
            The rounded weights are summed, so a weight's error e moves the output by e (v - o),
            and all of them by 2^-8 sum_j p_j |v_j - o| at most; a transformed cache's output is
            1/32 of the sum over a block of such terms
  sums      fp32: 2^-22 a summed key
  output    bf16: 2^-8 of itself, and half of the smallest step, 2^-134
  lse       the logarithm of what the weights' rounding and the sums move: 2^-8 + 2^-21, and 2^-22
            a key, and its own rounding
"""
import math

import numpy as np

from oracle import block_oracle as B

LOG2E = np.float32(1.4426950408889634)


def exact_scale(k: int, had: int) -> float:
    """A scale whose product with log2(e) (over 32 for a transformed cache) is 2^-k."""
    return float(np.float32(2.0 ** -k * (32.0 if had else 1.0) / float(LOG2E)))


def whole_queries(rng, tokens: int, heads: int, dim: int, most: int = 2) -> np.ndarray:
    return rng.integers(-most, most + 1, (tokens, heads, dim)).astype(np.float32)


def problem(seed: int, lens, qs, hq: int, hk: int, dim: int, ps: int, had: int, k: int = 3, most: int = 2,
            causal: bool = True) -> dict:
    """Keys and values of a normal distribution in pages of any order, whole queries, scale 2^-k."""
    rng = np.random.default_rng(seed)
    need = [(n + ps - 1) // ps for n in lens]
    table = np.full((len(lens), max(need + [1])), -1, np.int32)
    order, at = rng.permutation(sum(need) + 2), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    x = rng.standard_normal((2, len(order) * ps, hk, dim)).astype(np.float32)
    arr = {}
    for name, y in zip("kv", x):
        codes, scales = B.mx_rows(y, had)
        for part, z in (("codes", codes), ("scales", scales)):
            arr[f"{name}_{part}"] = np.ascontiguousarray(
                z.reshape(len(order), ps, hk, -1).transpose(0, 2, 1, 3))
    cu = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
    return dict(arr=arr, table=table, lens=list(lens), cu=cu, q=whole_queries(rng, int(cu[-1]), hq, dim, most),
                scale=exact_scale(k, had), causal=causal, D=dim, had=had)


def gathered(arr, table_row, n: int):
    """fp64 keys and values [hk][n][Dp] of one sequence, and which of them are in the cache."""
    kc, ks, vc, vs = (arr[x] for x in ("k_codes", "k_scales", "v_codes", "v_scales"))
    ps, j = kc.shape[2], np.arange(n)
    page = np.asarray(table_row)[j // ps] if n else np.zeros(0, int)
    there = (page >= 0) & (page < kc.shape[0])
    page = np.where(there, page, 0)
    k = B.mx_values(kc[page, :, j % ps], ks[page, :, j % ps]).transpose(1, 0, 2)
    v = B.mx_values(vc[page, :, j % ps], vs[page, :, j % ps]).transpose(1, 0, 2)
    return k, v, there


def scores(q, k, scale: float, had: int):
    """fp64 scores in base e of q [..][D] with k [n][Dp], and their absolute sums."""
    x = B.padded(np.asarray(q, np.float64))
    if had:
        x = B.hadamard_blocks(x)
    c = scale / (32.0 if had else 1.0)
    return x @ k.T * c, np.abs(x) @ np.abs(k).T * abs(c)


def joined(w, v, had: int, dim: int):
    """Outputs [rows][dim] of weights [rows][n] that add up to one."""
    o = w @ v
    return B.unrotated(o, had)[:, :dim]


def want(q, arr, table, lens, cu, scale: float, causal: bool, dim: int, had: int):
    """fp64 out [T][hq][dim], lse [T][hq] and the bounds of their errors."""
    T, hq, _ = q.shape
    hk = arr["k_codes"].shape[1]
    group = hq // hk
    out, room = np.zeros((T, hq, dim)), np.zeros((T, hq, dim))
    lse, lroom = np.full((T, hq), -np.inf), np.zeros((T, hq))
    for b in range(len(lens)):
        n, ln = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or ln == 0:
            continue
        ks, vs, there = gathered(arr, table[b], ln)
        for h in range(hk):
            k, v = ks[h], vs[h]
            rows = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].reshape(n * group, -1)
            s, spread = scores(rows, k, scale, had)
            i = np.arange(n).repeat(group)
            seen = there[None] & ((np.arange(ln)[None] <= (ln - n + i)[:, None]) | (not causal))
            k0 = seen.sum(1)
            s = np.where(seen, s, -np.inf)
            m = s.max(1, keepdims=True)
            m[np.isinf(m)] = 0.0
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
            o = p @ v
            eps = 2.0 ** -8 + 2.0 ** -20 + np.expm1((np.where(seen, spread, 0) * 2.0 ** -20).max(1))
            off = np.empty_like(o)
            for r in range(len(o)):       # sum_j p_j |v_j - o|
                off[r] = p[r] @ np.abs(v - o[r])
            e = off * eps[:, None] * 1.01 + (p @ np.abs(v)) * ((k0 + 64) * 2.0 ** -22)[:, None]
            if had:
                e = np.repeat(e.reshape(len(e), -1, 32).sum(2) / 32.0, 32, 1)
            res = B.unrotated(o, had)[:, :dim]
            e = e[:, :dim] + np.abs(res) * 2.0 ** -8 + 2.0 ** -134
            at = slice(cu[b], cu[b + 1]), slice(h * group, (h + 1) * group)
            out[at], room[at] = res.reshape(n, group, dim), e.reshape(n, group, dim)
            with np.errstate(divide="ignore"):
                ls = np.where(l[:, 0] > 0, m[:, 0] + np.log(l[:, 0]), -np.inf)
            lr = eps * 1.01 + (k0 + 64) * 2.0 ** -22 + np.abs(np.where(k0 > 0, ls, 0)) * 2.0 ** -21
            lse[at], lroom[at] = ls.reshape(n, group), lr.reshape(n, group)
    return out, lse, room, lroom


def outside(got, ref, room) -> float:
    """The share of elements that are farther from the reference than their room."""
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= room) & ~((got == ref) & np.isinf(ref))
    return float(bad.mean())


def check(out, lse, w) -> None:
    ref, rlse, room, lroom = w
    assert outside(out, ref, room) == 0.0, (outside(out, ref, room), np.nanmax(np.abs(out - ref)))
    assert outside(lse, rlse, lroom) == 0.0, (outside(lse, rlse, lroom), lse.ravel()[:8], rlse.ravel()[:8])
    assert math.isfinite(float(np.abs(ref).max()))


def steep_problem(seed: int, n: int, rows: int, heads: int, dim: int, had: int, v_bytes, top: int = 36,
                  noise: int = 124, causal: bool = False, ps: int = 16) -> dict:
    """Scores (base 2) of +top in even rows and -top in odd ones and, where there is more than one
    block, a few tenths beside: the first block of each key is one code of 6 that a query of 3 (or
    1.5 in every element, for a transformed cache) meets.  v_bytes(rng, shape): the values' scale
    bytes [pages][heads][ps][blocks].  top is 36 times a power of two."""
    rng = np.random.default_rng(seed)
    dp = (dim + 31) // 32 * 32
    pages = max((n + ps - 1) // ps, 1)
    nib = lambda w: rng.integers(0, 256, (pages, heads, ps, w), dtype=np.uint8)    # noqa: E731
    kc, vc = nib(dp // 2), nib(dp // 2)
    vc = (vc & 0x77) | (rng.integers(0, 256, dp // 2, dtype=np.uint8) & 0x88)   # a sign for each element:
    for c in (kc, vc):                                                          # sums of many stay large
        if not had and dim % 32:
            c[..., dim // 2:] = 0
    kc[..., :16] = 0
    kc[..., 0] = 7                                     # E2M1 code of 6, the other elements 0
    ks = np.full((pages, heads, ps, dp // 32), noise, np.uint8)
    ks[..., 0] = 127 + 4 + round(math.log2(top / 36))
    vs = v_bytes(rng, (pages, heads, ps, dp // 32)).astype(np.uint8)
    q = rng.integers(-1, 2, (rows, heads, dim)).astype(np.float32)
    sign = (1.0 - 2.0 * (np.arange(rows) % 2))[:, None, None]
    q[..., :32] = 0.0
    if had:
        q[..., :32] = 1.5 * sign
    else:
        q[..., :1] = 3.0 * sign
    return dict(arr=dict(k_codes=kc, k_scales=ks, v_codes=vc, v_scales=vs),
                table=rng.permutation(pages).astype(np.int32)[None], lens=[n], cu=np.array([0, rows], np.int32),
                q=q, scale=exact_scale(7 if had else 3, had), causal=causal, D=dim, had=had)


# ---------------------------------------------------------------- references that move
_CODE = {6.0: 7, 4.0: 6, 3.0: 5, 2.0: 4, 1.5: 3, 1.0: 2, 0.5: 1}


def _codes_of(target: int):
    """E2M1 codes of sixteen elements whose values add up to target / 2, a whole number in [-96, 96]."""
    left, out = abs(target) / 2.0, []
    for _ in range(16):
        c = next((c for c in _CODE if c <= left), 0.0)
        out.append((_CODE[c] if c else 0) | (8 if c and target < 0 else 0))
        left -= c
    assert left == 0, target
    return out


CLIMBS = ("late", "straddle", "straddle low", "high", "low", "stairs", "falls", "levels")


def climb(kind: str, n: int, rng) -> np.ndarray:
    """Scores (base 2, whole numbers) of n keys that make a row's reference move between tiles of 64
    while what was summed before still counts, or has to be scaled away."""
    j = np.arange(n)
    part = j / n
    jitter = rng.integers(-2, 3, n)
    if kind == "late":         # next to nothing, then 60
        s = np.where(part < 0.6, 0, 60) + jitter
    elif kind == "straddle":   # one key of 38 to 43 in each 64: raised past 40, after some that count
        s = 20 + jitter
        first = np.arange(0, n, 64)
        at = np.minimum(first + rng.integers(0, 64, len(first)), n - 1)
        s[at] = np.array([38, 39, 39, 41, 39, 43, 38])[np.arange(len(first)) % 7]
    elif kind == "straddle low":   # the same above a first tile of -50: a reference of -46 or so, then -4
        s = -50 + jitter
        first = np.arange(0, n, 64)
        at = np.minimum(first + rng.integers(0, 64, len(first)), n - 1)
        s[at] = np.array([-46, -9, -8, -8, -5, -4, -46])[np.arange(len(first)) % 7]
    elif kind == "high":       # a reference of 45 from the start, raised to 90
        s = np.where(part < 0.5, 43, 88) + jitter
        s[rng.choice(n // 2, max(n // 50, 2), replace=False)] = 87
    elif kind == "low":        # -60, then -15, then -14
        s = np.where(part < 0.4, -60, -16) + jitter
    elif kind == "stairs":     # up by a few every 64 keys
        s = -90 + np.minimum(9 * (j // 64), 180) + jitter
    elif kind == "falls":      # 60 first, then 58 and less: what comes later counts less
        s = 60 - np.minimum(2 * (j // 64), 60) + jitter
    else:                      # a level for each 64 keys
        s = rng.integers(-94, 95, n // 64 + 1)[j // 64] + jitter
    return s.clip(-96, 96)


def climb_problem(seed: int, kind: str, n: int, rows: int, heads: int, dim: int, had: int, copies: int = 1,
                  ps: int = 16) -> dict:
    """Keys whose scores are factor * climb(kind), the factor of a row one of +-1, +-1/2, 1/4; values
    of a sign for each element, the other one after the keys' middle, so that sums of the wrong scale
    show.  The
    `heads` heads are repeated `copies` times."""
    rng = np.random.default_rng(seed)
    dp = (dim + 31) // 32 * 32
    pages = (n + ps - 1) // ps
    kc = np.zeros((pages * ps, heads, dp // 2), np.uint8)
    vc = rng.integers(0, 128, (pages * ps, heads, dp // 2), dtype=np.uint8) & 0x77
    vc |= rng.integers(0, 256, dp // 2, dtype=np.uint8) & 0x88
    vc[n // 2:] ^= 0x88
    for h in range(heads):
        t = climb(kind, n, rng)
        c = np.array([_codes_of(int(x)) for x in t], np.uint8)
        kc[:n, h, :8] = c[:, 0::2] | c[:, 1::2] << 4
    if dim % 32 and not had:
        vc[..., dim // 2:] = 0
    ks = np.full((pages * ps, heads, dp // 32), 128, np.uint8)           # codes times 2
    vs = rng.integers(125, 129, (pages * ps, heads, dp // 32)).astype(np.uint8)
    arr = {m: np.ascontiguousarray(np.tile(x.reshape(pages, ps, heads, -1).transpose(0, 2, 1, 3),
                                           (1, copies, 1, 1)))
           for m, x in (("k_codes", kc), ("k_scales", ks), ("v_codes", vc), ("v_scales", vs))}
    pattern = np.zeros(dim)
    pattern[:16] = 1.0
    if had:                                                              # whose transform is the pattern
        pattern[:32] = B.hadamard_blocks(pattern[None, :32])[0] / 32.0
    factor = rng.choice([1.0, 1.0, -1.0, 0.5, -0.5, 0.25], (rows, heads))
    factor[0] = 1.0
    q = np.tile((factor[..., None] * pattern).astype(np.float32), (1, copies, 1))
    return dict(arr=arr, table=np.arange(pages, dtype=np.int32)[None], lens=[n],
                cu=np.array([0, rows], np.int32), q=q, scale=exact_scale(0, had), causal=False, D=dim,
                had=had, heads=heads)


def only_heads(p: dict, heads: int) -> dict:
    return dict(p, arr={m: np.ascontiguousarray(x[:, :heads]) for m, x in p["arr"].items()},
                q=np.ascontiguousarray(p["q"][:, :heads]))


def summed(s, v, runs: int, mistake: str = ""):
    """Out of one row by the kernel's rule (reference 0 until a first tile beyond +-40, or weights past
    2^40), the keys in `runs` runs that are joined, with one mistake planted."""
    tiles = (len(s) + 63) // 64
    per = (tiles + runs - 1) // runs
    parts = []
    for r in range(runs):
        ref, l, o, fresh = 0.0, 0.0, np.zeros(v.shape[1]), True
        for t in range(r * per, min(r * per + per, tiles)):
            x, y = s[t * 64:t * 64 + 64], v[t * 64:t * 64 + 64]
            by = 0.0
            if fresh and abs(x.max()) > 40:
                by = x.max() - ref
            elif not fresh and np.exp2(x - ref).sum() >= 2.0 ** 40:
                by = x.max() - ref
            alpha = 1.0 if fresh else 2.0 ** -by
            fresh = False
            ref += by
            w = np.exp2(x - (ref - by if mistake == "weights of the old reference" else ref))
            l = l * (1.0 if mistake == "sums of weights not scaled" else alpha) + w.sum()
            o = o * (1.0 if mistake == "sums of values not scaled" else
                     alpha * alpha if mistake == "sums of values scaled twice" else alpha) + w @ y
        if not fresh:
            parts.append((ref, l, o))
    top = max(p[0] for p in parts)
    f = [1.0 if mistake == "parts joined as they are" else 2.0 ** (p[0] - top) for p in parts]
    if mistake == "one part lost":
        f[len(f) // 2] = 0.0
    return sum(a * p[2] for a, p in zip(f, parts)) / sum(a * p[1] for a, p in zip(f, parts))


MISTAKES = ("weights of the old reference", "sums of weights not scaled", "sums of values not scaled",
            "sums of values scaled twice", "parts joined as they are", "one part lost")
