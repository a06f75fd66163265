"""References in 64 bits of the operators for serving many requests (test support)."""
import numpy as np
import torch

from oracle import block_oracle as B
from tests import attention_check as A
import timestep_adaptive_bit_amd as T

DEV = "cuda:0"


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def cache_of(p):
    return T.KVCache(*[dev(p["arr"][x]) for x in ("k_codes", "k_scales", "v_codes", "v_scales")],
                     head_dim=p["D"], had_block=p["had"])


# ------------------------------------------------------------------ trees
def random_parents(rng, n, roots=0.1, back=8):
    """Parents of n nodes: some hang on the last token, the others on one of the `back` before."""
    return np.array([-1 if i == 0 or rng.random() < roots else rng.integers(max(i - back, 0), i) for i in range(n)],
                    np.int32)


def ancestors(parents):
    """bool [n][n]: node i sees node j (itself and its ancestors); depths."""
    n = len(parents)
    see, depth = np.zeros((n, n), bool), np.zeros(n, np.int32)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            see[i], depth[i] = see[p], depth[p] + 1
        see[i, i] = True
    return see, depth


def packed(see, words):
    """int64 [n][words] of bool [n][m]."""
    out = np.zeros((see.shape[0], words), np.uint64)
    for j in range(min(see.shape[1], 64 * words)):
        out[:, j // 64] |= see[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)


def tree_want(p, see):
    """As attention_check.want, for rows that see of the last n keys what see[b] bool [n][n] says."""
    q, arr, table, lens, cu = p["q"], p["arr"], p["table"], p["lens"], p["cu"]
    scale, dim, had = p["scale"], p["D"], p["had"]
    T_, hq, _ = q.shape
    hk = arr["k_codes"].shape[1]
    group = hq // hk
    out, room = np.zeros((T_, hq, dim)), np.zeros((T_, hq, dim))
    lse, lroom = np.full((T_, hq), -np.inf), np.zeros((T_, hq))
    for b in range(len(lens)):
        n, ln = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or ln == 0:
            continue
        ks, vs, there = A.gathered(arr, table[b], ln)
        node = np.arange(ln) - (ln - n)
        mine = np.ones((n, ln), bool)
        mine[:, node >= 0] = see[b][:, node[node >= 0]]
        seen = np.repeat(mine & there[None], group, 0)
        for h in range(hk):
            k, v = ks[h], vs[h]
            rows = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].reshape(n * group, -1)
            s, spread = A.scores(rows, k, scale, had)
            k0 = seen.sum(1)
            s = np.where(seen, s, -np.inf)
            m = s.max(1, keepdims=True)
            m[np.isinf(m)] = 0.0
            w = np.exp(s - m)
            l = w.sum(1, keepdims=True)
            w = np.divide(w, l, out=np.zeros_like(w), where=l > 0)
            o = w @ v
            eps = 2.0 ** -8 + 2.0 ** -20 + np.expm1((np.where(seen, spread, 0) * 2.0 ** -20).max(1))
            off = np.stack([w[r] @ np.abs(v - o[r]) for r in range(len(o))])
            e = off * eps[:, None] * 1.01 + (w @ np.abs(v)) * ((k0 + 64) * 2.0 ** -22)[:, None]
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


# ------------------------------------------------------------------ accumulated weights
def weigh_want(p, sums, causal, rope=None, positions=None):
    """fp64 sums after a call, the room of each and lse.

    Per unit of a row's largest spread (the sum over blocks of the largest |q'| times sum |k'|,
    times the scale) a score errs by 2^-21 from the query's terms, by 2^-19 at most from the fp32
    rotation and butterflies (six roundings of a sum whose absolute value is at most sqrt(32) of
    the block's largest element) and by 2^-20 from the fp32 products' sums: below 2^-18 together.
    A weight errs by twice its row's largest score error (its own score and the row's sum),
    by 2^-20 for |L| up to 16 in the exponential's argument, and by one rounding per summand.
    """
    q = np.asarray(p["q"], np.float64)
    if rope is not None:
        cos, sin, inter = rope
        q = B.rotate_f64(q, cos, sin, positions, inter)
    arr, table, lens, cu, D, had = p["arr"], p["table"], p["lens"], p["cu"], p["D"], p["had"]
    hk, ps = arr["k_codes"].shape[1], arr["k_codes"].shape[2]
    hq = q.shape[1]
    group = hq // hk
    out, room = sums.astype(np.float64).copy(), np.zeros(sums.shape)
    lse = np.full(q.shape[:2], -np.inf)
    c = p["scale"] / (32.0 if had else 1.0)
    for b in range(len(lens)):
        n, ln = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or ln == 0:
            continue
        ks, _, there = A.gathered(arr, table[b], ln)
        i = np.arange(n).repeat(group)
        seen = there[None] & ((np.arange(ln)[None] <= (ln - n + i)[:, None]) | (not causal))
        new = np.arange(ln) >= ln - n
        for h in range(hk):
            k = ks[h]
            number = ~np.isnan(k).any(1)
            x = B.padded(q[cu[b]:cu[b + 1], h * group:(h + 1) * group].reshape(n * group, -1))
            if had:
                x = B.hadamard_blocks(x)
            with np.errstate(invalid="ignore", divide="ignore"):
                s = np.where(seen, x @ k.T * c, -np.inf)
                m = s.max(1, keepdims=True)
                m = np.where(np.isinf(m), 0.0, m)
                w = np.exp(s - m)
                l = w.sum(1, keepdims=True)
                ls = m[:, 0] + np.log(l[:, 0])
                counts = np.isfinite(ls)
                w = np.where(counts[:, None], w / np.where(l > 0, l, 1), 0.0)
            w = np.where(number[None], w, 0.0)
            big = np.abs(x).reshape(len(x), -1, 32).max(2)
            spread = big @ np.nan_to_num(np.abs(k)).reshape(ln, -1, 32).sum(2).T * abs(c)
            spread = np.where(seen & counts[:, None], spread, 0).max(1)
            rel = np.expm1(2 * np.nan_to_num(spread) * 2.0 ** -18) + 2.0 ** -20 + (np.abs(np.nan_to_num(ls)) / 16 + 1) * 2.0 ** -20
            rel += (seen.sum(1) / 32 + 64) * 2.0 ** -23
            tot, err = w.sum(0), (w * rel[:, None]).sum(0)
            for j in np.nonzero(there)[0]:
                at = table[b][j // ps], h, j % ps
                old = 0.0 if causal and new[j] else out[at]
                room[at] = err[j] + (tot[j] + abs(old)) * (n * group / 16 + 2) * 2.0 ** -24 + 1e-38
                out[at] = old + tot[j]
            lse[cu[b]:cu[b + 1], h * group:(h + 1) * group] = np.where(l[:, 0] == 0, -np.inf, ls).reshape(n, group)
    return out, room, lse


# ------------------------------------------------------------------ eviction
def evict_want(sums, table, lens, budget, sinks, recent):
    """keep [B][hk][budget], new lengths: sums [pages][hk][ps]."""
    pages, hk, ps = sums.shape
    keep, new = np.full((len(lens), hk, budget), -1, np.int32), np.minimum(lens, budget).astype(np.int32)
    for b, n in enumerate(lens):
        j = np.arange(n)
        page = np.asarray(table[b])[j // ps] if n else np.zeros(0, int)
        there = (page >= 0) & (page < pages)
        for h in range(hk):
            w = np.where(there, sums[np.where(there, page, 0), h, j % ps], np.nan)
            kept = j
            if n > budget:
                w = np.where(np.isnan(w), -np.inf, w.astype(np.float64))
                low = np.isinf(w) & (w < 0) & (~there | np.isnan(sums[np.where(there, page, 0), h, j % ps]))
                order = sorted(range(sinks, n - recent), key=lambda i: (low[i], -w[i], i))
                kept = np.array(sorted(list(range(sinks)) + order[:budget - sinks - recent] + list(range(n - recent, n))), int)
            keep[b, h, :len(kept)] = kept
    return keep, new


def compact_want(arrays, table, keep, counts, starts=None):
    """Copies of arrays [pages][hk][ps][..] with the rows moved."""
    out = [a.copy() for a in arrays]
    pages, hk, ps = arrays[0].shape[:3]
    for b in range(len(counts)):
        for h in range(hk):
            ks = keep[b, h if keep.shape[1] > 1 else 0]
            for j in range(min(max(int(counts[b]), 0), keep.shape[2])):
                src, dst = int(ks[j]), j + (0 if starts is None else int(starts[b]))
                if src < 0 or dst < 0 or src // ps >= table.shape[1] or dst // ps >= table.shape[1]:
                    continue
                s, d = table[b][src // ps], table[b][dst // ps]
                if not (0 <= s < pages and 0 <= d < pages):
                    continue
                for a, o in zip(arrays, out):
                    o[d, h, dst % ps] = a[s, h, src % ps]
    return out
