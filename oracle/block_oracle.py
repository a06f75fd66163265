"""CPU oracle of the operators between a block's linears: the paged MXFP4 cache,
attention over it, the block norms.  Test infrastructure only (numpy).

Stored codes are decided in fp32 in the order the operator defines (rotation
products and sums, butterflies, scaling), so they are expected bit for bit; the
attention and the norms are evaluated in fp64 from their definitions.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np

from . import tabit_oracle as O


# ------------------------------------------------------------------ rotation
def rotate_f32(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, pos: np.ndarray,
               interleaved: bool) -> np.ndarray:
    """x fp32 [T][heads][D]; tables fp32 [P][R/2]: each product and sum rounded to fp32."""
    out = x.copy()
    half = cos.shape[1]
    for t in range(x.shape[0]):
        c, s = cos[pos[t]], sin[pos[t]]
        for i in range(half):
            u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = x[t, :, u], x[t, :, w]
            out[t, :, u] = a * c[i] - b * s[i]
            out[t, :, w] = b * c[i] + a * s[i]
    return out


def rotate_f64(x, cos, sin, pos, interleaved):
    return rotate_f32(x.astype(np.float64), cos.astype(np.float64), sin.astype(np.float64), pos,
                      interleaved)


def padded(x: np.ndarray) -> np.ndarray:
    d = x.shape[-1]
    return np.concatenate([x, np.zeros(x.shape[:-1] + (-d % 32,), x.dtype)], -1)


def hadamard_blocks(x: np.ndarray) -> np.ndarray:
    """x [..][32 n] fp64 times H32, block by block."""
    y = x.reshape(x.shape[:-1] + (-1, 32)) @ O.sylvester_hadamard(32).astype(np.float64)
    return y.reshape(x.shape)


# ------------------------------------------------------------------ cache
def mx_rows(x: np.ndarray, had: int) -> Tuple[np.ndarray, np.ndarray]:
    """MXFP4 of fp32 [T][heads][D]: codes [T][heads][Dp/2], E8M0 [T][heads][Dp/32]."""
    p = padded(x.astype(np.float32))
    codes, e8 = O.mx_quantize_rows(np.ascontiguousarray(p.reshape(-1, p.shape[-1])), had)
    return codes.reshape(p.shape[:-1] + (-1,)), e8.reshape(p.shape[:-1] + (-1,))


def mx_values(codes: np.ndarray, e8: np.ndarray) -> np.ndarray:
    """fp64 values of packed rows [..][Dp/2], [..][Dp/32]; scale 255 gives NaN."""
    lead = codes.shape[:-1]
    v = O.mx_unpack(np.ascontiguousarray(codes.reshape(-1, codes.shape[-1])),
                    np.ascontiguousarray(e8.reshape(-1, e8.shape[-1]))).astype(np.float64)
    v = v.reshape(lead + (-1, 32))
    v = np.where((e8 == 255)[..., None], np.nan, v)
    return v.reshape(lead + (-1,))


def unrotated(v: np.ndarray, had: int) -> np.ndarray:
    return hadamard_blocks(v) / 32.0 if had else v


# ------------------------------------------------------------------ attention
def attention(q: np.ndarray, cache: Dict[str, np.ndarray], table: np.ndarray, lens, cu, scale: float,
              causal: bool, head_dim: int, had: int, rope: Optional[tuple] = None,
              max_kv: Optional[int] = None):
    """fp64 attention of q fp64 [T][hq][D] over a cache of arrays [P][hk][ps][..].

    Returns (out [T][hq][D], lse [T][hq], weight [T][hq][D], spread [T][hq]): weight is
    (1/32) sum over the block of sum_j p_j |v'_j| (what a relative error of every p_j
    can move), spread the largest sum over blocks of (largest |q'|) sum |k'| times
    scale (what a relative error of every block of q' can move a score).
    """
    kc, ks, vc, vs = (cache[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales"))
    P, hk, ps = kc.shape[:3]
    T, hq, D = q.shape
    group = hq // hk
    if rope is not None:
        cos, sin, pos, inter = rope
        q = rotate_f64(q, cos, sin, pos, inter)
    qr = padded(q)
    if had:
        qr = hadamard_blocks(qr)
    c = scale / (32.0 if had else 1.0)
    out = np.zeros((T, hq, D))
    weight = np.zeros((T, hq, D))
    lse = np.full((T, hq), -np.inf)
    spread = np.zeros((T, hq))
    for b in range(len(lens)):
        n, ln = int(cu[b + 1] - cu[b]), int(lens[b])
        if max_kv is not None:
            ln = min(ln, max_kv)
        if ln == 0:
            continue        # zeros, -inf
        j = np.arange(ln)
        pages = table[b][j // ps]
        there = (pages >= 0) & (pages < P)
        pg = np.where(there, pages, 0)
        for h in range(hk):
            k = mx_values(kc[pg, h, j % ps], ks[pg, h, j % ps])
            v = mx_values(vc[pg, h, j % ps], vs[pg, h, j % ps])
            for i in range(n):
                seen = there & (j <= ln - n + i) if causal else there
                if not seen.any():
                    continue
                for g in range(group):
                    x = qr[cu[b] + i, h * group + g]
                    s = k[seen] @ x * c
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p = p / l
                    o = unrotated(p @ v[seen], had)
                    w = p @ np.abs(v[seen])
                    if had:
                        w = np.repeat(w.reshape(-1, 32).sum(1) / 32.0, 32)
                    at = (cu[b] + i, h * group + g)
                    out[at], weight[at], lse[at] = o[:D], w[:D], m + np.log(l)
                    top = np.abs(x).reshape(-1, 32).max(1)
                    spread[at] = (np.abs(k[seen]).reshape(len(s), -1, 32).sum(2) @ top).max() * abs(c)
    return out, lse, weight, spread


_E2M3 = np.array([m / 8.0 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** e for e in range(3) for m in range(8)])


def e2m3(x: np.ndarray) -> np.ndarray:
    """x rounded to FP6 E2M3 (0 to 7.5 in steps of 1/8 to 1/2), to nearest even, saturating."""
    a = np.abs(np.asarray(x, np.float64))
    hi = np.searchsorted(_E2M3, a).clip(1, len(_E2M3) - 1)
    lo = hi - 1
    dl, dh = a - _E2M3[lo], _E2M3[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.copysign(_E2M3[np.where(up, hi, lo)], x)


def query_terms(x: np.ndarray):
    """The three terms of blocks x [..][32] that the attention holds a query as, fp64 [3][..][32]:
    each E2M3 times 2^e, 2^(e-4), 2^(e-8), e the exponent that puts the block's largest element in
    [3.75, 7.5) of 2^e."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1, keepdims=True)
    unit = 2.0 ** np.ceil(np.log2(np.where(top > 0, top, 1.0) / 7.5))
    unit = np.where(top >= 7.5 * unit, 2 * unit, unit)
    left, terms = x.copy(), []
    for t in range(3):
        u = unit * 2.0 ** (-4 * t)
        terms.append(e2m3(left / u) * u)
        left = left - terms[-1]
    return np.stack(terms)


# ------------------------------------------------------------------ norms
NONE, LAYER, RMS = 0, 1, 2


def norm(v: np.ndarray, kind: int, w, eps: float) -> np.ndarray:
    if kind == NONE:
        return v
    if kind == LAYER:
        v = v - v.mean(1, keepdims=True)
    v = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v if w is None else v * w


def block_norm(x, y=None, post=NONE, post_w=None, gate=None, res_scale=1.0, pre=NONE, pre_w=None,
               scale=None, shift=None, eps=1e-6):
    """fp64 (x', h) of fp64 inputs; gate, scale, shift [samples][H]."""
    M = x.shape[0]
    rep = lambda t: np.repeat(t, M // t.shape[0], 0)   # noqa: E731
    out = res_scale * x
    if y is not None:
        t = norm(y, post, post_w, eps)
        out = out + (t if gate is None else rep(gate) * t)
    h = norm(out, pre, pre_w, eps)
    if scale is not None:
        h = h * (1.0 + rep(scale))
    if shift is not None:
        h = h + rep(shift)
    return out, h
