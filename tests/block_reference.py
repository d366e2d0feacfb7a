"""Block scales and block-sparse decode in plain 64-bit numpy, from the
definitions in include/pfkv.h, one row or page at a time; shares no code with
the kernels.  Used by the GPU tests of those calls."""
from __future__ import annotations

import math

import numpy as np


def _code_values():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


VALUES = _code_values()


def encode(x):
    """Nearest e4m3 code of doubles, ties to even, saturating at 448; the sign
    of zero is kept."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = np.exp2(e - 3)
    a = np.minimum(np.rint(a / step) * step, 448.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    sub = a < 2.0 ** -6
    mant = np.where(sub, a * 2.0 ** 9, a / np.exp2(e) * 8 - 8)
    code = np.where(sub, mant, (e + 7) * 8 + mant).astype(np.int64)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(x, cache, scales, bt, lens, start, max_new):
    """kv_append_fp8_block of one tensor, in place: x float64 [T][H][D]."""
    pages, H, P, _ = cache.shape
    T, B, maxp = x.shape[0], bt.shape[0], bt.shape[1]
    for b in range(B):
        s0, n, L = int(start[b]), int(start[b + 1]) - int(start[b]), int(lens[b])
        if n <= 0 or n > max_new or s0 < 0 or s0 + n > T or n > L or L > maxp * P:
            continue
        for i in range((L - n) // P, (L - 1) // P + 1):
            page = int(bt[b, i])
            if not 0 <= page < pages:
                continue
            lo, hi = max(0, L - n - i * P), min(P, L - i * P)
            for h in range(H):
                new = x[s0 + i * P + lo - (L - n):s0 + i * P + hi - (L - n), h]
                old = float(scales[page, h]) if lo else 0.0
                s = max(old, block_scale(float(np.abs(new).max())))
                if lo and s > old:
                    cache[page, h, :lo] = encode(VALUES[cache[page, h, :lo]] * (old / s))
                cache[page, h, lo:hi] = encode(new / s)
                scales[page, h] = s


def bounds(k_cache, out, out_scales, bt, lens, start, max_new):
    """page_key_bounds, in place."""
    pages, H, P, _ = k_cache.shape
    for b in range(bt.shape[0]):
        n, L = int(start[b + 1]) - int(start[b]), int(lens[b])
        if n <= 0 or n > max_new or n > L or L > bt.shape[1] * P:
            continue
        for i in range((L - n) // P, (L - 1) // P + 1):
            page = int(bt[b, i])
            if not 0 <= page < pages:
                continue
            x = VALUES[k_cache[page, :, :min(P, L - i * P)]]
            lo, hi = np.nanmin(x, 1), np.nanmax(x, 1)
            for h in range(H):
                a, s = max(np.abs(lo[h]).max(), np.abs(hi[h]).max()), 2.0 ** -15
                while a > 127 * s:
                    s *= 2
                out[page, h, 0], out[page, h, 1] = np.floor(lo[h] / s), np.ceil(hi[h] / s)
                out_scales[page, h] = s


def group_query(q):
    """q float64 [G][D] -> (Q-, Q+) whole numbers [2][D] (Python-exact int64)."""
    amax = float(np.abs(q).max())
    e = math.frexp(amax)[1]
    n = np.array([[round(math.ldexp(v, 14 - e)) for v in row] for row in q.tolist()], np.int64)  # ties to even
    parts = np.stack([np.minimum(n, 0).sum(0), np.maximum(n, 0).sum(0)])
    most, j = int(np.abs(parts).max()), 0
    while most > 127 << j:
        j += 1
    return np.array([[round(math.ldexp(float(v), -j)) for v in row] for row in parts.tolist()], np.int64)


def select(q, bnd, bnd_scales, k_scales, bt, lens, P, top, sink, recent):
    """select_pages: q float64 [B][Hq][D] -> int32 [B][Hkv][top]."""
    B, Hq, _ = q.shape
    Hkv = bnd.shape[1]
    G = Hq // Hkv
    out = np.full((B, Hkv, top), -1, np.int32)
    for b in range(B):
        n = -(-int(lens[b]) // P)
        pages = bt[b, :n].astype(np.int64)
        for h in range(Hkv):
            if n <= top:
                out[b, h, :n] = np.arange(n)
                continue
            Q = group_query(q[b, h * G:(h + 1) * G])
            score = (bnd[pages, h].astype(np.int64) * Q).sum((1, 2)) * bnd_scales[pages, h].astype(np.float64)
            if k_scales is not None:
                score = score * k_scales[pages, h].astype(np.float64)
            score[:sink] = np.inf
            score[n - recent:] = np.inf
            out[b, h] = np.sort(np.argsort(-score, kind="stable")[:top])
    return out


def attend(q, keys, values, softmax_scale, vscales):
    """Softmax attention of q [G][D] over keys, values [T][D] in 64 bits ->
    (out, lse, weight of rounding errors, floor of rounding errors, score
    error), the last three for tolerance().  vscales [T]: each row's V scale."""
    s = q @ keys.T * softmax_scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    den = p.sum(1, keepdims=True)
    # Q enters the products as two e4m3 parts after a scale that takes its largest
    # value above 224: what is left over is at most half a subnormal step, 2^-10,
    # so at most 2^-10 / 224 < 2^-17 of the head's largest |q| per element
    ds = softmax_scale * np.abs(q).max(1) * 2.0 ** -17 * np.abs(keys).sum(1).max()
    floor = (np.abs(values) / vscales[:, None]).sum(0) * vscales.max() * 2.0 ** -25
    return p @ values / den, (m + np.log(den))[:, 0], p @ np.abs(values) / den, floor, ds


def tolerance(ref, weight, floor, ds):
    """Bound on |out - ref|.  A term enters the P.V product as p w times V's
    code, with p = 2^(s - m_ref) and w = vs / v_ref, v_ref at most the largest V
    scale; p w is rounded to f16: by 2^-11 of itself, or by half a subnormal
    step, 2^-25, where it is below 2^-14.  The sum of p is at least 1 (m_ref is
    the score of one of the tokens), so the latter costs at most 2^-25 |code|
    v_ref a term: `floor`.  A score error ds changes each weight and their sum
    by e^ds - 1 at most, f32 sums and exp2 add less than 2^-16 together, and the
    output is rounded to bf16 (2^-8)."""
    rel = 2.0 ** -11 + 2 * np.expm1(ds)[:, None] + 2.0 ** -16
    return weight * rel + floor + np.abs(ref) * 2.0 ** -8 + 1e-30


def lse_tolerance(lse, ds):
    """f32 score, sum and logarithm: 2^-19 of |lse| + 1, and the score's error."""
    return ds + (np.abs(lse) + 1) * 2.0 ** -19
