"""Plain 64-bit restatements of the calls around the attention: rotary
positions, page copies, verification of drafts.  numpy on the host, sharing no
code with the library; used by tests/test_*rotary*, test_*copy* and
test_*verify*."""
from __future__ import annotations

import numpy as np

BF16_HALF = 2.0 ** -8  # half a step of bf16, relative (finfo.eps / 2)


# --------------------------------------------------------------------- rotary
def pair_channels(n_pairs, first, neighbours):
    i = np.arange(n_pairs)
    return (first + 2 * i, first + 2 * i + 1) if neighbours else (first + i, first + n_pairs + i)


def turned(x, positions, freq, axes, first, neighbours):
    """Rows x float64 [T][H][D] turned; positions [A][T] -> (rows, |x| + |y| of
    each channel's pair, 0 where it does not turn, and the pair's |angle|)."""
    a, b = pair_channels(len(freq), first, neighbours)
    angle = positions[np.asarray(axes)].astype(np.float64).T * freq   # [T][pairs]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    out, size, far = x.copy(), np.zeros_like(x), np.zeros_like(x)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    far[..., a] = far[..., b] = np.abs(angle)[:, None]
    return out, size, far


def turn_slack(size, far):
    """How far a pair turned in fp32 may be off: the angle 2^-24 rad and what a
    double's rounding of frequency / 2 pi and of this reference's own product
    make of a far one (2^-52 and 2^-53 of it, taken as 2^-51), sine and cosine
    2 ulp of 1 (2^-23 each), two products and a sum rounded (3 * 2^-24)."""
    return size * (2.0 ** -24 + 2 * 2.0 ** -23 + 3 * 2.0 ** -24 + far * 2.0 ** -51)


def e4m3_values():
    """The 256 values of the format: bias 7, 3 bits of mantissa, no infinity."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


def e4m3_half_step(x):
    """Half the distance of e4m3 values around |x| <= 448."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return np.exp2(e - 4)


# --------------------------------------------------------------------- verify
def weights(p, q):
    """floor(2^42 clamp(p - q, 0, 1)) of float32 rows, as Python-sized ints."""
    with np.errstate(invalid="ignore"):
        r = p.astype(np.float32) - q.astype(np.float32)
    r = np.where(r > 0, np.minimum(r, np.float32(1)), np.float32(0))   # NaN counts as 0
    return np.floor(np.ldexp(r.astype(np.float64), 42)).astype(np.int64)


def draw(w, u):
    total = int(w.sum())
    bar = total * int(min(max(float(u), 0.0), 1 - 2.0 ** -24) * 2 ** 24) >> 24
    return int(np.searchsorted(np.cumsum(w), bar, side="right"))


def verify(p, q, tokens, u, q_start, lens=None):
    """-> (next_tokens, accepted, status, lens) of verify_drafts; p, q float32
    [T][V] (q None: drafts that were not sampled)."""
    T, V = p.shape
    B = len(q_start) - 1
    following = np.full(T, -7, np.int64)   # -7: not written
    accepted, status = np.zeros(B, np.int64), np.zeros(B, np.int64)
    lens = None if lens is None else np.array(lens, np.int64)
    for b in range(B):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        if lo < 0 or hi < lo or hi > T:
            status[b] = 2
            continue
        if lo == hi:
            continue
        kept = 0
        while kept < hi - lo - 1:
            x = int(tokens[lo + kept + 1])
            if not 0 <= x < V:
                status[b] |= 4
                break
            qx = 1.0 if q is None else float(q[lo + kept, x])
            if not float(u[lo + kept]) * qx < float(p[lo + kept, x]):
                break
            following[lo + kept] = x
            kept += 1
        at = lo + kept
        other = np.zeros(V, np.float32)
        if kept < hi - lo - 1:
            if q is not None:
                other = q[at]
            elif 0 <= tokens[at + 1] < V:
                other[tokens[at + 1]] = 1
        w = weights(p[at], other)
        if not w.sum():
            w = weights(p[at], np.zeros(V, np.float32))
        if w.sum():
            following[at] = draw(w, u[hi - 1])
        else:
            following[at] = -1
            status[b] |= 8
        following[at + 1:hi] = -1
        accepted[b] = kept
        if lens is not None:
            lens[b] -= hi - lo - 1 - kept
    return following, accepted, status, lens
