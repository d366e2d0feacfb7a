"""Attention over pages of an e4m3 cache in 64 bits, with the bound that the
warp-level kernels' arithmetic allows: K widened to f16 against Q in f16, the
probabilities times their V scale in f16, everything summed in fp32."""
from __future__ import annotations

import numpy as np

import block_reference as ref


class Pool:
    """A small pool of pages with random codes (no NaN) and scales; tables may
    name a page many times, so that long lists cost the reference little."""

    def __init__(self, rng, pages, H, P, kbin=(-10, -6), vbin=(-10, -6)):
        self.H, self.P, self.pages = H, P, pages
        self.codes, self.scales = {}, {}
        for x, (lo, hi) in (("k", kbin), ("v", vbin)):
            c = rng.integers(0, 256, (pages, H, P, 128)).astype(np.uint8)
            c[(c & 127) > 0x70] -= 0x18
            c[(c & 127) == 127] = 0x30
            self.codes[x] = c
            self.scales[x] = np.exp2(rng.integers(lo, hi + 1, (pages, H))).astype(np.float32)

    def rows(self, x, table, h, pages, L):
        """Dequantised rows of logical pages (their tokens below L) of head h."""
        t, at = self.tokens(pages, L)
        phys = np.asarray(table, np.int64)[t // self.P]
        return ref.VALUES[self.codes[x][phys, h, at]] * self.scales[x][phys, h].astype(np.float64)[:, None]

    def tokens(self, pages, L):
        pages = np.asarray(pages, np.int64)
        t = (pages[:, None] * self.P + np.arange(self.P)).ravel()
        t = t[t < L]
        return t, t % self.P

    def unit(self, table, h, pages, L):
        """(keys, values, V scale of each row) of one (request, KV head)."""
        t, _ = self.tokens(pages, L)
        vs = self.scales["v"][np.asarray(table, np.int64)[t // self.P], h].astype(np.float64)
        return self.rows("k", table, h, pages, L), self.rows("v", table, h, pages, L), vs


def attend(q, keys, values, vs, softmax_scale):
    """q [G][D] over the rows -> (out, lse, bound on |out - got|, on lse)."""
    T = len(keys)
    s = q @ keys.T * softmax_scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    den = p.sum(1, keepdims=True)
    out, lse = p @ values / den, (m + np.log(den))[:, 0]
    # Score.  Q times its power of two lies in f16 exactly down to 2^-29 of the
    # group's largest |q|; below, half a subnormal step, 2^-25, of values up to
    # 2^15: 2^-39 of that largest.  The 128 products are exact, each of their
    # additions loses at most 2^-23 of the sum of magnitudes (truncation to 24
    # bits), and the scales, log2(e) and the exponent's fma another 4 x 2^-24.
    mag = np.abs(q) @ np.abs(keys).T
    ds = softmax_scale * (mag * (130 * 2.0 ** -23) + np.abs(q).max() * 2.0 ** -39 * np.abs(keys).sum(1)).max(1)[:, None]
    # Terms.  p vs rounded to f16: 2^-11 of itself, or half a subnormal step,
    # 2^-25, of a unit that is no more than the largest p vs of the rows.  A score
    # error ds changes a term and the sum of p by e^ds - 1 each; T additions of
    # the output lose 2^-23 each (truncated), those of the denominator 2^-24; the
    # logarithm of a V scale (up to 126 in magnitude) and its sums, exponentials
    # and the join 2^-16.
    rel = 2.0 ** -11 + 2 * np.expm1(ds) + 1.5 * T * 2.0 ** -23 + 2.0 ** -16
    unit = (p * vs).max(1, keepdims=True) / den
    codes = (np.abs(values) / np.where(vs > 0, vs, 1.0)[:, None]).sum(0)
    bound = p @ np.abs(values) / den * rel + unit * codes * 2.0 ** -25 + np.abs(out) * 2.0 ** -8 + 2.0 ** -133
    return out, lse, bound, ds[:, 0] + (np.abs(lse) + 1) * 2.0 ** -19 + T * 2.0 ** -24


def check_unit(out, lse, q, keys, values, vs, softmax_scale, what):
    """One (request, KV head) of a call's results; no rows: zeros and -inf."""
    if not len(keys):
        assert np.all(out == 0) and np.all(np.isneginf(lse)), what
        return 0.0
    o, l, bound, lbound = attend(q, keys, values, vs, softmax_scale)
    worst = float((np.abs(out - o) / bound).max()), float((np.abs(lse - l) / lbound).max())
    assert worst[0] <= 1 and worst[1] <= 1, (what, worst)
    return max(worst)
