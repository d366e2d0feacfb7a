// pfkv_tile.cuh -- one warp's work on a tile of 16 tokens of one KV head: query
// fragments, scores and P.V with warp-level matrix products on e4m3 K and V rows
// in shared memory (128-byte swizzle, as the TMA writes them).
//
// Lane = 4 g + t.  Scores are S^T[16 tokens x 8 heads] per head tile j: a lane
// holds tokens g and g + 8 of heads 8j + 2t and 8j + 2t + 1.  The output is
// O^T[128 x 8] per head tile: o[j][i][e] and o[j][i][2 + e] are head_dim values
// 16g + 2i and 16g + 2i + 1 of head 8j + 2t + e.
#pragma once
#include <math.h>
#include <stdint.h>

#include "pfkv_ptx.cuh"

namespace pfkv {
namespace tile {

constexpr int kTokens = 16;
constexpr int kRowBytes = 128;                       // head_dim 128 in e4m3
constexpr int kSlabBytes = kTokens * kRowBytes;      // K or V of one tile

// Swizzled offset of 16-byte chunk c of row r (the slab starts on 1024 bytes).
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * kRowBytes + ((c ^ (r & 7)) << 4)); }

// Rows of the group's queries [G][128] in bf16: head_dim 32t .. 32t + 31 of head
// 8j + g (zeros past G).
template <int NT>
__device__ __forceinline__ void load_q(const uint16_t* q, int G, int lane, uint4 (&r)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint4* p = reinterpret_cast<const uint4*>(q + (8 * j + g) * 128) + 4 * t;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[j][k] = 8 * j + g < G ? __ldg(p + k) : make_uint4(0, 0, 0, 0);
  }
}

// Those rows in f16 after a power-of-two scale per head that takes its largest
// |q| into (2^14, 2^15]: every finite bf16 query fits, and each value at least
// 2^-29 of that largest is exact.  qf[j][i >> 1][i & 1] is the pair 2i, 2i + 1 of the
// lane's 32 values; qinv[j][e] is 1 / s of head 8j + 2t + e.
template <int NT>
__device__ __forceinline__ void scale_q(const uint4 (&rows)[NT][4], int lane, uint32_t (&qf)[NT][8][2],
                                        float (&qinv)[NT][2]) {
  const int t = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint4* r = rows[j];
    const uint32_t w[16] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w,
                            r[2].x, r[2].y, r[2].z, r[2].w, r[3].x, r[3].y, r[3].z, r[3].w};
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const float s = pow2_scale(32768.f, amax);
    const float inv = 1.f / s;  // exact
    qinv[j][0] = __shfl_sync(0xFFFFFFFFu, inv, 8 * t);
    qinv[j][1] = __shfl_sync(0xFFFFFFFFu, inv, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 16; ++i) qf[j][i >> 1][i & 1] = pack_f16x2(bf16_lo(w[i]) * s, bf16_hi(w[i]) * s);
  }
}

// s[j] = raw scores K . (q s); the caller multiplies by qinv and the K scale.  K
// widens to f16 (exactly) and the products are f16: an m16n8k32 product of e4m3
// against Q in two e4m3 parts took a warp 494 cycles here where this takes about
// 250, and whole calls are faster with this (41 -> 37 us for 64 lists x 8 heads of up
// to 128 pages of 16 tokens).  Two chains of four products for each head tile.
template <int NT>
__device__ __forceinline__ void scores(const uint8_t* kb, int lane, const uint32_t (&qf)[NT][8][2],
                                       float (&s)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
  float r[NT][4];  // the odd steps' sum
  const uint4 x0 = lds128(kb + swz(g, 2 * t)), x1 = lds128(kb + swz(g, 2 * t + 1));
  const uint4 y0 = lds128(kb + swz(g + 8, 2 * t)), y1 = lds128(kb + swz(g + 8, 2 * t + 1));
  const uint32_t xr[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  const uint32_t yr[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
  for (int j = 0; j < NT; ++j)
    s[j][0] = s[j][1] = s[j][2] = s[j][3] = r[j][0] = r[j][1] = r[j][2] = r[j][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    uint32_t a0, a1, a2, a3;
    e4m3x4_to_f16x2x2(xr[ks], a0, a2);
    e4m3x4_to_f16x2x2(yr[ks], a1, a3);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (ks & 1)
        mma_f16(r[j], a0, a1, a2, a3, qf[j][ks][0], qf[j][ks][1]);
      else
        mma_f16(s[j], a0, a1, a2, a3, qf[j][ks][0], qf[j][ks][1]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[j][i] += r[j][i];
}

// Softmax where every page has a V scale of its own.  A head column keeps two
// references in log2 units: m of the scores, and c of scores plus log2 of the V
// scale.  l is a sum of 2^(s - m), o one of 2^(s + log2 vs - c) times V's codes, so
//   out = (o 2^(c - m)) / l.
// The terms of o are rounded to f16, so their unit has to follow the largest p vs:
// relative to the largest V scale alone, a page of small values would lose its bits,
// or vanish, beside one of large values, however small the probability of that one.
// One exponential takes s + log2 vs - c: of the product 2^(s - m) times vs 2^(m - c)
// one factor can underflow where the other overflows.  c >= m - 126 keeps 2^(c - m)
// a normal number.
constexpr float kNoUnit = -3.0e38f;  // c before the first token

// Both references of the columns that a tile's scores s (raw; times sc they are in
// log2 units) exceed by more than `slack` are raised, and l and o follow.  lvs:
// log2 of the tile's V scale, -inf where that is 0.
template <int NT>
__device__ __forceinline__ void raise_references(const float (&s)[NT][4], float sc, float lvs, float slack,
                                                 float (&m)[NT][2], float (&c)[NT][2], float (&l)[NT][2],
                                                 float (&o)[NT][8][4]) {
  bool grow = false;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = fmaxf(s[j][e], s[j][2 + e]);
      grow |= (fmaf(x, sc, -m[j][e]) > slack) | (fmaf(x, sc, lvs - c[j][e]) > slack);
    }
  if (!__any_sync(0xFFFFFFFFu, grow)) return;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(s[j][e], s[j][2 + e]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
      x *= sc;
      const float mn = fmaxf(m[j][e], x), cn = fmaxf(fmaxf(c[j][e], x + lvs), mn - 126.f);
      l[j][e] *= fast_exp2(m[j][e] - mn);
      const float r = fast_exp2(c[j][e] - cn);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[j][i][e] *= r;
        o[j][i][2 + e] *= r;
      }
      m[j][e] = mn;
      c[j][e] = cn;
    }
}
// Factor from o's unit to p times V; 0 where no token was met.
__device__ __forceinline__ float unit(float m, float c) { return m == -INFINITY ? 0.f : fast_exp2(c - m); }

// o += V^T P^T over the tile's first n tokens (rows past them may hold any
// bytes, NaN codes too, and are taken as zeros).  pb: P^T fragments in f16.
template <int NT>
__device__ __forceinline__ void accumulate(const uint8_t* vb, int lane, int n, const uint32_t (&pb)[NT][2],
                                           float (&o)[NT][8][4]) {
  const int g = lane >> 2, t = lane & 3;
  uint4 r0 = lds128(vb + swz(2 * t, g)), r1 = lds128(vb + swz(2 * t + 1, g));
  uint4 r2 = lds128(vb + swz(2 * t + 8, g)), r3 = lds128(vb + swz(2 * t + 9, g));
  if (n < kTokens) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    if (2 * t >= n) r0 = z;
    if (2 * t + 1 >= n) r1 = z;
    if (2 * t + 8 >= n) r2 = z;
    if (2 * t + 9 >= n) r3 = z;
  }
  const uint32_t R0[4] = {r0.x, r0.y, r0.z, r0.w}, R1[4] = {r1.x, r1.y, r1.z, r1.w};
  const uint32_t R2[4] = {r2.x, r2.y, r2.z, r2.w}, R3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
    uint32_t A0, A1, A2, A3;
    e4m3x4_to_f16x2x2(prmt(R0[i >> 1], R1[i >> 1], sel), A0, A1);
    e4m3x4_to_f16x2x2(prmt(R2[i >> 1], R3[i >> 1], sel), A2, A3);
#pragma unroll
    for (int j = 0; j < NT; ++j) mma_f16(o[j][i], A0, A1, A2, A3, pb[j][0], pb[j][1]);
  }
}

}  // namespace tile
}  // namespace pfkv
