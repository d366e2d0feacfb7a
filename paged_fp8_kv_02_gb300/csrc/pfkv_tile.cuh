// pfkv_tile.cuh -- one warp's work on a tile of 16 tokens of one KV head: query
// fragments, scores and P.V with warp-level matrix products on e4m3 K and V rows
// in shared memory (128-byte swizzle, as the TMA writes them).
//
// Lane = 4 g + t.  Scores are S^T[16 tokens x 8 heads] per head tile j: a lane
// holds tokens g and g + 8 of heads 8j + 2t and 8j + 2t + 1.  The output is
// O^T[128 x 8] per head tile: o[j][i][e] and o[j][i][2 + e] are head_dim values
// 16g + 2i and 16g + 2i + 1 of head 8j + 2t + e.
#pragma once
#include <stdint.h>

#include "pfkv_ptx.cuh"

namespace pfkv {
namespace tile {

constexpr int kTokens = 16;
constexpr int kRowBytes = 128;                       // head_dim 128 in e4m3
constexpr int kSlabBytes = kTokens * kRowBytes;      // K or V of one tile

// Swizzled offset of 16-byte chunk c of row r (the slab starts on 1024 bytes).
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * kRowBytes + ((c ^ (r & 7)) << 4)); }

// Q of the group's heads as two e4m3 parts after a power-of-two scale per head:
// x = q s with max |x| in (224, 448], part 1 = e4m3(x), part 2 = e4m3(x - part 1)
// -- a bf16 value has 8 significant bits and each part 4, so values of at least
// 1/896 of the head's largest are split exactly and smaller ones within 2^-10.
// qf[j][2kk + p] holds part p of head_dim 32t + 8kk .. + 7 of head 8j + g;
// qinv[j][e] is 1 / s of head 8j + 2t + e.  q: the group's [G][128] bf16 rows.
template <int NT>
__device__ __forceinline__ void load_q(const uint16_t* q, int G, int lane, uint32_t (&qf)[NT][8][2],
                                       float (&qinv)[NT][2]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int head = 8 * j + g;
    uint4 r[4] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (head < G) {
      const uint4* p = reinterpret_cast<const uint4*>(q + head * 128) + 4 * t;
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = __ldg(p + k);
    }
    const uint32_t w[16] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w,
                            r[2].x, r[2].y, r[2].z, r[2].w, r[3].x, r[3].y, r[3].z, r[3].w};
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const float s = pow2_scale(448.f, amax);
    const float inv = 1.f / s;  // exact
    qinv[j][0] = __shfl_sync(0xFFFFFFFFu, inv, 8 * t);
    qinv[j][1] = __shfl_sync(0xFFFFFFFFu, inv, 8 * t + 4);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t c1w = 0u, c2w = 0u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = w[4 * kk + 2 * h + e];
          const float x0 = bf16_lo(x) * s, x1 = bf16_hi(x) * s;
          const uint16_t c1 = f32x2_to_e4m3x2(x0, x1);
          const uint32_t hf = e4m3x2_to_f16x2(c1);
          const uint16_t c2 = f32x2_to_e4m3x2(x0 - f16_lo(hf), x1 - f16_hi(hf));  // exact difference
          c1w |= (uint32_t)c1 << (16 * e);
          c2w |= (uint32_t)c2 << (16 * e);
        }
        qf[j][2 * kk][h] = c1w;
        qf[j][2 * kk + 1][h] = c2w;
      }
  }
}

// s[j] = raw scores K . (q s); the caller multiplies by qinv and the K scale.
template <int NT>
__device__ __forceinline__ void scores(const uint8_t* kb, int lane, const uint32_t (&qf)[NT][8][2],
                                       float (&s)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
  const uint4 x0 = lds128(kb + swz(g, 2 * t)), x1 = lds128(kb + swz(g, 2 * t + 1));
  const uint4 y0 = lds128(kb + swz(g + 8, 2 * t)), y1 = lds128(kb + swz(g + 8, 2 * t + 1));
  const uint32_t xr[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  const uint32_t yr[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
  for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      mma_e4m3(s[j], xr[2 * kk], yr[2 * kk], xr[2 * kk + 1], yr[2 * kk + 1], qf[j][2 * kk][0], qf[j][2 * kk][1]);
      mma_e4m3(s[j], xr[2 * kk], yr[2 * kk], xr[2 * kk + 1], yr[2 * kk + 1], qf[j][2 * kk + 1][0],
               qf[j][2 * kk + 1][1]);
    }
}

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
