// page_bounds.cu -- channelwise bounds of the keys of each (page, KV head), in
// 8-bit integers: the summary from which select_pages scores a page without
// reading its keys (the summary of Tang et al., "Quest: query-aware sparsity for
// efficient long-context LLM inference", 2024, here in integers).
//
// Over the rows t < L of a page, in units of the page's K scale,
//   lo_d = min_t K_t[d],  hi_d = max_t K_t[d],  A = max_d max(|lo_d|, |hi_d|),
//   s = the smallest power of two >= 2^-15 with A <= 127 s,
//   stored: floor(lo_d / s), ceil(hi_d / s) and s.
// Rounding outwards keeps them bounds; the power of two makes every step exact
// (e4m3 values have four significant bits), and one scale for a page's 128
// channels lets the score be an integer product (see page_select.cu).
//
// One warp per (page, head): eight lanes take a 128-byte row, four rows at a
// time, minima and maxima as packed f16 (every e4m3 value is an f16).  The
// bytes read are the page's K codes, once; HBM bounds it (4 prompts of 32K-256K
// tokens x 8 heads in 64-token pages, 208 MB: 37.1 us, 5.6 TB/s; a contiguous read of
// as much takes about 36 us from launch to end).
#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"

namespace pfkv {
namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kUnroll = 4;  // loads of four rows in flight per warp

struct BoundsArgs {
  int8_t* bounds;        // [pages][H][2][128]
  float* bound_scales;   // [pages][H]
  const uint8_t* k_cache;  // [pages][H][P][128]
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* new_start;
  int B, H, P, max_pages, max_new, span;
  int64_t num_pages;
};

__device__ __forceinline__ uint32_t min_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Exact whole number of one end of the interval, clamped into int8.
__device__ __forceinline__ uint32_t to_byte(float x) {
  const int i = __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
  return (uint32_t)(i & 0xFF);
}

__global__ void __launch_bounds__(kWarps * 32) page_bounds_kernel(const BoundsArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t job = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);  // (b * span + i) * H + h
  const int h = (int)(job % a.H);
  const int64_t bi = job / a.H;
  const int i = (int)(bi % a.span);
  const int64_t b = bi / a.span;
  if (b >= a.B) return;
  const int n = a.new_start[b + 1] - a.new_start[b], L = a.context_lens[b];
  if (n <= 0 || n > a.max_new || n > L || (int64_t)L > (int64_t)a.max_pages * a.P) return;
  const int logical = (L - n) / a.P + i;
  if ((int64_t)logical * a.P >= L) return;
  const int page = a.block_tables[b * a.max_pages + logical];
  if (page < 0 || (int64_t)page >= a.num_pages) return;  // skipped; validate_tables reports
  const int rows = min(L - logical * a.P, a.P);
  const int64_t ph = (int64_t)page * a.H + h;
  const int c = lane & 7, r0 = lane >> 3;
  const uint8_t* src = a.k_cache + ph * a.P * kD + c * 16;

  uint32_t lo[8], hi[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    lo[k] = 0x7C007C00u;  // +inf, +inf
    hi[k] = 0xFC00FC00u;
  }
  for (int r = r0; r < rows; r += 4 * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)  // past the end: the first row again
      v[u] = __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)(r + 4 * u < rows ? r + 4 * u : r) * kD));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t p, q;
        e4m3x4_to_f16x2x2(w[k], p, q);
        lo[2 * k] = min_f16x2(lo[2 * k], p);
        hi[2 * k] = max_f16x2(hi[2 * k], p);
        lo[2 * k + 1] = min_f16x2(lo[2 * k + 1], q);
        hi[2 * k + 1] = max_f16x2(hi[2 * k + 1], q);
      }
    }
  }
  // Join the four row groups, halving what a lane holds at each step: lanes
  // whose bit 3 is set keep the upper bounds, the others the lower ones; then
  // bit 4 chooses the channels 8 .. 15 or 0 .. 7 of the sixteen.
  const bool up = lane & 8, half = lane & 16;
  uint32_t e[8], f[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo[k] : hi[k], 8);
    e[k] = up ? max_f16x2(hi[k], got) : min_f16x2(lo[k], got);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, half ? e[k] : e[k + 4], 16);
    const uint32_t mine = half ? e[k + 4] : e[k];
    f[k] = up ? max_f16x2(mine, got) : min_f16x2(mine, got);
  }
  auto largest = [&]() {  // over the warp
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(f16_lo(f[k])), fabsf(f16_hi(f[k]))));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
  };
  float m = largest();
  if (m > 448.f) {  // a channel with NaN codes only still has infinite ends: it counts as 0
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (fabsf(f16_lo(f[k])) > 448.f) f[k] &= 0xFFFF0000u;
      if (fabsf(f16_hi(f[k])) > 448.f) f[k] &= 0x0000FFFFu;
    }
    m = largest();
  }
  // smallest power of two s with m <= 127 s = 1.984375 2^6 s, at least 2^-15
  const uint32_t u = __float_as_uint(m);
  const int ex = max((int)(u >> 23) - 6 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0), 127 - 15);
  const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);  // 1 / s
  uint32_t out[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float x[4] = {f16_lo(f[2 * k]) * inv, f16_hi(f[2 * k]) * inv, f16_lo(f[2 * k + 1]) * inv,
                        f16_hi(f[2 * k + 1]) * inv};
    out[k] = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) out[k] |= to_byte(up ? ceilf(x[q]) : floorf(x[q])) << (8 * q);
  }
  *reinterpret_cast<uint2*>(a.bounds + ph * (2 * kD) + (up ? kD : 0) + c * 16 + (half ? 8 : 0)) =
      make_uint2(out[0], out[1]);
  if (lane == 0) a.bound_scales[ph] = __uint_as_float((uint32_t)ex << 23);
}

}  // namespace
}  // namespace pfkv

extern "C" int pfkv_page_key_bounds(int8_t* bounds, float* bound_scales, const void* k_cache,
                                    const int32_t* block_tables, int max_pages_per_seq,
                                    const int32_t* context_lens, const int32_t* new_start, int batch,
                                    int max_new_len, int num_kv_heads, int head_dim, int page_size,
                                    int64_t num_pages, pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  if (batch < 0 || max_new_len < 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || num_pages <= 0 ||
      max_pages_per_seq <= 0)
    return fail(PFKV_ERR_INVALID_ARG, "page_key_bounds: bad sizes");
  if (head_dim != kD) return fail(PFKV_ERR_UNSUPPORTED, "page_key_bounds: head_dim %d != 128", head_dim);
  if ((int64_t)max_pages_per_seq * page_size >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "page_key_bounds: block table too long");
  if (batch == 0 || max_new_len == 0) return PFKV_OK;
  if (!bounds || !bound_scales || !k_cache || !block_tables || !context_lens || !new_start)
    return fail(PFKV_ERR_INVALID_ARG, "page_key_bounds: null pointer");
  if (!aligned(bounds, 16) || !aligned(bound_scales, 4) || !aligned(k_cache, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(new_start, 4))
    return fail(PFKV_ERR_INVALID_ARG, "page_key_bounds: misaligned pointer");
  BoundsArgs a;
  a.bounds = bounds;
  a.bound_scales = bound_scales;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.new_start = new_start;
  a.B = batch;
  a.H = num_kv_heads;
  a.P = page_size;
  a.max_pages = max_pages_per_seq;
  a.max_new = max_new_len;
  int64_t span = ((int64_t)max_new_len + page_size - 2) / page_size + 1;
  if (span > max_pages_per_seq) span = max_pages_per_seq;
  a.span = (int)span;
  a.num_pages = num_pages;
  const int64_t blocks = ((int64_t)batch * span * num_kv_heads + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFF) return fail(PFKV_ERR_UNSUPPORTED, "page_key_bounds: too many pages");
  page_bounds_kernel<<<(unsigned)blocks, kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return check_cuda("page_key_bounds launch");
}
