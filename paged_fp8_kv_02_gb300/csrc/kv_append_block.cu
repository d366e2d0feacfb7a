// kv_append_block.cu -- quantise new bf16 K/V rows to e4m3 with one scale per
// (page, KV head) and write them into the pages a request's block table names.
//
// For a page that receives new rows, with a = max |x| over them and
//   need(a) = the smallest power of two s >= 2^-126 with a <= 448 s,
// the page's scale becomes s = max(old, need(a)), where old is the stored scale
// if the page holds earlier rows of the request and 0 otherwise; the new codes
// are e4m3(x / s), and where s > old the earlier codes become e4m3(c old / s).
//
// Why powers of two: e4m3 is a floating-point format, so its relative step is
// the same under any scale; rounding amax / 448 up to a power of two gives
// away at most one of its 18 binades at the subnormal end.  In return x / s
// and c old / s are exact shifts, so a growing scale re-rounds nothing that
// stays in the normal range, and every code and scale is the same in any
// precision of arithmetic.
//
// Prompts are bounded by HBM: every row is read and every code written once (8
// prompts of 0.3K-16K tokens x 8 heads, 69 MB: 14.2 us on the device, 4.9 TB/s with
// the launch; 15.6 with the rows loaded after the block table).  A decode step is
// one warp per (request, head) and tensor and the chain lengths -> block table ->
// scale -> store (64 requests: 2.6 us).
#include <cuda_bf16.h>

#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"

namespace pfkv {
namespace {

struct BlockAppendArgs {
  const uint16_t* x[2];  // K, V sources (bf16 bits) [T][H][D]
  uint8_t* cache[2];     // [pages][H][P][D]
  float* scale[2];       // [pages][H]
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* new_start;  // [B + 1]
  int B, T, H, D, P, max_pages, max_new, span;  // span: pages max_new tokens can touch
  int64_t num_pages;
};

// Bits of the smallest power of two s >= 2^-126 with a <= 448 s = 1.75 2^8 s.
__device__ __forceinline__ uint32_t need_bits(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e) << 23;
}

__device__ __forceinline__ float amax16(const uint4& lo, const uint4& hi) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
  return m;
}

__device__ __forceinline__ uint4 encode16(const uint4& lo, const uint4& hi, float inv) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t p[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t q0 = w[2 * k], q1 = w[2 * k + 1];
    p[k] = (uint32_t)f32x2_to_e4m3x2(bf16_lo(q0) * inv, bf16_hi(q0) * inv) |
           ((uint32_t)f32x2_to_e4m3x2(bf16_lo(q1) * inv, bf16_hi(q1) * inv) << 16);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float f) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(codes, lo, hi);
  return (uint32_t)f32x2_to_e4m3x2(f16_lo(lo) * f, f16_hi(lo) * f) |
         ((uint32_t)f32x2_to_e4m3x2(f16_lo(hi) * f, f16_hi(hi) * f) << 16);
}

// One CTA per (request, touched page, head) of K or V.  A thread keeps up to
// kHold 16-element pieces of the page's new rows in registers between the
// maximum and the conversion (the launch gives the block enough threads that
// all of them fit for pages of up to 2048 pieces, 256 rows of head_dim 128 or 64 of
// 512; larger pages read the rest again).
// The rows' place does not depend on the page, so they are on their way while the
// block table and the old scale are read.  kChunks: 16-element pieces of a row, or
// 0 where it is not known beforehand.
constexpr int kHold = 4;
constexpr int kMaxThreads = 512;

template <int kChunks>
__global__ void __launch_bounds__(kMaxThreads) kv_append_block_kernel(const BlockAppendArgs a) {
  __shared__ float warp_max[kMaxThreads / 32];
  const int which = blockIdx.y;
  const int h = (int)(blockIdx.x % a.H);
  const int bi = (int)(blockIdx.x / a.H);
  const int i = bi % a.span, b = bi / a.span;
  const int s0 = a.new_start[b], n = a.new_start[b + 1] - s0, L = a.context_lens[b];
  // a request whose numbers do not fit together is left alone
  if (n <= 0 || n > a.max_new || s0 < 0 || n > a.T - s0 || n > L || (int64_t)L > (int64_t)a.max_pages * a.P) return;
  const int t0 = L - n;               // position of the first new token
  const int logical = t0 / a.P + i;
  if ((int64_t)logical * a.P >= L) return;
  const int base = logical * a.P;
  const int lo = max(t0 - base, 0), hi = min(L - base, a.P);  // the page's new rows
  const int chunks = kChunks ? kChunks : a.D >> 4;
  const uint16_t* const src =
      (which ? a.x[1] : a.x[0]) + ((int64_t)(s0 + base + lo - t0) * a.H + h) * a.D;
  const int64_t row_stride = (int64_t)a.H * a.D;
  const int pieces = (hi - lo) * chunks;

  uint4 x0[kHold], x1[kHold];
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int j = threadIdx.x + k * blockDim.x;
    if (j < pieces) {
      const int r = j / chunks, c = j - r * chunks;
      const uint4* p = reinterpret_cast<const uint4*>(src + r * row_stride + c * 16);
      x0[k] = __ldcs(p);
      x1[k] = __ldcs(p + 1);
    }
  }
  const int page = a.block_tables[(int64_t)b * a.max_pages + logical];
  if (page < 0 || (int64_t)page >= a.num_pages) return;  // skipped; validate_tables reports
  const int64_t sidx = (int64_t)page * a.H + h;
  float* const scale = (which ? a.scale[1] : a.scale[0]) + sidx;
  uint8_t* const dst = (which ? a.cache[1] : a.cache[0]) + sidx * a.P * a.D;
  // a stored scale that is none (never written) counts as 0
  const float stored = lo > 0 ? *scale : 0.f;
  const float old = stored > 0.f ? stored : 0.f;
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (threadIdx.x + k * blockDim.x < pieces) m = fmaxf(m, amax16(x0[k], x1[k]));
  for (int j = threadIdx.x + kHold * blockDim.x; j < pieces; j += blockDim.x) {
    const int r = j / chunks, c = j - r * chunks;
    const uint4* p = reinterpret_cast<const uint4*>(src + r * row_stride + c * 16);
    m = fmaxf(m, amax16(p[0], p[1]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (blockDim.x > 32) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
    m = warp_max[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) m = fmaxf(m, warp_max[w]);
  } else {
    __syncwarp();
  }
  // every thread has read the old scale and its pieces' maximum is in m
  const float s = fmaxf(old, __uint_as_float(need_bits(m)));
  const float inv = 1.f / s;  // exact: s is a power of two
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int j = threadIdx.x + k * blockDim.x;
    if (j < pieces) *reinterpret_cast<uint4*>(dst + (int64_t)lo * a.D + (int64_t)j * 16) = encode16(x0[k], x1[k], inv);
  }
  for (int j = threadIdx.x + kHold * blockDim.x; j < pieces; j += blockDim.x) {
    const int r = j / chunks, c = j - r * chunks;
    const uint4* p = reinterpret_cast<const uint4*>(src + r * row_stride + c * 16);
    *reinterpret_cast<uint4*>(dst + (int64_t)lo * a.D + (int64_t)j * 16) = encode16(p[0], p[1], inv);
  }
  if (s > old) {
    if (lo > 0) {  // earlier rows move to the larger scale
      const float f = old * inv;
      for (int j = threadIdx.x; j < lo * chunks; j += blockDim.x) {
        uint4* p = reinterpret_cast<uint4*>(dst + (int64_t)j * 16);
        const uint4 v = *p;
        *p = make_uint4(rescale4(v.x, f), rescale4(v.y, f), rescale4(v.z, f), rescale4(v.w, f));
      }
    }
    if (threadIdx.x == 0) *scale = s;
  }
}

}  // namespace
}  // namespace pfkv

extern "C" int pfkv_kv_append_fp8_block(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                                        float* k_scales, float* v_scales, const int32_t* block_tables,
                                        int max_pages_per_seq, const int32_t* context_lens,
                                        const int32_t* new_start, int batch, int num_tokens, int max_new_len,
                                        int num_kv_heads, int head_dim, int page_size, int64_t num_pages,
                                        pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  if (batch < 0 || num_tokens < 0 || max_new_len < 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 ||
      num_pages <= 0 || max_pages_per_seq <= 0)
    return fail(PFKV_ERR_INVALID_ARG, "kv_append_fp8_block: bad sizes");
  if (head_dim % 16 != 0)
    return fail(PFKV_ERR_UNSUPPORTED, "kv_append_fp8_block: head_dim %d not a multiple of 16", head_dim);
  if ((int64_t)max_pages_per_seq * page_size >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "kv_append_fp8_block: block table too long");
  if ((int64_t)page_size * head_dim >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "kv_append_fp8_block: page too large");
  if (batch == 0 || num_tokens == 0 || max_new_len == 0) return PFKV_OK;
  const bool has_v = v_new || v_cache || v_scales;
  if (!k_new || !k_cache || !k_scales || !block_tables || !context_lens || !new_start)
    return fail(PFKV_ERR_INVALID_ARG, "kv_append_fp8_block: null pointer");
  if (has_v && (!v_new || !v_cache || !v_scales))
    return fail(PFKV_ERR_INVALID_ARG, "kv_append_fp8_block: v_new, v_cache and v_scales must all be set or all NULL");
  if (!aligned(k_new, 16) || !aligned(k_cache, 16) || !aligned(k_scales, 4) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(new_start, 4) ||
      (has_v && (!aligned(v_new, 16) || !aligned(v_cache, 16) || !aligned(v_scales, 4))))
    return fail(PFKV_ERR_INVALID_ARG, "kv_append_fp8_block: misaligned pointer");
  BlockAppendArgs a;
  a.x[0] = static_cast<const uint16_t*>(k_new);
  a.x[1] = static_cast<const uint16_t*>(v_new);
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(v_cache);
  a.scale[0] = k_scales;
  a.scale[1] = v_scales;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.new_start = new_start;
  a.B = batch;
  a.T = num_tokens;
  a.H = num_kv_heads;
  a.D = head_dim;
  a.P = page_size;
  a.max_pages = max_pages_per_seq;
  a.max_new = max_new_len < num_tokens ? max_new_len : num_tokens;
  int64_t span = ((int64_t)a.max_new + page_size - 2) / page_size + 1;
  if (span > max_pages_per_seq) span = max_pages_per_seq;
  a.span = (int)span;
  a.num_pages = num_pages;
  const int64_t blocks = (int64_t)batch * span * num_kv_heads;
  if (blocks > 0x7FFFFFFF) return fail(PFKV_ERR_UNSUPPORTED, "kv_append_fp8_block: too many pages");
  // threads: the new rows of one page, kHold pieces each; a decode step is one warp
  const int64_t rows = a.max_new < page_size ? a.max_new : page_size;
  int64_t threads = (rows * (head_dim / 16) + kHold * 32 - 1) / (kHold * 32) * 32;
  if (threads > kMaxThreads) threads = kMaxThreads;
  const dim3 grid((unsigned)blocks, has_v ? 2 : 1);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (head_dim == 128)
    kv_append_block_kernel<8><<<grid, (unsigned)threads, 0, s>>>(a);
  else
    kv_append_block_kernel<0><<<grid, (unsigned)threads, 0, s>>>(a);
  return check_cuda("kv_append_fp8_block launch");
}
