// copy_pages.cu -- pages copied within the caches of all layers, in one launch.
//
// Bound by HBM: every page is read once and written once.  A warp copies up to 2 KB
// of one page of one array (four 16-byte loads a lane, in flight together); K and V
// pages, scales and bounds of every layer are units of the same list, so that one
// launch takes a few small pages and many large ones alike.  1,361 pages of 64 KB in
// two arrays, 357 MB: 52.9 us on the device, 6.74 TB/s, a plain copy's rate; 64 pages
// of 16 KB in 64 arrays with their scales, 138 MB: 22.8; one page: 2.0.  4 KB a warp
// in one go took 59.7 us of the first (fewer warps for the registers), stores without
// the streaming policy 56.8, blocks of 256 threads 53.2.
#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"

namespace pfkv {
namespace {

constexpr int kMaxArrays = 128;  // of a launch: its arguments stay below 4 KB
constexpr int kUnit = 2048;      // bytes of a page that a warp copies
constexpr int kThreads = 128;

struct CopyArray {
  char* base;
  int64_t stride;
  int bytes;
  int first_unit : 28;  // units of the arrays before it
  unsigned width : 4;   // log2 of the widest access that its alignment allows
};

struct CopyArgs {
  const int2* pairs;
  int32_t* status;
  int64_t num_pages, total;  // total: (pair, unit)s
  int num_arrays, units;     // units of one pair
  CopyArray array[kMaxArrays];
};

template <class T>
__device__ __forceinline__ void copy_part(char* dst, const char* src, int bytes, int lane) {
  constexpr int kStep = 4;
  const int n = bytes / (int)sizeof(T);
  T* const d = reinterpret_cast<T*>(dst);
  const T* const s = reinterpret_cast<const T*>(src);
  for (int i0 = lane; i0 < n; i0 += 32 * kStep) {
    T v[kStep];
#pragma unroll
    for (int k = 0; k < kStep; ++k)
      if (i0 + 32 * k < n) v[k] = __ldcs(s + i0 + 32 * k);
#pragma unroll
    for (int k = 0; k < kStep; ++k)
      if (i0 + 32 * k < n) __stcs(d + i0 + 32 * k, v[k]);
  }
}

__global__ void __launch_bounds__(kThreads, 8) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < a.total; w += step) {
    const int64_t i = w / a.units;
    const int u = (int)(w - i * a.units);
    const int2 pair = a.pairs[i];
    const bool padding = pair.x < 0 || pair.y < 0;
    const bool bad = !padding && (pair.x >= a.num_pages || pair.y >= a.num_pages);
    if (a.status && u == 0 && lane == 0) a.status[i] = bad ? kErrBadPage : 0;
    if (padding || bad || pair.x == pair.y) continue;
    int lo = 0, hi = a.num_arrays - 1;  // the last array with first_unit <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.array[mid].first_unit <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    const CopyArray& x = a.array[lo];
    const int at = (u - x.first_unit) * kUnit;
    const int bytes = min(kUnit, x.bytes - at);
    const char* const src = x.base + pair.x * x.stride + at;
    char* const dst = x.base + pair.y * x.stride + at;
    switch (x.width) {
      case 4: copy_part<uint4>(dst, src, bytes, lane); break;
      case 3: copy_part<uint2>(dst, src, bytes, lane); break;
      case 2: copy_part<uint32_t>(dst, src, bytes, lane); break;
      case 1: copy_part<uint16_t>(dst, src, bytes, lane); break;
      default: copy_part<uint8_t>(dst, src, bytes, lane); break;
    }
  }
}

}  // namespace
}  // namespace pfkv

extern "C" int pfkv_copy_pages(const pfkv_paged_array* arrays, int num_arrays, const int32_t* pairs, int num_pairs,
                               int64_t num_pages, int32_t* pair_status, pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  if (num_arrays < 0 || num_pairs < 0 || num_pages <= 0) return fail(PFKV_ERR_INVALID_ARG, "copy_pages: bad sizes");
  if (num_arrays > 0 && !arrays) return fail(PFKV_ERR_INVALID_ARG, "copy_pages: null arrays");
  for (int k = 0; k < num_arrays; ++k) {
    const pfkv_paged_array& x = arrays[k];
    if (!x.base || x.page_bytes <= 0 || x.page_stride < x.page_bytes)
      return fail(PFKV_ERR_INVALID_ARG, "copy_pages: array %d: null, or pages of %lld bytes %lld apart", k,
                  (long long)x.page_bytes, (long long)x.page_stride);
    if (x.page_bytes >= (int64_t)1 << 31)
      return fail(PFKV_ERR_UNSUPPORTED, "copy_pages: array %d: pages of %lld bytes", k, (long long)x.page_bytes);
    if (x.page_stride > INT64_MAX / num_pages)
      return fail(PFKV_ERR_INVALID_ARG, "copy_pages: array %d: pages %lld bytes apart", k, (long long)x.page_stride);
  }
  if (num_pairs == 0 || num_arrays == 0) return PFKV_OK;
  if (!pairs || !aligned(pairs, 8) || (pair_status && !aligned(pair_status, 4)))
    return fail(PFKV_ERR_INVALID_ARG, "copy_pages: null or misaligned pointer (pairs start on 8 bytes)");
  if (arrays_meet(pairs, 8ull * num_pairs, pair_status, 4ull * num_pairs))
    return fail(PFKV_ERR_INVALID_ARG, "copy_pages: pair_status overlaps pairs");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CopyArgs a;
  a.pairs = reinterpret_cast<const int2*>(pairs);
  a.num_pages = num_pages;
  for (int done = 0; done < num_arrays;) {
    int64_t units = 0;
    int n = 0;
    for (; n < kMaxArrays && done + n < num_arrays; ++n) {
      const pfkv_paged_array& x = arrays[done + n];
      const int64_t more = (x.page_bytes + kUnit - 1) / kUnit;
      if (units + more >= 1 << 27) break;  // the next launch's; one array alone always fits
      CopyArray& y = a.array[n];
      y.base = static_cast<char*>(x.base);
      y.stride = x.page_stride;
      y.bytes = (int)x.page_bytes;
      y.first_unit = (int)units;
      const uint64_t all = reinterpret_cast<uintptr_t>(x.base) | (uint64_t)x.page_bytes | (uint64_t)x.page_stride;
      unsigned width = 0;
      while (width < 4 && all % (2u << width) == 0) ++width;
      y.width = width;
      units += more;
    }
    a.num_arrays = n;
    a.units = (int)units;
    a.total = units * num_pairs;
    a.status = done == 0 ? pair_status : nullptr;
    const int64_t blocks = (a.total + kThreads / 32 - 1) / (kThreads / 32);
    copy_pages_kernel<<<(unsigned)(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF), kThreads, 0, s>>>(a);
    if (int rc = check_cuda("copy_pages launch")) return rc;
    done += n;
  }
  return PFKV_OK;
}
