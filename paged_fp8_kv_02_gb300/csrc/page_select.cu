// page_select.cu -- the pages a decode query attends: every page of a request
// scored per KV head from its key bounds, the best ones listed in order.
//
// For request b and KV head h with the G query heads of its group:
//   whole numbers  n_g[d] = rint(q_g[d] 2^(14 - e)), e the frexp exponent of the
//                  group's largest |q| (so |n| <= 2^14),
//   parts          S+[d] = sum_g max(n_g[d], 0),  S-[d] = sum_g min(n_g[d], 0),
//                  Q+-[d] = rint(S+-[d] / 2^j), j >= 0 the smallest with
//                  max |S+-| <= 127 2^j,
//   score(page)    (sum_d Q+[d] hi[d] + Q-[d] lo[d]) * s(page) [* ks(page, h)],
// with lo, hi and s the page's bounds and their scale (page_bounds.cu) and ks its
// K scale when scales are per block.  sum_d max(q lo, q hi) is at least q . k for
// every key k of the page, and summed over the group it separates into one
// positive and one negative query: 256 products a page however many heads.
// Numbers are integers of 8 bits, sums stay below 2^23 and the scales are powers
// of two, so a score is exact and the same in any order of summation: ties are
// real ties, and go to the lower page.
//
// One cluster of up to 8 CTAs per (request, KV head).  Each CTA scores a
// contiguous share of the pages (half a warp reads the 256 bytes of a page's
// bounds; dp4a) and keeps the scores in shared memory as order-preserving
// 32-bit keys.  The K-th largest key is found by its digits, 8 bits a round:
// the CTAs' 256-bin histograms are summed through distributed shared memory,
// one cluster barrier a round.  Pages above it, and the lowest-numbered ones
// equal to it, are then written in order from prefix sums of the counts.  No
// score goes to global memory and one launch does it all; large calls are
// bounded by reading the bounds once, small ones by the chain of rounds.
#include <cuda_bf16.h>
#include <float.h>

#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"
#include "pfkv_tc.cuh"

namespace pfkv {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 8;            // pages per half warp and step
constexpr int kMaxCluster = 8;       // portable cluster size
constexpr int kMaxShare = 49152;     // pages per CTA: keys of 4 bytes in shared memory

struct SelectArgs {
  int32_t* selected;  // [B][Hkv][K]
  int32_t* status;    // [B][Hkv] or null
  const uint16_t* q;
  const int8_t* bounds;
  const float* bound_scales;
  const float* k_scales;  // [pages][Hkv] or null
  const int32_t* block_tables;
  const int32_t* context_lens;
  int Hq, Hkv, G, P, max_pages, K, sink, recent;
  int64_t num_pages;
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 (an underflow) counts as 0
  return u ^ ((u & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) select_pages_kernel(const SelectArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[4][256];
  __shared__ __align__(16) int8_t qs[2 * kD];  // Q-, then Q+: the order of a page's bounds
  __shared__ float red_f[kWarps];
  __shared__ int red_i[kWarps];
  __shared__ uint64_t red_u[kWarps];
  __shared__ uint32_t digit_of, above_of, in_bin_of;
  __shared__ uint32_t totals[3];  // this CTA's keys above the threshold, equal to it, and error bits

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nc = (int)tc::cluster_nctarank(), rank = (int)tc::cluster_ctarank();
  const int64_t unit = blockIdx.x / nc;
  const int b = (int)(unit / a.Hkv), h = (int)(unit % a.Hkv);
  int32_t* const out = a.selected + unit * a.K;

  int bits = 0;
  int L = a.context_lens[b];
  const int cap = a.max_pages * a.P;
  if (L < 0 || L > cap) {
    bits = kErrBadContext;
    L = L < 0 ? 0 : cap;
  }
  const int npages = (L + a.P - 1) / a.P;
  if (npages <= a.K) {  // every page is listed (the whole cluster takes this path)
    if (rank == 0) {
      for (int i = tid; i < a.K; i += kThreads) out[i] = i < npages ? i : -1;
      if (a.status && tid == 0) a.status[unit] = bits;
    }
    return;
  }
  const int share = (npages + nc - 1) / nc;
  const int first = min(rank * share, npages), count = min(share, npages - first);

  // ---------------- the group's query in 8-bit whole numbers
  for (int i = tid; i < 4 * 256; i += kThreads) hist[i >> 8][i & 255] = 0;
  {
    const uint16_t* qp = a.q + ((int64_t)b * a.Hq + (int64_t)h * a.G) * kD + tid;
    float m = 0.f;
    if (tid < kD)
      for (int g = 0; g < a.G; ++g) m = fmaxf(m, fabsf(bf16_lo(qp[g * kD])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0) red_f[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red_f[0], red_f[1]), fmaxf(red_f[2], red_f[3]));  // warps 0-3 hold the 128 channels
    int e = 0;
    frexpf(fminf(m, FLT_MAX), &e);
    int sp = 0, sn = 0;
    if (tid < kD)
      for (int g = 0; g < a.G; ++g) {
        const float x = rintf(ldexpf(bf16_lo(qp[g * kD]), 14 - e));
        const int n = (int)fminf(fmaxf(x, -16384.f), 16384.f);
        sp += max(n, 0);
        sn += min(n, 0);
      }
    int most = max(sp, -sn);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) red_i[warp] = most;
    __syncthreads();
    most = max(max(red_i[0], red_i[1]), max(red_i[2], red_i[3]));
    int j = 0;
    while ((127 << j) < most) ++j;
    if (tid < kD) {  // S < 2^24 and the power of two: exact until the rounding
      qs[tid] = (int8_t)__float2int_rn(ldexpf((float)sn, -j));
      qs[kD + tid] = (int8_t)__float2int_rn(ldexpf((float)sp, -j));
    }
    __syncthreads();
  }

  // ---------------- scores of this CTA's pages
  {
    const int l16 = lane & 15, hw = tid >> 4;  // half warp of the CTA
    const uint4 qv = *reinterpret_cast<const uint4*>(qs + 16 * l16);
    const int own = l16 >> 1;  // the page of the eight whose sum this lane ends up with
    const int32_t* table = a.block_tables + (int64_t)b * a.max_pages + first;
    constexpr int kStep = kThreads / 16 * kBatch;
    int next = -1;
    if (hw * kBatch + own < count) next = __ldg(table + hw * kBatch + own);
    for (int i0 = hw * kBatch; i0 - hw * kBatch < count; i0 += kStep) {
      const int i = i0 + own;
      int page = next;
      next = i + kStep < count ? __ldg(table + i + kStep) : -1;
      const bool there = i < count;
      if (there && (page < 0 || (int64_t)page >= a.num_pages)) bits |= kErrBadPage;
      const bool ok = there && page >= 0 && (int64_t)page < a.num_pages;
      const int64_t at = ok ? (int64_t)page * a.Hkv + h : 0;  // entry 0 stands in for one that is not there
      float scale = 0.f;
      if (!(l16 & 1)) {
        scale = __ldg(a.bound_scales + at);
        if (a.k_scales) scale *= __ldg(a.k_scales + at);
      }
      uint4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int64_t pu = __shfl_sync(0xFFFFFFFFu, at, 2 * u, 16);
        v[u] = __ldg(reinterpret_cast<const uint4*>(a.bounds + pu * (2 * kD)) + l16);
      }
      int s[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        s[u] = __dp4a((int)v[u].x, (int)qv.x,
                      __dp4a((int)v[u].y, (int)qv.y, __dp4a((int)v[u].z, (int)qv.z, __dp4a((int)v[u].w, (int)qv.w, 0))));
      // sums over the 16 lanes, each step halving the pages a lane holds: page
      // `own` ends in lanes 2 own and 2 own + 1
      int s4[4], s2[2];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        s4[u] = ((l16 & 8) ? s[u + 4] : s[u]) + __shfl_xor_sync(0xFFFFFFFFu, (l16 & 8) ? s[u] : s[u + 4], 8);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        s2[u] = ((l16 & 4) ? s4[u + 2] : s4[u]) + __shfl_xor_sync(0xFFFFFFFFu, (l16 & 4) ? s4[u] : s4[u + 2], 4);
      int sum = ((l16 & 2) ? s2[1] : s2[0]) + __shfl_xor_sync(0xFFFFFFFFu, (l16 & 2) ? s2[0] : s2[1], 2);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      if (there && !(l16 & 1)) {
        uint32_t key = ok ? order_key((float)sum * scale) : 0u;
        const int index = first + i;
        if (index < a.sink || index >= npages - a.recent) key = 0xFFFFFFFFu;  // above every finite score
        keys[i] = key;
      }
    }
  }
  __syncthreads();

  // ---------------- the K-th largest key, digit by digit
  uint32_t prefix = 0, mask = 0;
  uint32_t want = (uint32_t)a.K;  // of the keys that agree with the prefix, how many are listed
#pragma unroll 1
  for (int p = 0; p < 4; ++p) {
    const int shift = 24 - 8 * p;
    for (int i = tid; i < count; i += kThreads) {
      const uint32_t k = keys[i];
      if ((k & mask) == prefix) atomicAdd(&hist[p][(k >> shift) & 255], 1u);
    }
    __syncwarp();
    tc::cluster_sync();
    uint32_t n = 0;
    const uint32_t mine = smem_u32(&hist[p][tid]);
    for (int r = 0; r < nc; ++r) n += tc::ld_cluster_u32(tc::mapa(mine, r));
    // keys in this bin or a higher one
    uint32_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_down_sync(0xFFFFFFFFu, sum, o);
      if (lane + o < 32) sum += x;
    }
    if (lane == 0) red_i[warp] = (int)sum;
    __syncthreads();
    for (int w = warp + 1; w < kWarps; ++w) sum += (uint32_t)red_i[w];
    if (sum >= want && sum - n < want) {  // one bin only
      digit_of = (uint32_t)tid;
      above_of = sum - n;
      in_bin_of = n;
    }
    __syncthreads();
    prefix |= digit_of << shift;
    mask |= 255u << shift;
    want -= above_of;
    if (in_bin_of == want) break;  // the whole bin is listed: the same in every CTA
    __syncthreads();  // digit_of and red_i are written again in the next round
  }

  // ---------------- the list, in order: each thread a contiguous piece of odd
  // length (so that the threads' shared-memory reads spread over the banks)
  const int piece = ((count + kThreads - 1) / kThreads) | 1;
  const int p0 = min(tid * piece, count), p1 = min(p0 + piece, count);
  uint32_t gt = 0, eq = 0;
  for (int i = p0; i < p1; ++i) {
    const uint32_t k = keys[i] & mask;
    gt += k > prefix;
    eq += k == prefix;
  }
  const uint64_t own = ((uint64_t)gt << 32) | eq;
  uint64_t inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) red_u[warp] = inc;
  if (tid == 0) totals[2] = 0;
  __syncthreads();
  bits = __reduce_or_sync(0xFFFFFFFFu, bits);
  if (lane == 0 && bits) atomicOr(&totals[2], (uint32_t)bits);
  uint64_t before = inc - own;
  for (int w = 0; w < warp; ++w) before += red_u[w];
  if (tid == kThreads - 1) {
    const uint64_t all = before + own;
    totals[0] = (uint32_t)(all >> 32);
    totals[1] = (uint32_t)all;
  }
  __syncwarp();
  tc::cluster_sync();
  uint32_t gt_before = (uint32_t)(before >> 32), eq_before = (uint32_t)before, all_bits = 0;
  const uint32_t t0 = smem_u32(totals);
  for (int r = 0; r < nc; ++r) {
    const uint32_t at = tc::mapa(t0, r);
    if (r < rank) {
      gt_before += tc::ld_cluster_u32(at);
      eq_before += tc::ld_cluster_u32(at + 4);
    }
    all_bits |= tc::ld_cluster_u32(at + 8);
  }
  for (int i = p0; i < p1; ++i) {
    const uint32_t k = keys[i] & mask;
    const bool above = k > prefix, equal = k == prefix;
    if (above || (equal && eq_before < want)) out[gt_before + min(eq_before, want)] = first + i;
    gt_before += above;
    eq_before += equal;
  }
  if (a.status && rank == 0 && tid == 0) a.status[unit] = (int32_t)all_bits;
  __syncwarp();
  tc::cluster_sync();  // no CTA leaves while another may still read its shared memory
}

// CTAs per (request, KV head): enough clusters' CTAs for about two on every
// SM, as long as a CTA keeps at least 256 pages to score; more where a share
// would not fit in shared memory.
int cluster_size(int64_t units, int max_pages, int sms) {
  int c = 1;
  while (c < kMaxCluster && units * c < 2 * (int64_t)sms && max_pages / (2 * c) >= 256) c *= 2;
  while (c < kMaxCluster && (max_pages + c - 1) / c > kMaxShare) c *= 2;
  return c;
}

}  // namespace
}  // namespace pfkv

extern "C" int pfkv_select_pages(int32_t* selected, const void* q, const int8_t* bounds, const float* bound_scales,
                                 const float* k_scales, const int32_t* block_tables, int max_pages_per_seq,
                                 const int32_t* context_lens, int batch, int num_q_heads, int num_kv_heads,
                                 int head_dim, int page_size, int64_t num_pages, int top_pages, int sink_pages,
                                 int recent_pages, int32_t* unit_status, pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || num_pages <= 0 ||
      max_pages_per_seq <= 0 || top_pages <= 0 || sink_pages < 0 || recent_pages < 0)
    return fail(PFKV_ERR_INVALID_ARG, "select_pages: bad sizes");
  if (num_q_heads % num_kv_heads != 0)
    return fail(PFKV_ERR_INVALID_ARG, "select_pages: num_q_heads %% num_kv_heads != 0");
  if ((int64_t)sink_pages + recent_pages > top_pages)
    return fail(PFKV_ERR_INVALID_ARG, "select_pages: sink_pages + recent_pages > top_pages");
  const int G = num_q_heads / num_kv_heads;
  if (G > 16) return fail(PFKV_ERR_UNSUPPORTED, "select_pages: group size %d > 16", G);
  if (head_dim != kD) return fail(PFKV_ERR_UNSUPPORTED, "select_pages: head_dim %d != 128", head_dim);
  if ((int64_t)max_pages_per_seq * page_size >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "select_pages: block table too long");
  if (max_pages_per_seq > kMaxCluster * kMaxShare)
    return fail(PFKV_ERR_UNSUPPORTED, "select_pages: more than %d pages per request", kMaxCluster * kMaxShare);
  const int64_t units = (int64_t)batch * num_kv_heads;
  if (units > 0x7FFFFFFF / kMaxCluster) return fail(PFKV_ERR_UNSUPPORTED, "select_pages: batch too large");
  if (batch == 0) return PFKV_OK;
  if (!selected || !q || !bounds || !bound_scales || !block_tables || !context_lens)
    return fail(PFKV_ERR_INVALID_ARG, "select_pages: null pointer");
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(selected, 4) || !aligned(bound_scales, 4) ||
      (k_scales && !aligned(k_scales, 4)) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      (unit_status && !aligned(unit_status, 4)))
    return fail(PFKV_ERR_INVALID_ARG, "select_pages: misaligned pointer");
  SelectArgs a;
  a.selected = selected;
  a.status = unit_status;
  a.q = static_cast<const uint16_t*>(q);
  a.bounds = bounds;
  a.bound_scales = bound_scales;
  a.k_scales = k_scales;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.G = G;
  a.P = page_size;
  a.max_pages = max_pages_per_seq;
  a.K = top_pages;
  a.sink = sink_pages;
  a.recent = recent_pages;
  a.num_pages = num_pages;
  const int c = cluster_size(units, max_pages_per_seq, device_sm_count());
  const int smem = (max_pages_per_seq + c - 1) / c * 4;
  static std::atomic<uint64_t> smem_set{0};
  const int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(select_pages_kernel), kMaxShare * 4, smem_set,
                                      "select_pages set smem attribute");
  if (rc != PFKV_OK) return rc;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * c));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, select_pages_kernel, a) != cudaSuccess) return check_cuda("select_pages launch");
  return check_cuda("select_pages launch");
}
