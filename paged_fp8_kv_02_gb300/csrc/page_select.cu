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
// positive and one negative query: 256 products a page however many heads.  (Bounds
// of a page's keys and the largest product they allow are the score of Tang et al.,
// "Quest: query-aware sparsity for efficient long-context LLM inference", 2024.)
// Numbers are integers of 8 bits, sums stay below 2^23 and the scales are powers
// of two, so a score is exact and the same in any order of summation: ties are
// real ties, and go to the lower page.  A score beyond fp32's range (keys above
// about 2^100) counts as the largest number.
//
// Two stages.  Scores: a warp takes some tens of consecutive pages of one
// (request, KV head), makes the 8-bit query for itself, and reads the 256 bytes
// of a page's bounds with half a warp (dp4a, two steps of four pages in flight
// per half; table entries and scales for 32 pages at a time, a group ahead).
// Scores are kept in fp32, 1/64 of the bytes read, beside each warp's smallest and
// largest; +inf stands for a page that is listed whatever its score and -inf for one
// outside the pool.
// List: one CTA per (request, KV head) finds the K-th largest score and writes the
// list.  A histogram over 256 equal parts of the scores' range says which part
// holds it; that part's scores, usually few, are compared with one another, or,
// where scores repeat, counted by the digits of an order-preserving key, 8 bits a
// round.  (Parts of the range spread the shared-memory atomics; a float's leading
// digits would put most scores into a few bins.)  Pages above the threshold, and
// the lowest-numbered ones equal to it, are written in order from prefix sums.  The
// digits cost more than comparing: with all scores equal the three workloads below
// take 10.8, 63.6 and 46.5 us.
//
// Few short lists run both stages in one launch: a cluster of 1 to 8 CTAs per list
// scores into its first CTA's shared memory, and that CTA lists.  Otherwise two
// kernels with the scores in the workspace: the first is spread evenly over all SMs
// with neighbouring warps on neighbouring heads, so that a page's bounds are read
// as one run, and the second is resident and waiting when the first ends.
// Device time: one request of 128K tokens (8 lists of 2K pages) 7.9 us, a chain of
// loads and block barriers; 64 requests of up to 32K tokens (512 lists of up to 2K
// pages, 55 MB) 20.4 us, of which the list takes about 4; 8 requests of 256K-1M
// tokens (64 lists of 4K-16K pages, 153 MB) 37.5 us: scores 26 us at 5.9 TB/s, and
// the longest list 8 us on its SM.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"
#include "pfkv_tc.cuh"

namespace pfkv {
namespace {

constexpr int kD = 128;
constexpr int kMaxG = 16;
constexpr int kScoreWarps = 8;
constexpr int kBatch = 4;                 // pages per half warp and step
constexpr int kStep = 2 * kBatch;         // pages per warp and step
constexpr int kBins = 256;
constexpr int kMaxListThreads = 1024;
constexpr int kMaxCluster = 8;             // CTAs of a list in one launch
constexpr int kFusedPages = 2048;          // pages that such a list may have
constexpr int kCandidates = 512;           // scores compared with one another instead of by digits

// What a warp leaves beside its scores: the smallest and largest of those that
// are not set by rule.
struct __align__(16) Extent {
  float low, high;
  int32_t bits;     // errors met
  int32_t unused;
};

struct SelectArgs {
  int32_t* selected;  // [B][Hkv][K]
  int32_t* status;    // [B][Hkv] or null
  float* scores;      // [B * Hkv][stride]
  Extent* extents;    // [B * Hkv][chunks]
  const uint16_t* q;
  const int8_t* bounds;
  const float* bound_scales;
  const float* k_scales;  // [pages][Hkv] or null
  const int32_t* block_tables;
  const int32_t* context_lens;
  int B, Hq, Hkv, G, P, max_pages, K, sink, recent;
  int chunk, chunks, runs;  // pages per warp of the first kernel; warps, and CTAs, per list
  int64_t num_pages, stride;
};

// A whole number that grows with x.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_order_key(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// The cluster's barrier in two halves, by every thread of the cluster.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Generic address of the same shared array in the cluster's first CTA.
template <class T>
__device__ __forceinline__ T* map_to_first(T* p) {
  uint64_t r;
  asm("mapa.u64 %0, %1, 0;" : "=l"(r) : "l"(p));
  return reinterpret_cast<T*>(r);
}

__device__ __forceinline__ float warp_min(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fminf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// Pages of request b's context; *bits: a length outside the table is clamped.
__device__ __forceinline__ int pages_of(const SelectArgs& a, int b, int* bits) {
  int L = a.context_lens[b];
  const int cap = a.max_pages * a.P;
  *bits = 0;
  if (L < 0 || L > cap) {
    *bits = kErrBadContext;
    L = L < 0 ? 0 : cap;
  }
  return (L + a.P - 1) / a.P;
}

// ------------------------------------------------------------------- scores
struct ScoreShared {
  __align__(16) int8_t q[2 * kD];  // Q-, then Q+: the order of a page's bounds
  uint32_t largest[4], most[4];
};

// The pages first .. first + 8 chunk - 1 of (b, h) by one CTA, chunk to a warp:
// scores to scores[page] and each warp's extent to extents[page / chunk], in global
// memory or in a cluster CTA's shared memory; `ready` is called by every thread
// before the first write.  False, and nothing done, where every page is listed.
// What does not depend on the length or the query is loaded ahead of them: the
// chain is block table -> bounds, and the query is made while those arrive.
template <class Ready>
__device__ __forceinline__ bool score_block(const SelectArgs& a, ScoreShared& sh, int64_t b, int h, int first,
                                            int chunk, float* scores, Extent* extents, Ready ready) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l16 = lane & 15, half = lane >> 4;
  const int own = l16 >> 2;  // the page of the half warp's four whose sum this lane ends up with
  first += warp * chunk;
  const int32_t* table = a.block_tables + b * a.max_pages + first;
  const int room = min(chunk, a.max_pages - first);
  // the table's entries of 32 pages, one per lane
  auto entries = [&](int g) { return 32 * g + lane < room ? __ldg(table + 32 * g + lane) : -1; };
  const int pages0 = entries(0);
  int pages_next = entries(1);
  // thread d < 128: channel d of the group's rows
  uint32_t row[kMaxG];
  {
    const uint16_t* q = a.q + (b * a.Hq + (int64_t)h * a.G) * kD + tid;
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) row[g] = tid < kD && g < a.G ? __ldg(q + g * kD) : 0u;
  }
  int bits;
  const int npages = pages_of(a, (int)b, &bits);
  if (npages <= a.K) return false;
  const int count = max(min(chunk, npages - first), 0);

  float low = INFINITY, high = -INFINITY;
  // the lane's page of a group: its place in the bounds and its scale, in two parts
  // so that nothing waits for them here
  struct Group {
    int at;
    float bs, ks;
  };
  auto look_up = [&](int g, int page) {
    Group x{0, NAN, 1.f};  // entry 0 stands in for one that is not there; its score is no number
    const bool ok = page >= 0 && (int64_t)page < a.num_pages;
    if (32 * g + lane < count && !ok) bits |= kErrBadPage;
    if (ok) {
      x.at = page * a.Hkv + h;
      x.bs = __ldg(a.bound_scales + x.at);
      if (a.k_scales) x.ks = __ldg(a.k_scales + x.at);
    }
    return x;
  };
  struct Step {
    uint4 v[kBatch];
  };
  // bounds of pages 8 s .. 8 s + 7 of a group; read once by one warp: they leave L1
  // and L2 first, and the scales and tables beside them stay
  auto load = [&](Step& st, const Group& x, int g, int s) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int pu = __shfl_sync(0xFFFFFFFFu, x.at, kStep * s + kBatch * half + u);
      st.v[u] = __ldcs(reinterpret_cast<const uint4*>(a.bounds) + (int64_t)pu * (2 * kD / 16) + l16);
    }
  };
  Group cur = look_up(0, pages0);
  Step x, y;
  load(x, cur, 0, 0);

  // ---------------- the group's query in 8-bit whole numbers
  uint32_t largest = 0;
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) largest = max(largest, row[g] & 0x7FFFu);
  largest = __reduce_max_sync(0xFFFFFFFFu, largest);
  if (tid < kD && lane == 0) sh.largest[warp] = largest;
  __syncthreads();
  largest = max(max(sh.largest[0], sh.largest[1]), max(sh.largest[2], sh.largest[3]));
  // 2^(e-1) <= largest < 2^e: by the exponent, or a subnormal's leading bit
  const int e = largest >= 0x7F80u ? 128 : (largest >> 7 ? (int)(largest >> 7) - 126 : (largest ? -101 - __clz((int)largest) : 0));
  // 2^(14 - e) in two exact factors: it can leave fp32's range, its halves cannot
  const int h1 = (14 - e) / 2, h2 = 14 - e - h1;
  const float f1 = __uint_as_float((uint32_t)(127 + h1) << 23), f2 = __uint_as_float((uint32_t)(127 + h2) << 23);
  // S+ and -S-, both as magnitudes
  uint32_t sp = 0, sm = 0;
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    const float n = fminf(fmaxf(rintf(__uint_as_float(row[g] << 16) * f1 * f2), -16384.f), 16384.f);
    sp += (uint32_t)fmaxf(n, 0.f);
    sm += (uint32_t)fmaxf(-n, 0.f);
  }
  uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(sp, sm));
  if (tid < kD && lane == 0) sh.most[warp] = most;
  __syncthreads();
  most = max(max(sh.most[0], sh.most[1]), max(sh.most[2], sh.most[3]));
  int j = 0;
  while ((127u << j) < most) ++j;
  const float f = __uint_as_float((uint32_t)(127 - j) << 23);  // 2^-j
  if (tid < kD) {  // below 2^24 and a power of two: exact until the rounding
    sh.q[tid] = (int8_t)-__float2int_rn((float)sm * f);
    sh.q[kD + tid] = (int8_t)__float2int_rn((float)sp * f);
  }
  __syncthreads();
  const uint4 qv = *reinterpret_cast<const uint4*>(sh.q + 16 * l16);
  ready();
  if (count == 0) return true;

  // ---------------- the warp's pages, two steps of loads in flight
  auto sum_up = [&](const Step& st, float group_scale, int g, int step) {
    int s[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      s[u] = __dp4a((int)st.v[u].x, (int)qv.x,
                    __dp4a((int)st.v[u].y, (int)qv.y,
                           __dp4a((int)st.v[u].z, (int)qv.z, __dp4a((int)st.v[u].w, (int)qv.w, 0))));
    // sums over the 16 lanes, two steps halving the pages a lane holds: page
    // `own` ends in lanes 4 own .. 4 own + 3
    int s2[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      s2[u] = ((l16 & 8) ? s[u + 2] : s[u]) + __shfl_xor_sync(0xFFFFFFFFu, (l16 & 8) ? s[u] : s[u + 2], 8);
    int sum = ((l16 & 4) ? s2[1] : s2[0]) + __shfl_xor_sync(0xFFFFFFFFu, (l16 & 4) ? s2[0] : s2[1], 4);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    const int mine = kStep * step + kBatch * half + own, i = 32 * g + mine;
    const float scale = __shfl_sync(0xFFFFFFFFu, group_scale, mine);
    if (i < count && !(l16 & 3)) {
      const int index = first + i;
      float score = (float)sum * scale + 0.f;  // + 0: -0 (an underflow) counts as 0
      if (index < a.sink || index >= npages - a.recent) {
        score = INFINITY;
      } else if (score != score) {
        score = -INFINITY;  // a page outside the pool, a scale that is none
      } else {
        // beyond the range: the largest number, so that the infinities keep their meaning
        score = fminf(fmaxf(score, -FLT_MAX), FLT_MAX);
        low = fminf(low, score);
        high = fmaxf(high, score);
      }
      scores[index] = score;
    }
  };
#pragma unroll 1
  for (int g = 0; 32 * g < count; ++g) {
    const Group nxt = look_up(g + 1, pages_next);
    pages_next = entries(g + 2);
    float scale = cur.bs * cur.ks;
    if (scale > FLT_MAX) scale = FLT_MAX;  // products with 0 stay 0
    load(y, cur, g, 1);
    sum_up(x, scale, g, 0);
    load(x, cur, g, 2);
    sum_up(y, scale, g, 1);
    load(y, cur, g, 3);
    sum_up(x, scale, g, 2);
    load(x, nxt, g + 1, 0);
    sum_up(y, scale, g, 3);
    cur = nxt;
  }
  low = warp_min(low);
  high = -warp_min(-high);
  bits = (int)__reduce_or_sync(0xFFFFFFFFu, (unsigned)bits);
  if (lane == 0) extents[first / chunk] = Extent{low, high, bits, 0};
  return true;
}

__global__ void __launch_bounds__(kScoreWarps * 32, 4) score_pages_kernel(const SelectArgs a) {
  __shared__ ScoreShared sh;
  grid_launch_dependents();  // the listing kernel may take its place and wait
  const int h = (int)(blockIdx.x % a.Hkv);  // neighbouring CTAs: neighbouring heads of the same pages
  const int64_t br = blockIdx.x / a.Hkv;
  const int run = (int)(br % a.runs);
  const int64_t b = br / a.runs, unit = b * a.Hkv + h;
  const int first = run * kScoreWarps * a.chunk;
  if ((int64_t)first * a.P >= a.context_lens[b]) return;
  score_block(a, sh, b, h, first, a.chunk, a.scores + unit * a.stride, a.extents + unit * a.chunks, [] {});
}

// --------------------------------------------------------------------- lists
// Sum of x over this thread and later ones of the block's first kBins threads
// (others pass 0 and get no answer).
__device__ __forceinline__ uint32_t suffix_sum(uint32_t x, uint32_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_down_sync(0xFFFFFFFFu, x, o);
    if (lane + o < 32) x += y;
  }
  if (warp < kBins / 32 && lane == 0) red[warp] = x;
  __syncthreads();
#pragma unroll
  for (int w = 1; w < kBins / 32; ++w) x += w > warp ? red[w] : 0u;
  return x;
}

struct ListShared {
  uint32_t hist[5][kBins];  // of parts of the range, then of four digits
  float2 cand[kCandidates];  // scores of the part, and which warp's they are
  uint32_t above[kMaxListThreads / 32], equal[kMaxListThreads / 32];  // listed keys of each warp's piece
  float range[2][kMaxListThreads / 32];
  uint32_t bins[kBins / 32];
  uint32_t found[6];
  uint32_t err;
};

// Every page is listed: a CTA writes them.
__device__ __forceinline__ void list_all(const SelectArgs& a, int64_t unit, int npages, int bits) {
  for (int i = threadIdx.x; i < a.K; i += blockDim.x) a.selected[unit * a.K + i] = i < npages ? i : -1;
  if (a.status && threadIdx.x == 0) a.status[unit] = bits;
}

// One CTA: the list of `unit` from its npages > K scores (16-byte aligned) and the
// nchunks extents of their scores; `ready` is called before they are read.
template <class Ready>
__device__ __forceinline__ void list_unit(const SelectArgs& a, ListShared& sh, int64_t unit, int npages,
                                          const float* scores, const Extent* extents, int nchunks, int bits,
                                          Ready ready) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int threads = blockDim.x, warps = threads >> 5;
  int32_t* const out = a.selected + unit * a.K;
  for (int i = tid; i < 5 * kBins; i += threads) sh.hist[i / kBins][i % kBins] = 0;
  if (lane == 0) sh.above[warp] = sh.equal[warp] = 0;
  if (tid == 0) {
    sh.found[3] = 0;
    sh.err = 0;
  }
  // scores: each warp a contiguous piece, 128 at a time, four to a lane
  const int piece = ((npages + warps - 1) / warps + 127) & ~127;
  const int p0 = min(warp * piece, npages), p1 = min(p0 + piece, npages);
  // fn(first index, four scores, how many indices are left); whole warps
  auto piece_at = [&](int i) {
    return i < p1 ? *reinterpret_cast<const float4*>(scores + i) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto each = [&](auto&& fn) {
    int i = p0 + 4 * lane;
    float4 next = piece_at(i);
#pragma unroll 1
    for (; i - 4 * lane < p1; i += 128) {
      const float4 x = next;
      next = piece_at(i + 128);  // on its way while x is looked at
      const float v[4] = {x.x, x.y, x.z, x.w};
      fn(i, v, p1 - i);
    }
  };
  ready();

  float low = INFINITY, high = -INFINITY;
  for (int i = tid; i < nchunks; i += threads) {
    const Extent e = extents[i];
    low = fminf(low, e.low);
    high = fmaxf(high, e.high);
    bits |= e.bits;
  }
  low = warp_min(low);
  high = -warp_min(-high);
  bits = (int)__reduce_or_sync(0xFFFFFFFFu, (unsigned)bits);
  if (lane == 0) {
    sh.range[0][warp] = low;
    sh.range[1][warp] = high;
  }
  __syncthreads();
  if (lane == 0 && bits) atomicOr(&sh.err, (uint32_t)bits);
  low = warp_min(lane < warps ? sh.range[0][lane] : INFINITY);
  high = -warp_min(lane < warps ? -sh.range[1][lane] : INFINITY);

  // ---------------- which of 256 equal parts of the scores' range holds the
  // K-th largest; equal scores, or a range that is no number: one part
  float per = (float)kBins / (high - low);
  if (!(high > low) || !isfinite(per)) per = 0.f;
  auto part_of = [&](float x) {  // grows with x; +inf: the last, or 0 if there is one part
    return min(max(__float2int_rd((x - low) * per), 0), kBins - 1);
  };
  each([&](int, const float (&x)[4], int n) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < n) atomicAdd(&sh.hist[0][part_of(x[c])], 1u);
  });
  uint32_t want = (uint32_t)a.K;  // of the scores of the part, how many are listed
  // the bin that holds the want-th largest, by the block's first 256 threads
  auto find = [&](const uint32_t* bins) {
    __syncthreads();
    const uint32_t n = tid < kBins ? bins[tid] : 0u;
    const uint32_t sum = suffix_sum(n, sh.bins);
    if (tid < kBins && sum >= want && sum - n < want) {  // one bin only
      sh.found[0] = (uint32_t)tid;
      sh.found[1] = sum - n;
      sh.found[2] = n;
    }
    __syncthreads();
    want -= sh.found[1];
  };
  find(sh.hist[0]);
  const int part = (int)sh.found[0];
  const uint32_t in_part = sh.found[2];

  // ---------------- the threshold: listed are the scores above edge and the
  // first `want` equal to it; sh.above and sh.equal count both in each warp's piece
  float edge = 0.f;
  bool whole = false;  // every score equal to edge is listed
  if (in_part <= kCandidates) {  // few: compared with one another
    uint32_t above = 0;
    // below every score of the part, by half a part
    const float floor = part > 0 ? low + ((float)part - 0.5f) / per : -INFINITY;
    each([&](int, const float (&x)[4], int n) {
      if (fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) < floor) return;  // most, where few pages of many are listed
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n && x[c] >= floor) {
          const int at = part_of(x[c]);
          above += at > part;
          if (at == part) sh.cand[atomicAdd(&sh.found[3], 1u)] = make_float2(x[c], __int_as_float(warp));
        }
    });
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    if (lane == 0) sh.above[warp] = above;
    __syncthreads();
    for (uint32_t i = tid; i < in_part; i += threads) {
      const float x = sh.cand[i].x;
      uint32_t gt = 0, eq = 0;
#pragma unroll 4
      for (uint32_t j = 0; j < in_part; ++j) {
        const float o = sh.cand[j].x;
        gt += o > x;
        eq += o == x;
      }
      const int w = __float_as_int(sh.cand[i].y);
      if (gt + eq < want) {  // above the want-th largest
        atomicAdd(&sh.above[w], 1u);
      } else if (gt < want) {  // equal to it: all of these write the same
        atomicAdd(&sh.equal[w], 1u);
        sh.found[0] = __float_as_uint(x);
        sh.found[4] = want - gt;
        sh.found[5] = eq;
      }
    }
    __syncthreads();
    edge = __uint_as_float(sh.found[0]);
    want = sh.found[4];
    whole = sh.found[5] == want;
  } else {  // many, as where scores repeat: by the digits of their keys
    uint32_t key = 0, mask = 0;
#pragma unroll 1
    for (int p = 1; p <= 4; ++p) {
      const int shift = 32 - 8 * p;
      each([&](int, const float (&x)[4], int n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t k = order_key(x[c]);
          if (c < n && (k & mask) == key && part_of(x[c]) == part) atomicAdd(&sh.hist[p][(k >> shift) & 255], 1u);
        }
      });
      find(sh.hist[p]);
      key |= sh.found[0] << shift;
      mask |= 255u << shift;
    }
    edge = of_order_key(key);
    uint32_t above = 0, equal = 0;
    each([&](int, const float (&x)[4], int n) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) {
          above += x[c] > edge;
          equal += x[c] == edge;
        }
    });
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    equal = __reduce_add_sync(0xFFFFFFFFu, equal);
    if (lane == 0) {
      sh.above[warp] = above;
      sh.equal[warp] = equal;
    }
    __syncthreads();
  }

  // ---------------- the list, in order
  uint32_t above = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.above[lane] : 0u);  // in earlier warps' pieces
  uint32_t equal = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.equal[lane] : 0u);
  const uint32_t below = (1u << lane) - 1;
  if (whole) {
    uint32_t at = above + equal;
    each([&](int i, const float (&x)[4], int n) {
      uint32_t before = at;
      bool in[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        in[c] = c < n && x[c] >= edge;
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, in[c]);
        before += __popc(all & below);
        at += __popc(all);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (in[c]) out[before] = i + c;
        before += in[c];
      }
    });
  } else {
    each([&](int i, const float (&x)[4], int n) {
      // this lane's two counts in one word, then those of the lanes before it
      uint32_t mine = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) mine += x[c] > edge ? 0x10000u : (x[c] == edge ? 1u : 0u);
      if (!__any_sync(0xFFFFFFFFu, mine)) return;
      uint32_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t all = __shfl_sync(0xFFFFFFFFu, sum, 31);
      uint32_t a2 = above + ((sum - mine) >> 16), e2 = equal + ((sum - mine) & 0xFFFFu);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) {
          const bool gt = x[c] > edge, eq = x[c] == edge;
          if (gt || (eq && e2 < want)) out[a2 + min(e2, want)] = i + c;
          a2 += gt;
          e2 += eq;
        }
      above += all >> 16;
      equal += all & 0xFFFFu;
    });
  }
  if (a.status && tid == 0) a.status[unit] = (int32_t)sh.err;
}

__global__ void __launch_bounds__(kMaxListThreads, 1) list_pages_kernel(const SelectArgs a) {
  __shared__ ListShared sh;
  const int64_t unit = blockIdx.x;
  int bits;
  const int npages = pages_of(a, (int)(unit / a.Hkv), &bits);
  if (npages <= a.K) {
    grid_dependency_wait();
    list_all(a, unit, npages, bits);
    return;
  }
  list_unit(a, sh, unit, npages, a.scores + unit * a.stride, a.extents + unit * a.chunks,
            (npages + a.chunk - 1) / a.chunk, bits, [] { grid_dependency_wait(); });  // the scores are visible
}

// ------------------------------------------------------- both stages at once
__global__ void __launch_bounds__(kScoreWarps * 32, 2) select_pages_kernel(const SelectArgs a) {
  __shared__ ListShared sh;
  __shared__ ScoreShared ssh;
  __shared__ __align__(16) float scores[kFusedPages];
  __shared__ Extent extents[kMaxCluster * kScoreWarps];
  const int nc = (int)tc::cluster_nctarank(), rank = (int)tc::cluster_ctarank();
  const int64_t unit = blockIdx.x / nc, b = unit / a.Hkv;
  int bits;
  const int npages = pages_of(a, (int)b, &bits);
  if (npages <= a.K) {  // the whole cluster takes this path
    if (rank == 0) list_all(a, unit, npages, bits);
    return;
  }
  // even chunks, a multiple of what a warp takes at once
  const int per = (npages + nc * kScoreWarps - 1) / (nc * kScoreWarps);
  const int chunk = (per + kStep - 1) / kStep * kStep;
  cluster_arrive();  // this CTA is running: its shared memory may be written
  // the first CTA's arrays, as this CTA sees them
  score_block(a, ssh, b, (int)(unit % a.Hkv), rank * kScoreWarps * chunk, chunk, map_to_first(scores),
              map_to_first(extents), [] { cluster_wait(); });
  cluster_arrive();
  if (rank != 0) {
    cluster_wait();
    return;
  }
  list_unit(a, sh, unit, npages, scores, extents, (npages + chunk - 1) / chunk, bits, [] { cluster_wait(); });
}

// CTAs per list if scores and list are done in one launch, 0 if by two kernels.  One
// launch while all its CTAs are resident at once, two to an SM, and the pages are few:
// no more than 64 for a warp.  Device us (and of a call from Python) by size of the
// cluster, and by two kernels:
//   lists x pages      8            4            2            1            two
//     8 x 2048     7.8 (10.7)   9.2 (11.6)  11.8 (14.6)  17.3 (19.2)   8.3 (23.0)
//    32 x 1024     7.9 (10.6)   7.5 (10.2)   8.7 (10.8)  11.4 (14.2)  10.8 (21.2)
//    64 x 512     13.5 (16.7)   7.8 (10.4)   7.5 (10.6)   8.7 (11.0)  10.4 (22.7)
//    64 x 2048    17.1 (20.4)  12.2 (14.6)  15.3 (18.4)  24.7 (26.8)  12.6 (21.3)
//   128 x 1024    24.4 (27.1)  16.2 (18.8)  11.6 (14.6)  14.8 (16.9)  12.9 (21.3)
//   256 x 512     41.4 (43.8)  25.2 (27.1)  16.7 (18.8)  11.8 (14.6)  12.4 (20.5)
//   256 x 2048    54.8 (57.7)  42.9 (45.6)  36.2 (39.2)  30.4 (33.1)  31.0 (34.2)
//   512 x 512     78.6 (81.6)  45.3 (47.6)  32.4 (35.1)  23.5 (26.1)  19.0 (22.5)
// 8 lists of 8192 pages take 17.1 us in one launch of eight and 11.8 in two.
int one_launch(int64_t units, int max_pages, int sms) {
  int c = kMaxCluster;
  while (c > 1 && units * c > 2 * (int64_t)sms) c /= 2;
  const bool fits = units * c <= 2 * (int64_t)sms && max_pages <= min(kFusedPages, c * kScoreWarps * 64);
  return fits ? c : 0;
}

// Pages per warp of the first kernel: about 32 warps on every SM if all lists were
// as long as the table, at least the step that a warp takes at once, at most 64:
// lists shorter than the table then still spread (64 requests of up to 2K pages, 32
// to 256 pages a warp: 21.5, 20.5, 23.7, 31.9 us; 8 of 4K-16K pages: 38.6, 37.9, 36.7,
// 41.6; 8 of 64K pages: 216.8, 209.2, 205.6, 208.1).  Three CTAs per SM instead of four:
// 23.2, 40.1 and 220.0 us with 64.  Bounds through the ordinary cache policy instead of
// streaming ones: 21.9, 42.9 and 258.5.
int pages_per_warp(int64_t pairs, int sms) {
  const int64_t even = pairs / ((int64_t)sms * 32);
  int c = kStep;
  while (c < 64 && c < even) c *= 2;
  return c;
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
size_t scores_bytes(int64_t units, int64_t stride) { return align_up((size_t)units * (size_t)stride * 4); }
int64_t stride_of(int max_pages) { return ((int64_t)max_pages + 63) / 64 * 64; }

}  // namespace
}  // namespace pfkv

extern "C" size_t pfkv_select_pages_workspace_size(int batch, int num_kv_heads, int max_pages_per_seq) {
  if (batch < 0 || num_kv_heads <= 0 || max_pages_per_seq <= 0) return 0;
  const int64_t units = (int64_t)batch * num_kv_heads;
  if (pfkv::one_launch(units, max_pages_per_seq, pfkv::device_sm_count()) > 0) return 0;
  const int64_t chunks = ((int64_t)max_pages_per_seq + pfkv::kStep - 1) / pfkv::kStep;
  return pfkv::scores_bytes(units, pfkv::stride_of(max_pages_per_seq)) +
         pfkv::align_up((size_t)units * (size_t)chunks * sizeof(pfkv::Extent)) + 256;
}

extern "C" int pfkv_select_pages(int32_t* selected, const void* q, const int8_t* bounds, const float* bound_scales,
                                 const float* k_scales, const int32_t* block_tables, int max_pages_per_seq,
                                 const int32_t* context_lens, int batch, int num_q_heads, int num_kv_heads,
                                 int head_dim, int page_size, int64_t num_pages, int top_pages, int sink_pages,
                                 int recent_pages, void* workspace, size_t workspace_bytes, int32_t* unit_status,
                                 pfkv_stream_t stream) {
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
  if (G > kMaxG) return fail(PFKV_ERR_UNSUPPORTED, "select_pages: group size %d > 16", G);
  if (head_dim != kD) return fail(PFKV_ERR_UNSUPPORTED, "select_pages: head_dim %d != 128", head_dim);
  if ((int64_t)max_pages_per_seq * page_size >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "select_pages: block table too long");
  if (num_pages > (((int64_t)1 << 31) - 1) / num_kv_heads)
    return fail(PFKV_ERR_UNSUPPORTED, "select_pages: 2^31 or more (page, KV head) pairs");
  const int64_t units = (int64_t)batch * num_kv_heads;
  if (units > 0x7FFFFFFF) return fail(PFKV_ERR_UNSUPPORTED, "select_pages: batch too large");
  if (batch == 0) return PFKV_OK;
  const size_t need = pfkv_select_pages_workspace_size(batch, num_kv_heads, max_pages_per_seq);
  if (!selected || !q || !bounds || !bound_scales || !block_tables || !context_lens || (need > 0 && !workspace))
    return fail(PFKV_ERR_INVALID_ARG, "select_pages: null pointer");
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(selected, 4) || !aligned(bound_scales, 4) ||
      (k_scales && !aligned(k_scales, 4)) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(workspace, 256) || (unit_status && !aligned(unit_status, 4)))
    return fail(PFKV_ERR_INVALID_ARG, "select_pages: misaligned pointer");
  if (workspace_bytes < need)
    return fail(PFKV_ERR_WORKSPACE, "select_pages: workspace of %zu bytes is too small", workspace_bytes);
  SelectArgs a;
  a.selected = selected;
  a.status = unit_status;
  a.stride = stride_of(max_pages_per_seq);
  a.scores = static_cast<float*>(workspace);
  a.extents = reinterpret_cast<Extent*>(static_cast<uint8_t*>(workspace) + scores_bytes(units, a.stride));
  a.q = static_cast<const uint16_t*>(q);
  a.bounds = bounds;
  a.bound_scales = bound_scales;
  a.k_scales = k_scales;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.B = batch;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.G = G;
  a.P = page_size;
  a.max_pages = max_pages_per_seq;
  a.K = top_pages;
  a.sink = sink_pages;
  a.recent = recent_pages;
  a.num_pages = num_pages;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int sms = device_sm_count();
  if (sms <= 0) {
    const int rc = check_cuda("select_pages device query");
    return rc != PFKV_OK ? rc : fail(PFKV_ERR_CUDA, "select_pages: no device");
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (const int c = one_launch(units, max_pages_per_seq, sms); c > 0) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(units * c));
    cfg.blockDim = dim3(kScoreWarps * 32);
    (void)cudaLaunchKernelEx(&cfg, select_pages_kernel, a);
    return check_cuda("select_pages launch");
  }
  a.chunk = pages_per_warp(units * max_pages_per_seq, sms);
  a.chunks = (max_pages_per_seq + a.chunk - 1) / a.chunk;
  a.runs = (a.chunks + kScoreWarps - 1) / kScoreWarps;
  const int64_t blocks = units * a.runs;
  if (blocks > 0x7FFFFFFF) return fail(PFKV_ERR_UNSUPPORTED, "select_pages: too many pages");
  score_pages_kernel<<<(unsigned)blocks, kScoreWarps * 32, 0, s>>>(a);
  // the listing kernel is launched as a programmatic dependent: its CTAs wait
  // (griddepcontrol.wait) for the scores.  A list's threads: as many as its pages
  // keep busy, and as leave every list resident twice over (whole calls with 256 / 512
  // / 1024: 512 lists of 2K pages 70.5 / 72.9 / 81.7 us, 256 of 1K 21.8 / 21.1 / 25.4, 64 of
  // 16K 94.7 / 79.2 / 73.0)
  int threads = kBins;
  while (threads < kMaxListThreads && threads * 4 < max_pages_per_seq && units * 4 * threads <= (int64_t)sms * 2048)
    threads *= 2;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)units);
  cfg.blockDim = dim3((unsigned)threads);
  if (cudaLaunchKernelEx(&cfg, list_pages_kernel, a) != cudaSuccess) return check_cuda("select_pages launch");
  return check_cuda("select_pages launch");
}
