// sparse_decode.cu -- one decode step's attention over a list of pages per
// (request, KV head) of the paged e4m3 cache.
//
// For request b, KV head h and its list of logical pages, with T the tokens
// t < L_b of the listed pages:
//   s_t = softmax_scale * sum_d q[d] * val(K_t[d]) * ks(t),
//   out = sum_{t in T} e^{s_t - m} val(V_t) vs(t) / sum_{t in T} e^{s_t - m},
// with the scales of the tensor, the KV head, or the page.
//
// One cluster of up to 8 CTAs per (request, KV head), four warps a CTA (eight where
// there are few lists).  Each warp takes a contiguous run of the list's 16-token
// tiles: its lanes look up 32 pages at a time (list, block table, scales: one chain
// of loads for all of them), and a ring of TMA stages of its own keeps its K and V
// tiles in flight.
// The warps' states (m, l, o) stay in shared memory and are joined by log-sum-exp
// through distributed shared memory, so the whole step is one launch without
// scratch in global memory.  Long lists are bounded by HBM; short ones by the
// chain list -> block table -> first tile -> join, so everything that does not
// depend on the length is loaded before it is known, and the first copies are
// under way before the scales are.
// Device time: 8 lists of 64 pages x 64 tokens (8.4 MB) 8.2 us; 512 lists of up to 128
// pages x 16 tokens (203 MB) 37.1 us, 5.5 TB/s; 64 lists of 256 pages x 64 tokens (268 MB)
// 46.4 us, 5.8 TB/s, each with about 5 us of launch and ramp.  Finding the next tile
// before the scores instead of after P.V, the states joined per CTA before they
// cross the cluster, and f16 score products took these from 13.0, 41.4 and 52.2 us.
#include <cuda_bf16.h>
#include <math.h>

#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"
#include "pfkv_tc.cuh"
#include "pfkv_tile.cuh"

namespace pfkv {
namespace {

constexpr int kD = 128;
constexpr int kTile = tile::kTokens;
constexpr int kStages = 3;
constexpr int kBatches = 4;  // that tiles in the ring and the one being multiplied can be of, at least
static_assert(kBatches > kStages && (kBatches & (kBatches - 1)) == 0, "");
constexpr int kMaxCluster = 8;
constexpr int kStageBytes = 2 * tile::kSlabBytes;       // K, then V
constexpr int kWarpBytes = kStages * kStageBytes;       // also holds the warp's final state
constexpr int smem_bytes(int warps) { return warps * kWarpBytes + 1024; }  // + alignment slack
constexpr int kMaxG = 16;
constexpr int kStateFloats = kD + 4;  // of a head: o, m, l; whole 16-byte pieces
static_assert(kMaxG * kStateFloats * 4 <= kWarpBytes, "a warp's state fits its ring");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A head's references (pfkv_tile.cuh) are only raised when a token exceeds one by
// more than this (log2 units), so p and p vs stay at most 2^8 units: exact enough in
// f16 and f32.
constexpr float kRescaleLog2 = 8.f;

struct SparseArgs {
  uint16_t* out;
  const uint16_t* q;
  const float* k_scales;
  const float* v_scales;
  const int32_t* selected;  // [B][Hkv][K], or null: all pages in order
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* lse;
  int32_t* status;       // [B][Hkv] or null
  int32_t* status_word;  // one for the call, zeroed before, or null
  int Hq, Hkv, G, P, max_pages, K;
  int64_t num_pages;
  int page_stride, head_stride;  // scale index = page * page_stride + head * head_stride
  float logit_scale;             // softmax_scale * log2(e)
};

template <int NT, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, (NT == 1 ? 16 : 8) / kWarps)
    sparse_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const SparseArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int meta[kWarps][kStages];          // of the stage's tile: tokens << 8 | its page's place in scales
  __shared__ float2 scales[kWarps][kBatches * 32];  // K scale, log2 of the V scale: the last batches of pages looked up
  __shared__ uint32_t err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int nc = (int)tc::cluster_nctarank(), rank = (int)tc::cluster_ctarank();
  const int64_t unit = blockIdx.x / nc;
  const int b = (int)(unit / a.Hkv), h = (int)(unit % a.Hkv);
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t wbase = smem_base + warp * kWarpBytes;
  uint8_t* const wptr = smem_raw + (smem_base - smem_u32(smem_raw)) + warp * kWarpBytes;
  const uint32_t bar0 = smem_u32(&bars[warp][0]);
  const int32_t* const list = a.selected ? a.selected + unit * a.K : nullptr;
  const int tpp = a.P / kTile;  // tiles per page
  const int nw = nc * kWarps, gw = rank * kWarps + warp;
  // what does not depend on the length: the warp's first entries if the list is
  // as long as it may be, and the queries
  const int guess = (int)((uint32_t)gw * (uint32_t)(a.K * tpp) / nw / tpp);  // a list has fewer than 2^26 tiles, nw <= 64
  const int guessed = list ? __ldg(list + min(guess + lane, a.K - 1)) : guess + lane;
  uint4 qrow[NT][4];
  tile::load_q<NT>(a.q + ((int64_t)b * a.Hq + (int64_t)h * a.G) * kD, a.G, lane, qrow);

  if (threadIdx.x == 0) err = 0;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  __syncthreads();

  uint32_t bits = 0;
  int L = a.context_lens[b];
  const int cap = a.max_pages * a.P;
  if (L < 0 || L > cap) {
    bits |= kErrBadContext;
    L = L < 0 ? 0 : cap;
  }
  const int npages = (L + a.P - 1) / a.P;
  // The first npages entries, which hold every page of a list without gaps, are
  // split evenly over the warps; then those behind them, padding but for lists
  // with gaps (find() below).  All entries split alike would leave most warps of a
  // short context without work.
  const uint32_t F = (uint32_t)(min(a.K, npages) * tpp);
  bool behind = list && a.K > npages;
  int f_end = (int)((gw + 1) * F / nw);
  int f = (int)(gw * F / nw);  // next tile to issue
  int slot = f / tpp, sub = f - slot * tpp;

  // ---------------- pages of list entries slot0 .. slot0 + 31, one per lane
  int slot0 = 0, place = 0, page = 0, tokens = 0;  // place: of the batch in scales
  float ks = 0.f, vs = 0.f;
  auto find_page = [&](int s0) {
    slot0 = s0;
    tokens = 0;
    const int slot = s0 + lane;
    if (slot * tpp >= f_end) return;
    const int logical = s0 == guess ? guessed : (list ? __ldg(list + slot) : slot);
    if (logical < 0) return;  // padding
    if (logical >= npages) {
      bits |= kErrBadTopk;
      return;
    }
    page = __ldg(a.block_tables + (int64_t)b * a.max_pages + logical);
    if (page < 0 || (int64_t)page >= a.num_pages) {
      bits |= kErrBadPage;
      if (list) return;  // a list passes it over
      page = -1;         // dense decode reads zeros: boxes outside the tensor, zero scales
    }
    const int64_t si = (int64_t)page * a.page_stride + h * a.head_stride;
    ks = page >= 0 ? __ldg(a.k_scales + si) : 0.f;
    vs = page >= 0 ? __ldg(a.v_scales + si) : 0.f;
    tokens = min(a.P, L - logical * a.P);
  };
  auto look_up = [&](int s0) {
    find_page(s0);
    // a batch with tokens gets the next place; the last kStages of those stay
    if (__any_sync(0xFFFFFFFFu, tokens > 0)) place = (place + 32) % (kBatches * 32);
  };
  auto keep_scales = [&]() { scales[warp][place + lane] = make_float2(ks, __log2f(vs)); };
  if (f < f_end) look_up(slot);

  // ---------------- producer: find() the next tile with tokens, then issue() its
  // copies; apart, because a stage is free only at the end of an iteration
  const uint64_t kv_policy = l2_evict_first_policy();
  int issued = 0, next_row = 0, next_note = 0;  // next_note 0: there is no tile
  // the warp's entries behind the first npages, from about the first that is no padding
  auto go_behind = [&]() {
    behind = false;
    const uint32_t rest = (uint32_t)(a.K - npages);
    const int end = npages + (int)((gw + 1) * rest / nw);
    int e = npages + (int)(gw * rest / nw);
    for (; e < end; e += 128) {
      bool any = false;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = e + 32 * u + lane;
        any |= i < end && __ldg(list + i) >= 0;
      }
      if (__any_sync(0xFFFFFFFFu, any)) break;
    }
    slot = e;
    slot0 = e - 32;  // to be looked up
    sub = 0;
    f = e * tpp;
    f_end = end * tpp;
  };
  auto find = [&]() {
    next_note = 0;
    while (true) {
      if (f >= f_end) {
        if (!behind) return;
        go_behind();
        continue;
      }
      if (slot - slot0 >= 32) {
        keep_scales();  // the first batch's are still in registers only
        look_up(slot);
        keep_scales();
      }
      const int src = slot - slot0;
      const int valid = min(kTile, __shfl_sync(0xFFFFFFFFu, tokens, src) - sub * kTile);
      const int pg = __shfl_sync(0xFFFFFFFFu, page, src);
      if (valid <= 0) {  // nothing (more) in this page
        f += tpp - sub;
        ++slot;
        sub = 0;
        continue;
      }
      next_row = (pg * a.Hkv + h) * a.P + sub * kTile;  // the cache has fewer than 2^31 rows
      next_note = valid << 8 | (place + src);
      ++f;
      if (++sub == tpp) {
        sub = 0;
        ++slot;
      }
      return;
    }
  };
  auto issue = [&](int stage) {
    if (next_note == 0) return;
    if (lane == 0) {
      meta[warp][stage] = next_note;
      const uint32_t bar = bar0 + 8 * stage, dst = wbase + stage * kStageBytes;
      mbar_arrive_expect_tx(bar, kStageBytes);
      tma_load_2d_hint(dst, &tmK, 0, next_row, bar, kv_policy);
      tma_load_2d_hint(dst + tile::kSlabBytes, &tmV, 0, next_row, bar, kv_policy);
    }
    ++issued;
  };
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) {
    find();
    issue(s);
  }
  keep_scales();
  __syncwarp();

  // ---------------- consumer
  uint32_t qf[NT][8][2];
  float qinv[NT][2], mref[NT][2], cref[NT][2], l[NT][2], o[NT][8][4];
  tile::scale_q<NT>(qrow, lane, qf, qinv);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    mref[j][0] = mref[j][1] = -INFINITY;
    cref[j][0] = cref[j][1] = tile::kNoUnit;
    l[j][0] = l[j][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
  }
  const float sc = a.logit_scale;
  int stage = 0, done = 0;
  uint32_t phase = 0;
  bool timed_out = false;
  while (done < issued) {
    if (!mbar_wait(bar0 + 8 * stage, phase)) {
      timed_out = true;
      break;
    }
    const int mt = meta[warp][stage], n = mt >> 8;
    const float2 scale = scales[warp][mt & 255];
    const uint8_t* kb = wptr + stage * kStageBytes;
    find();
    float s[NT][4];
    tile::scores<NT>(kb, lane, qf, s);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float f0 = qinv[j][0] * scale.x, f1 = qinv[j][1] * scale.x;
      s[j][0] *= f0;
      s[j][1] *= f1;
      s[j][2] *= f0;
      s[j][3] *= f1;
      if (n < kTile) {
        if (g >= n) s[j][0] = s[j][1] = -INFINITY;
        if (g + 8 >= n) s[j][2] = s[j][3] = -INFINITY;
      }
    }
    tile::raise_references<NT>(s, sc, scale.y, kRescaleLog2, mref, cref, l, o);
    uint32_t pb[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float p0 = fast_exp2(fmaf(s[j][0], sc, -mref[j][0])), p1 = fast_exp2(fmaf(s[j][1], sc, -mref[j][1]));
      const float p2 = fast_exp2(fmaf(s[j][2], sc, -mref[j][0])), p3 = fast_exp2(fmaf(s[j][3], sc, -mref[j][1]));
      l[j][0] += p0 + p2;
      l[j][1] += p1 + p3;
      const float d0 = scale.y - cref[j][0], d1 = scale.y - cref[j][1];
      pb[j][0] = movmatrix_trans(pack_f16x2(fast_exp2(fmaf(s[j][0], sc, d0)), fast_exp2(fmaf(s[j][1], sc, d1))));
      pb[j][1] = movmatrix_trans(pack_f16x2(fast_exp2(fmaf(s[j][2], sc, d0)), fast_exp2(fmaf(s[j][3], sc, d1))));
    }
    tile::accumulate<NT>(kb + tile::kSlabBytes, lane, n, pb, o);
    // every load of the stage has returned (its values are in use): it can be
    // filled again
    __syncwarp();
    issue(stage);
    ++done;
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (timed_out) {
    bits |= kErrWaitTimeout;
    for (; done < issued; ++done) {  // copies in flight land before the ring is used again
      (void)mbar_wait(bar0 + 8 * stage, phase);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  bits = __reduce_or_sync(0xFFFFFFFFu, bits);
  if (lane == 0 && bits) atomicOr(&err, bits);

  // ---------------- the warp's state into its ring: o [G][128], then (m, l) [G]
  __syncwarp();
  float* const st = reinterpret_cast<float*>(wptr);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l[j][e];
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
      const int head = 8 * j + 2 * t + e;
      if (head < a.G) {
        float4* d = reinterpret_cast<float4*>(st + head * kD + 16 * g);
        const float unit = tile::unit(mref[j][e], cref[j][e]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          d[k] = make_float4(o[j][2 * k][e] * unit, o[j][2 * k][2 + e] * unit, o[j][2 * k + 1][e] * unit,
                             o[j][2 * k + 1][2 + e] * unit);
        if (g == 0) {
          st[a.G * kD + 2 * head] = mref[j][e];
          st[a.G * kD + 2 * head + 1] = v;
        }
      }
    }

  // ---------------- join: the CTA's states of a head into the first warp's place,
  // then the CTAs' by the CTA rank == head mod nc; a warp per head
  __syncthreads();
  for (int head = warp; head < a.G; head += kWarps) {
    float m[kWarps], M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* from = reinterpret_cast<const float*>(wptr - warp * kWarpBytes);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      m[k] = from[k * (kWarpBytes / 4) + a.G * kD + 2 * head];
      M = fmaxf(M, m[k]);
    }
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float* st = from + k * (kWarpBytes / 4);
      const float w = m[k] == -INFINITY ? 0.f : fast_exp2(m[k] - M);
      const float4 v = reinterpret_cast<const float4*>(st + head * kD)[lane];
      den = fmaf(w, st[a.G * kD + 2 * head + 1], den);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
    __syncwarp();
    float* to = reinterpret_cast<float*>(wptr - warp * kWarpBytes);
    reinterpret_cast<float4*>(to + head * kD)[lane] = acc;
    if (lane == 0) {
      to[a.G * kD + 2 * head] = M;
      to[a.G * kD + 2 * head + 1] = den;
    }
  }
  __syncwarp();
  tc::cluster_sync();
  for (int head = rank + nc * warp; head < a.G; head += nc * kWarps) {
    const uint32_t ml = smem_base + (a.G * kD + 2 * head) * 4, o4 = smem_base + (head * kD + 4 * lane) * 4;
    float m = -INFINITY, l1 = 0.f;
    if (lane < nc) {
      m = tc::ld_cluster_f32(tc::mapa(ml, lane));
      l1 = tc::ld_cluster_f32(tc::mapa(ml + 4, lane));
    }
    float4 v[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      v[k] = k < nc ? tc::ld_cluster_f32x4(tc::mapa(o4, k)) : make_float4(0.f, 0.f, 0.f, 0.f);
    float M = m;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
    const float w = m == -INFINITY ? 0.f : fast_exp2(m - M);
    float den = w * l1;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, off);
    M = __shfl_sync(0xFFFFFFFFu, M, 0);
    den = __shfl_sync(0xFFFFFFFFu, den, 0);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
      acc.x = fmaf(wk, v[k].x, acc.x);
      acc.y = fmaf(wk, v[k].y, acc.y);
      acc.z = fmaf(wk, v[k].z, acc.z);
      acc.w = fmaf(wk, v[k].w, acc.w);
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;  // nothing attended: zeros
    const int64_t row = (int64_t)b * a.Hq + (int64_t)h * a.G + head;
    reinterpret_cast<uint2*>(a.out + row * kD)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (a.lse && lane == 0) a.lse[row] = den > 0.f ? (M + __log2f(den)) * kLn2 : -INFINITY;
  }
  if (a.status && rank == 0 && threadIdx.x == 0) {
    uint32_t all = 0;
    for (int r = 0; r < nc; ++r) all |= tc::ld_cluster_u32(tc::mapa(smem_u32(&err), r));
    a.status[unit] = (int32_t)all;
  }
  if (a.status_word && threadIdx.x == 0 && err) atomicOr(a.status_word, (int32_t)err);
  __syncwarp();
  tc::cluster_sync();  // no CTA leaves while another may still read its shared memory
}

// CTAs per (request, KV head).  Few lists are spread as far as a cluster goes;
// otherwise two thirds of the CTAs that fit are asked for (`resident` per SM), so
// that the SMs which get one more than others still finish with them, but two per
// list where that many fit at all.  128-page lists of 64-token pages, 8 KV heads,
// 8 / 16 / 32 requests: 26.6 / 46.5 / 94.8 us with these 6 / 3 / 2 CTAs of four
// warps, 28.1 / 51.9 / 99.6 with 8, 30.4 / 49.7 / 90.3 with 4, 47.5 / 55.3 / 94.8 with 2.
int cluster_size(int64_t units, int64_t tiles, int warps, int resident, int sms) {
  const int64_t fit = (int64_t)resident * sms;
  int64_t c = 2 * fit / (3 * units);
  if (c < 2 && 2 * units <= fit) c = 2;
  if (c * warps > tiles) c = tiles / warps;  // a tile for every warp
  return (int)(c < 1 ? 1 : c > kMaxCluster ? kMaxCluster : c);
}

template <int NT, int kWarps>
int launch(const CUtensorMap& tmK, const CUtensorMap& tmV, const SparseArgs& a, int64_t units, cudaStream_t stream) {
  auto kern = sparse_decode_kernel<NT, kWarps>;
  static std::atomic<uint64_t> smem_set{0};
  const int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem_bytes(kWarps), smem_set,
                                      "paged_sparse_decode set smem attribute");
  if (rc != PFKV_OK) return rc;
  const int c = cluster_size(units, (int64_t)a.K * (a.P / kTile), kWarps, (NT == 1 ? 16 : 8) / kWarps, device_sm_count());
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * c));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem_bytes(kWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, tmK, tmV, a) != cudaSuccess) return check_cuda("paged_sparse_decode launch");
  return check_cuda("paged_sparse_decode launch");
}

int launch_for(const SparseArgs& a, const void* k_cache, const void* v_cache, int64_t units, cudaStream_t stream) {
  const cuuint64_t dims[2] = {kD, (cuuint64_t)a.num_pages * a.Hkv * a.P};
  const cuuint64_t strides[1] = {kD};
  const cuuint32_t box[2] = {kD, (cuuint32_t)kTile};
  CUtensorMap tmK, tmV;
  int rc = encode_tensor_map(&tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(k_cache), dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc == PFKV_OK)
    rc = encode_tensor_map(&tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(v_cache), dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != PFKV_OK) return rc;
  // lists of up to a quarter of the SMs' number: eight warps a CTA (1 / 2 / 4 requests
  // of the lists above 11.4 / 15.3 / 16.8 us instead of 15.4 / 17.7 / 18.2 with four, 8
  // requests 27.3 instead of 26.6)
  const bool wide = units * 4 <= device_sm_count();
  if (a.G <= 8) return wide ? launch<1, 8>(tmK, tmV, a, units, stream) : launch<1, 4>(tmK, tmV, a, units, stream);
  return wide ? launch<2, 8>(tmK, tmV, a, units, stream) : launch<2, 4>(tmK, tmV, a, units, stream);
}

}  // namespace

int decode_short_blocks(void* out, const void* q, const void* k_cache, const void* v_cache, const float* k_scales,
                        const float* v_scales, const int32_t* block_tables, int max_pages_per_seq,
                        const int32_t* context_lens, int batch, int num_q_heads, int num_kv_heads, int page_size,
                        int64_t num_pages, float softmax_scale, int32_t* status_word, float* lse_out,
                        cudaStream_t stream) {
  if (cudaMemsetAsync(status_word, 0, sizeof(int32_t), stream) != cudaSuccess)
    return check_cuda("paged_decode status reset");
  SparseArgs a;
  a.out = static_cast<uint16_t*>(out);
  a.q = static_cast<const uint16_t*>(q);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.selected = nullptr;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.lse = lse_out;
  a.status = nullptr;
  a.status_word = status_word;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.G = num_q_heads / num_kv_heads;
  a.P = page_size;
  a.max_pages = max_pages_per_seq;
  a.K = max_pages_per_seq;
  a.num_pages = num_pages;
  a.page_stride = num_kv_heads;
  a.head_stride = 1;
  a.logit_scale = softmax_scale * kLog2e;
  return launch_for(a, k_cache, v_cache, (int64_t)batch * num_kv_heads, stream);
}

}  // namespace pfkv

extern "C" int pfkv_paged_sparse_decode_attn(void* out, const void* q, const void* k_cache, const void* v_cache,
                                             pfkv_scale_granularity granularity, const float* k_scales,
                                             const float* v_scales, const int32_t* selected, int top_pages,
                                             const int32_t* block_tables, int max_pages_per_seq,
                                             const int32_t* context_lens, int batch, int num_q_heads,
                                             int num_kv_heads, int head_dim, int page_size, int64_t num_pages,
                                             float softmax_scale, float* lse_out, int32_t* unit_status,
                                             pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || num_pages <= 0 ||
      max_pages_per_seq <= 0 || top_pages <= 0)
    return fail(PFKV_ERR_INVALID_ARG, "paged_sparse_decode: bad sizes");
  if (num_q_heads % num_kv_heads != 0)
    return fail(PFKV_ERR_INVALID_ARG, "paged_sparse_decode: num_q_heads %% num_kv_heads != 0");
  const int G = num_q_heads / num_kv_heads;
  if (G > kMaxG) return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: group size %d > 16", G);
  if (head_dim != kD) return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: head_dim %d != 128", head_dim);
  if (page_size % kTile != 0)
    return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: page_size %d not a multiple of 16", page_size);
  int page_stride = 0, head_stride = 0;
  switch (granularity) {
    case PFKV_SCALE_TENSOR: break;
    case PFKV_SCALE_HEAD: head_stride = 1; break;
    case PFKV_SCALE_BLOCK:
      page_stride = num_kv_heads;
      head_stride = 1;
      break;
    case PFKV_SCALE_TOKEN:
      return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: scales per token are not supported");
    default:
      return fail(PFKV_ERR_INVALID_ARG, "paged_sparse_decode: unknown granularity %d", (int)granularity);
  }
  if ((int64_t)num_pages * num_kv_heads * page_size >= (int64_t)1 << 31)
    return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: cache has 2^31 or more token rows");
  if ((int64_t)max_pages_per_seq * page_size >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: block table too long");
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale))
    return fail(PFKV_ERR_INVALID_ARG, "paged_sparse_decode: softmax_scale must be finite and > 0");
  if ((int64_t)top_pages * page_size >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: list too long");
  const int64_t units = (int64_t)batch * num_kv_heads;
  if (units > 0x7FFFFFFF / kMaxCluster) return fail(PFKV_ERR_UNSUPPORTED, "paged_sparse_decode: batch too large");
  if (batch == 0) return PFKV_OK;
  if (!out || !q || !k_cache || !v_cache || !k_scales || !v_scales || !selected || !block_tables || !context_lens)
    return fail(PFKV_ERR_INVALID_ARG, "paged_sparse_decode: null pointer");
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(selected, 4) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || (lse_out && !aligned(lse_out, 4)) || (unit_status && !aligned(unit_status, 4)))
    return fail(PFKV_ERR_INVALID_ARG, "paged_sparse_decode: misaligned pointer");
  SparseArgs a;
  a.out = static_cast<uint16_t*>(out);
  a.q = static_cast<const uint16_t*>(q);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.selected = selected;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.lse = lse_out;
  a.status = unit_status;
  a.status_word = nullptr;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.G = G;
  a.P = page_size;
  a.max_pages = max_pages_per_seq;
  a.K = top_pages;
  a.num_pages = num_pages;
  a.page_stride = page_stride;
  a.head_stride = head_stride;
  a.logit_scale = softmax_scale * kLog2e;
  return launch_for(a, k_cache, v_cache, units, reinterpret_cast<cudaStream_t>(stream));
}
