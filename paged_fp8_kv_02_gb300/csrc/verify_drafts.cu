// verify_drafts.cu -- which drafted tokens stay after a verification pass, and
// the token that follows them.
//
// One cluster of CTAs per request.  Every CTA finds the first rejected draft (a
// lane per draft: token -> two probabilities -> ballot), then the cluster reads
// that row of the target's and the draft's probabilities once, as 64-bit whole
// weights, whose sum is the same in any order: each warp sums its part of the
// vocabulary and keeps the sum of every block of it (what its lanes have in
// flight at a time), the CTAs exchange their sums through distributed shared
// memory, and the CTA that holds the threshold reads one block again to find the
// token.
//
// 64 requests with up to seven drafts, 128,259 words in fp32 (62 MB): 13.7 us on the
// device; 96 with up to five looked-up drafts, 152,064 words in bf16 (29 MB): 11.6; one
// of 32,768 words: 4.8.  What bounds them: launch, the chain lengths -> token ->
// probability in front of the row and the exchange (a request alone has little else),
// then a warp's blocks one after the other, a trip to memory each (one request: 4.8
// us at 32,768 words, a block a warp, 6.3 at 128,259, four), and HBM last.  Word by
// word and with conversions to 64-bit integers these took 25.0, 65.5 and 6.0 us;
// reading a warp's whole part again for the token 14.1, 13.3 and 4.5.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"
#include "pfkv_tc.cuh"

namespace pfkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kVectors = 4;  // 16-byte loads of a lane in flight, of each of the two rows
constexpr int kWords = 16;   // single words, where the rows cannot be read in 16 bytes alike
constexpr int kMaxVocab = 1 << 20;

struct VerifyArgs {
  int32_t* next;
  int32_t* accepted;
  const void* target;
  const void* draft;
  int64_t target_stride, draft_stride;
  const int32_t* tokens;
  const float* uniforms;
  const int32_t* q_start;
  int32_t* context_lens;
  int32_t* status;
  int T, V;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// floor(2^42 min(max(x, 0), 1)); 0 for NaN.
__device__ __forceinline__ uint64_t whole(float x) { return (uint64_t)(__saturatef(x) * 4398046511104.f); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores a 64-bit word at the same place of another CTA of the cluster.
__device__ __forceinline__ void store_in_cta(uint64_t* p, int rank, uint64_t v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// The probabilities of one row of a request and what is taken off them: the
// draft's row (q), or one at a drafted token (token >= 0), or nothing.
template <class T>
struct Row {
  const T* p;
  const T* q;
  int token, V;
  __device__ __forceinline__ uint64_t at(int i) const {
    float x = to_float(p[i]);
    if (q) x -= to_float(q[i]);
    if (i == token) x -= 1.f;
    return whole(x);
  }
  // with the drafted token's word as it is
  __device__ __forceinline__ uint64_t whole_at(int i) const {
    float x = to_float(p[i]);
    if (q) x -= to_float(q[i]);
    return whole(x);
  }
};

// The words of one load, as fp32.
template <class T, int kSize>
struct Load;
template <class T>
struct Load<T, 1> {
  T x;
  __device__ __forceinline__ void from(const T* p) { x = *p; }
  __device__ __forceinline__ void zero() { x = T(0.f); }
  __device__ __forceinline__ float at(int) const { return to_float(x); }
};
template <>
struct Load<float, 4> {
  float4 x;
  __device__ __forceinline__ void from(const float* p) { x = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void zero() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float at(int e) const { return e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w; }
};
struct Load16 {
  uint4 x;
  __device__ __forceinline__ void zero() { x = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t pair(int e) const { return e < 2 ? x.x : e < 4 ? x.y : e < 6 ? x.z : x.w; }
};
template <>
struct Load<__nv_bfloat16, 8> : Load16 {
  __device__ __forceinline__ void from(const __nv_bfloat16* p) { x = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ float at(int e) const { return e & 1 ? bf16_hi(pair(e)) : bf16_lo(pair(e)); }
};
template <>
struct Load<__half, 8> : Load16 {
  __device__ __forceinline__ void from(const __half* p) { x = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ float at(int e) const { return e & 1 ? f16_hi(pair(e)) : f16_lo(pair(e)); }
};

// Words of a block: what the lanes of a warp read at a time.
template <class T>
__host__ __device__ constexpr int block_words(bool wide) {
  return 32 * (wide ? 16 / (int)sizeof(T) * kVectors : kWords);
}
constexpr int kMaxBlocks = kMaxVocab / kWarps / 512 + 1;  // of a warp; 512 is the smallest block

// Sums a warp's part of the row's weights, block by block, into sums[]; returns
// the part's sum.  Places count from `shift` words before the row, where the 16
// bytes begin that hold its first word; a part begins at a multiple of a block.
// Words of 16 bytes that reach beyond the row are read one by one.
// A weight is split in two halves of 21 bits without a conversion (one to 64-bit
// integers takes longer than the loads): x + 4 rounded towards zero holds floor(2^21
// x) in its lowest bits, and the rest, which is exact, plus 2^-19 likewise the next
// 21; the bits are summed as integers and the constants' taken off.  A lane has at
// most 32 words of a block: its sums stay below 2^27, the warp's below 2^32.
template <class T, int kSize, bool kMinus>
__device__ __forceinline__ uint64_t sum_part(const Row<T>& row, int shift, int begin, int end, int lane, uint64_t* sums) {
  constexpr int kDeep = kSize == 1 ? kWords : kVectors;
  constexpr int kBlock = 32 * kSize * kDeep;
  static_assert(kDeep * kSize <= 32 && kBlock >= 512, "see above");
  uint64_t total = 0;
  const int stop = min(end - shift, row.V - kSize + 1);
  for (int at = begin; at < end; at += kBlock) {
    const int i0 = at - shift + lane * kSize;
    Load<T, kSize> p[kDeep], q[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int i = i0 + 32 * kSize * k;
      if (i >= 0 && i < stop) {
        p[k].from(row.p + i);
        if (kMinus) q[k].from(row.q + i);
      } else {
        p[k].zero();
        if (kMinus) q[k].zero();
      }
    }
    uint32_t high = 0, low = 0;
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
#pragma unroll
      for (int e = 0; e < kSize; ++e) {
        const float x = __saturatef(kMinus ? p[k].at(e) - q[k].at(e) : p[k].at(e));
        const float u = __fadd_rz(x, 4.f);
        const float v = __fadd_rz(x - (u - 4.f), 1.9073486328125e-6f);  // 2^-19
        high += __float_as_uint(u);
        low += __float_as_uint(v);
      }
    constexpr uint32_t n = kDeep * kSize;
    high = __reduce_add_sync(0xFFFFFFFFu, high - n * 0x40800000u);
    low = __reduce_add_sync(0xFFFFFFFFu, low - n * 0x36000000u);
    const uint64_t sum = ((uint64_t)high << 21) + low;
    if (lane == 0) sums[(at - begin) / kBlock] = sum;
    total += sum;
  }
  // what is counted apart: the words beside the vectors at the row's ends, and a
  // drafted token's loss
  auto add = [&](int place, uint64_t more) {
    more = warp_sum(more);
    if (lane == 0) sums[(place - begin) / kBlock] += more;
    total += more;
  };
  if (kSize > 1) {
    const int head = shift ? min(kSize - shift, row.V) : 0;
    const int tail = max(head, (shift + row.V) / kSize * kSize - shift);
    if (begin == 0 && head > 0) add(0, lane < head ? row.whole_at(lane) : 0);
    if (tail < row.V && tail + shift >= begin && tail + shift < end)
      add(tail + shift, tail + lane < row.V ? row.whole_at(tail + lane) : 0);
  }
  const int at = row.token + shift;
  if (row.token >= 0 && at >= begin && at < end) add(at, lane == 0 ? row.at(row.token) - row.whole_at(row.token) : 0);
  return total;
}

template <class T>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_drafts_kernel(const VerifyArgs a) {
  __shared__ uint64_t totals[2][kMaxCluster];  // of each CTA, by pass
  __shared__ uint64_t sums[kWarps][kMaxBlocks];  // of each warp's blocks
  __shared__ uint64_t parts[kWarps], scan[kWarps];
  __shared__ int found[3];  // drafts that stay, whether a token outside ended them, the token behind them
  const int nc = (int)tc::cluster_nctarank(), rank = (int)tc::cluster_ctarank();
  const int b = blockIdx.x / nc;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
  const int n = s1 - s0;
  if (s0 < 0 || s1 <= s0 || s1 > a.T) {  // the whole cluster leaves
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[b] = 0;
      if (a.status) a.status[b] = s1 == s0 && s0 >= 0 && s1 <= a.T ? 0 : PFKV_REQ_BAD_INDEX;
    }
    return;
  }
  cluster_arrive();  // this CTA is running: its shared memory may be written
  const float u = a.uniforms[s1 - 1];
  const T* const target = static_cast<const T*>(a.target);
  const T* const draft = static_cast<const T*>(a.draft);
  if (warp == 0) {
    int kept = n - 1, bad = 0, token = -1;
    for (int j0 = 0; j0 < n - 1; j0 += 32) {
      const int64_t i = s0 + j0 + lane;
      bool rejects = false;
      int x = 0;
      if (j0 + lane < n - 1) {
        x = a.tokens[i + 1];
        const float chance = a.uniforms[i];
        rejects = true;
        if (x >= 0 && x < a.V) {
          const double p = to_float(target[i * a.target_stride + x]);
          const double q = draft ? to_float(draft[i * a.draft_stride + x]) : 1.f;
          rejects = !((double)chance * q < p);
        }
      }
      const unsigned r = __ballot_sync(0xFFFFFFFFu, rejects);
      if (r) {
        const int first = __ffs(r) - 1;
        kept = j0 + first;
        token = __shfl_sync(0xFFFFFFFFu, x, first);
        bad = token < 0 || token >= a.V;
        break;
      }
    }
    if (lane == 0) found[0] = kept, found[1] = bad, found[2] = bad ? -1 : token;
  }
  __syncthreads();
  const int kept = found[0];
  const bool rejected = kept < n - 1;
  const int64_t r = s0 + kept;
  Row<T> row;
  row.V = a.V;
  row.p = target + r * a.target_stride;
  row.q = draft && rejected ? draft + r * a.draft_stride : nullptr;
  row.token = draft ? -1 : found[2];
  int shift, places, block, part;
  uint64_t total = 0, before = 0;
  for (int pass = 0;; ++pass) {
    // where the two rows stand alike within 16 bytes they are read 16 bytes at a time,
    // else word by word (64 requests of 128,259 words: 13.5 us either way in fp32, 10.9
    // and 12.8 in bf16)
    const int p_at = (int)(reinterpret_cast<uintptr_t>(row.p) & 15), q_at = (int)(reinterpret_cast<uintptr_t>(row.q) & 15);
    const bool wide = !row.q || p_at == q_at;
    shift = wide ? p_at / (int)sizeof(T) : 0;
    places = shift + a.V, block = block_words<T>(wide);
    part = (places + nc * kWarps * block - 1) / (nc * kWarps * block) * block;
    const int begin = min((rank * kWarps + warp) * part, places), end = min(begin + part, places);
    constexpr int kSize = 16 / sizeof(T);
    uint64_t mine;
    if (!row.q)
      mine = sum_part<T, kSize, false>(row, shift, begin, end, lane, sums[warp]);
    else if (wide)
      mine = sum_part<T, kSize, true>(row, shift, begin, end, lane, sums[warp]);
    else
      mine = sum_part<T, 1, true>(row, shift, begin, end, lane, sums[warp]);
    if (lane == 0) parts[warp] = mine;
    __syncthreads();
    uint64_t all = 0;
    if (warp == 0) all = warp_sum(lane < kWarps ? parts[lane] : 0);
    if (pass == 0) cluster_wait();
    if (warp == 0 && lane < nc) store_in_cta(&totals[pass][rank], lane, all);
    cluster_arrive();
    cluster_wait();
    total = before = 0;
    for (int k = 0; k < nc; ++k) {
      if (k < rank) before += totals[pass][k];
      total += totals[pass][k];
    }
    if (total != 0 || pass == 1) break;
    row.q = nullptr;  // nothing is left: the target's own weights
    row.token = -1;
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (i != kept) a.next[s0 + i] = i < kept ? a.tokens[s0 + i + 1] : -1;
    if (threadIdx.x == 0) {
      a.accepted[b] = kept;
      if (total == 0) a.next[r] = -1;
      if (a.status) a.status[b] = (found[1] ? PFKV_REQ_BAD_TOKEN : 0) | (total == 0 ? PFKV_REQ_NO_MASS : 0);
      if (a.context_lens) a.context_lens[b] -= n - 1 - kept;
    }
  }
  if (total == 0) return;
  // floor(total * U / 2^24), total < 2^62
  const uint32_t U = (uint32_t)(fminf(fmaxf(u, 0.f), 0.99999994f) * 16777216.f);
  const uint64_t bar = (__umul64hi(total, U) << 40) | ((total * U) >> 24);
  uint64_t own = 0;
  for (int k = 0; k < kWarps; ++k) own += parts[k];
  if (bar < before || bar - before >= own) return;  // another CTA's
  uint64_t rest = bar - before;
  int holder = 0;
  while (rest >= parts[holder]) rest -= parts[holder++];
  // the block, by every warp for itself: 32 of them at a time
  const int first = (rank * kWarps + holder) * part;
  const int blocks = (min(first + part, places) - first + block - 1) / block;
  int at = 0;
  for (int k0 = 0;; k0 += 32) {
    uint64_t upto = k0 + lane < blocks ? sums[holder][k0 + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned beyond = __ballot_sync(0xFFFFFFFFu, upto > rest);
    if (beyond || k0 + 32 >= blocks) {
      const int hit = beyond ? __ffs(beyond) - 1 : 0;
      const uint64_t under = __shfl_sync(0xFFFFFFFFu, upto, hit > 0 ? hit - 1 : 0);
      if (hit > 0) rest -= under;
      at = k0 + hit;
      break;
    }
    rest -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  // this CTA reads the block again, a run of words per thread
  constexpr int kRun = block_words<T>(true) / kThreads > block_words<T>(false) / kThreads ? block_words<T>(true) / kThreads
                                                                                         : block_words<T>(false) / kThreads;
  const int run = block / kThreads;
  const int i0 = first + at * block - shift + (int)threadIdx.x * run;
  uint64_t w[kRun], mine = 0;
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int i = i0 + k;
    w[k] = k < run && i >= 0 && i < a.V ? row.at(i) : 0;
    mine += w[k];
  }
  uint64_t upto = mine;  // inclusive prefix over the CTA
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  for (int k = 0; k < warp; ++k) upto += scan[k];
  if (rest < upto && rest >= upto - mine) {
    uint64_t left = rest - (upto - mine);
    int hit = 0;
    bool past = true;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      past = past && left >= w[k];
      if (past) left -= w[k], hit = k + 1;
    }
    a.next[r] = i0 + hit;
  }
}

template <class T>
int launch(const VerifyArgs& a, int batch, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)batch * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  (void)cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T>, a);
  return check_cuda("verify_drafts launch");
}

}  // namespace
}  // namespace pfkv

extern "C" int pfkv_verify_drafts(int32_t* next_tokens, int32_t* accepted, const void* target_probs,
                                  int64_t target_stride, const void* draft_probs, int64_t draft_stride,
                                  pfkv_prob_dtype prob_dtype, const int32_t* tokens, const float* uniforms,
                                  const int32_t* q_start, int batch, int num_tokens, int vocab_size,
                                  int32_t* context_lens, int32_t* request_status, pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  if (batch < 0 || num_tokens < 0 || vocab_size <= 0) return fail(PFKV_ERR_INVALID_ARG, "verify_drafts: bad sizes");
  if (prob_dtype != PFKV_PROB_F32 && prob_dtype != PFKV_PROB_BF16 && prob_dtype != PFKV_PROB_F16)
    return fail(PFKV_ERR_INVALID_ARG, "verify_drafts: unknown type %d of probabilities", (int)prob_dtype);
  if (vocab_size > kMaxVocab) return fail(PFKV_ERR_UNSUPPORTED, "verify_drafts: vocabulary of %d words, at most 2^20", vocab_size);
  if (batch > 1 << 24) return fail(PFKV_ERR_UNSUPPORTED, "verify_drafts: too many requests");
  if (batch == 0) return PFKV_OK;
  if (!accepted || !q_start || (num_tokens > 0 && (!next_tokens || !target_probs || !tokens || !uniforms)))
    return fail(PFKV_ERR_INVALID_ARG, "verify_drafts: null pointer");
  const uintptr_t unit = prob_dtype == PFKV_PROB_F32 ? 4 : 2;
  if (!aligned(accepted, 4) || !aligned(q_start, 4) || !aligned(next_tokens, 4) || !aligned(target_probs, unit) ||
      !aligned(draft_probs, unit) || !aligned(tokens, 4) || !aligned(uniforms, 4) || !aligned(context_lens, 4) ||
      !aligned(request_status, 4))
    return fail(PFKV_ERR_INVALID_ARG, "verify_drafts: misaligned pointer");
  const int64_t most = ((int64_t)1 << 40);
  if (target_stride < vocab_size || target_stride > most || (draft_probs && (draft_stride < vocab_size || draft_stride > most)))
    return fail(PFKV_ERR_INVALID_ARG, "verify_drafts: rows are at least vocab_size elements apart");
  const int sms = device_sm_count();
  if (sms <= 0) return fail(PFKV_ERR_CUDA, "verify_drafts: no device");
  // what is written has a place of its own: rows are shifted and lengths taken off by
  // several CTAs, without an order between them
  const struct {
    const void* at;
    uint64_t bytes;
  } flat[] = {{next_tokens, 4ull * num_tokens}, {accepted, 4ull * batch},    {context_lens, 4ull * batch}, {request_status, 4ull * batch},
              {tokens, 4ull * num_tokens},      {uniforms, 4ull * num_tokens}, {q_start, 4ull * batch + 4}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 7; ++j)
      if (arrays_meet(flat[i].at, flat[i].bytes, flat[j].at, flat[j].bytes))
        return fail(PFKV_ERR_INVALID_ARG, "verify_drafts: an array that is written overlaps another one");
  // Powers of two up to what is resident at once, four CTAs per SM, while a CTA is left
  // with more than 2048 words.  us with clusters of 1, 2, 4 and 8 on 152 SMs: 20
  // requests of 20,000 words 7.1 6.0 5.7 5.3 (taken: 8), 64 of 128,259 32 20.0 14.7
  // 13.8 (8), 96 of 152,064 (bf16, looked up) 19.9 14.9 12.0 17.2 (4), 150 of 32,768
  // 12.5 10.0 11.7 14.3 (4), 200 of 50,000 18.3 15.2 19.0 21.2 (2)
  int cluster = kMaxCluster;
  while (cluster > 1 && (int64_t)batch * cluster > 4 * sms) cluster /= 2;
  while (cluster > 1 && vocab_size <= 4096 * (cluster / 2)) cluster /= 2;
  VerifyArgs a;
  a.next = next_tokens;
  a.accepted = accepted;
  a.target = target_probs;
  a.draft = draft_probs;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.tokens = tokens;
  a.uniforms = uniforms;
  a.q_start = q_start;
  a.context_lens = context_lens;
  a.status = request_status;
  a.T = num_tokens;
  a.V = vocab_size;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (prob_dtype) {
    case PFKV_PROB_F32: return launch<float>(a, batch, cluster, s);
    case PFKV_PROB_BF16: return launch<__nv_bfloat16>(a, batch, cluster, s);
    default: return launch<__half>(a, batch, cluster, s);
  }
}
