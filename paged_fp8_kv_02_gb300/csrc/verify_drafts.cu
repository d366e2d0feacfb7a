// verify_drafts.cu -- which drafted tokens stay after a verification pass, and
// the token that follows them.
//
// One cluster of CTAs per request.  Every CTA finds the first rejected draft (a
// lane per draft: token -> two probabilities -> ballot), then the cluster reads
// that row of the target's and the draft's probabilities once, as 64-bit whole
// weights: their sum is the same in any order, so each warp sums a stretch of
// the vocabulary, the CTAs exchange their sums through distributed shared
// memory, and the warp whose stretch holds the threshold is read again (from L2)
// by its CTA to find the token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"
#include "pfkv_tc.cuh"

namespace pfkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 8;  // loads of a lane in flight, of each of the two rows

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
  int T, V, stretch;  // stretch: words of the vocabulary per warp
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// floor(2^42 min(max(x, 0), 1)); 0 for NaN.
__device__ __forceinline__ uint64_t whole(float x) {
  return (uint64_t)(fminf(fmaxf(x, 0.f), 1.f) * 4398046511104.f);
}

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

// How a row's weights are made: the target's probabilities less the draft's, or
// less one at a drafted token, or as they are.
enum Kind { kMinusDraft, kMinusToken, kPlain };

template <class T>
struct Row {
  const T* p;
  const T* q;
  int token;
  Kind kind;
  __device__ __forceinline__ uint64_t at(int i) const {
    float x = to_float(p[i]);
    if (kind == kMinusDraft) x -= to_float(q[i]);
    if (kind == kMinusToken && i == token) x -= 1.f;
    return whole(x);
  }
};

template <class T>
__device__ __forceinline__ uint64_t sum_stretch(const Row<T>& row, int begin, int end, int lane) {
  uint64_t sum = 0;
  for (int i0 = begin + lane; i0 < end; i0 += 32 * kUnroll) {
    float p[kUnroll], q[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + 32 * k;
      p[k] = q[k] = 0.f;
      if (i < end) {
        p[k] = to_float(row.p[i]);
        if (row.kind == kMinusDraft) q[k] = to_float(row.q[i]);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (row.kind == kMinusToken && i0 + 32 * k == row.token) q[k] = 1.f;
      sum += whole(p[k] - q[k]);
    }
  }
  return warp_sum(sum);
}

template <class T>
__global__ void __launch_bounds__(kThreads) verify_drafts_kernel(const VerifyArgs a) {
  __shared__ uint64_t totals[2][kMaxCluster];  // of each CTA, by pass
  __shared__ uint64_t sums[kWarps];
  __shared__ uint64_t scan[kWarps];
  __shared__ int found_s[2];
  const int nc = (int)tc::cluster_nctarank(), rank = (int)tc::cluster_ctarank();
  const int b = blockIdx.x / nc;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
  const int n = s1 - s0;
  if (s0 < 0 || s1 < s0 || s1 > a.T || n == 0) {  // the whole cluster leaves
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[b] = 0;
      if (a.status) a.status[b] = n == 0 && s0 >= 0 && s1 <= a.T ? 0 : PFKV_REQ_BAD_INDEX;
    }
    return;
  }
  cluster_arrive();  // this CTA is running: its shared memory may be written
  const T* const target = static_cast<const T*>(a.target);
  const T* const draft = static_cast<const T*>(a.draft);
  if (warp == 0) {
    int kept = n - 1, bad = 0;
    for (int j0 = 0; j0 < n - 1; j0 += 32) {
      const int i = s0 + j0 + lane;
      bool rejects = false, outside = false;
      if (j0 + lane < n - 1) {
        const int x = a.tokens[i + 1];
        const float u = a.uniforms[i];
        outside = x < 0 || x >= a.V;
        rejects = true;
        if (!outside) {
          const double p = to_float(target[i * a.target_stride + x]);
          const double q = draft ? to_float(draft[i * a.draft_stride + x]) : 1.f;
          rejects = !((double)u * q < p);
        }
      }
      const unsigned r = __ballot_sync(0xFFFFFFFFu, rejects);
      if (r) {
        const int first = __ffs(r) - 1;
        kept = j0 + first;
        bad = __shfl_sync(0xFFFFFFFFu, outside ? 1 : 0, first);
        break;
      }
    }
    if (lane == 0) found_s[0] = kept, found_s[1] = bad;
  }
  __syncthreads();
  const int kept = found_s[0], bad_token = found_s[1];
  const int64_t r = s0 + kept;
  Row<T> row;
  row.p = target + r * a.target_stride;
  row.q = draft ? draft + r * a.draft_stride : nullptr;
  row.token = -1;
  row.kind = kPlain;
  if (kept < n - 1) {
    row.kind = draft ? kMinusDraft : kMinusToken;
    row.token = a.tokens[r + 1];
  }
  const float u = a.uniforms[s1 - 1];
  const uint32_t U = (uint32_t)(fminf(fmaxf(u, 0.f), 0.99999994f) * 16777216.f);
  const int first = (rank * kWarps + warp) * a.stretch;
  const int begin = min(first, a.V), end = min(first + a.stretch, a.V);
  uint64_t total = 0, before = 0;
  for (int pass = 0;; ++pass) {
    const uint64_t mine = sum_stretch(row, begin, end, lane);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    uint64_t all = 0;
    if (warp == 0) all = warp_sum(lane < kWarps ? sums[lane] : 0);
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
    row.kind = kPlain;
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (i != kept) a.next[s0 + i] = i < kept ? a.tokens[s0 + i + 1] : -1;
    if (threadIdx.x == 0) {
      a.accepted[b] = kept;
      if (total == 0) a.next[r] = -1;
      if (a.status) a.status[b] = (bad_token ? PFKV_REQ_BAD_TOKEN : 0) | (total == 0 ? PFKV_REQ_NO_MASS : 0);
      if (a.context_lens) a.context_lens[b] -= n - 1 - kept;
    }
  }
  if (total == 0) return;
  // floor(total * U / 2^24), total < 2^62
  const uint64_t bar = (__umul64hi(total, U) << 40) | ((total * U) >> 24);
  uint64_t own = 0;
  for (int k = 0; k < kWarps; ++k) own += sums[k];
  if (bar < before || bar - before >= own) return;  // another CTA's
  uint64_t rest = bar - before;
  int holder = 0;
  while (rest >= sums[holder]) rest -= sums[holder++];
  // this CTA reads the holder's stretch again, a run of words per thread
  const int h0 = min((rank * kWarps + holder) * a.stretch, a.V), h1 = min(h0 + a.stretch, a.V);
  const int run = (h1 - h0 + kThreads - 1) / kThreads;
  const int i0 = min(h0 + (int)threadIdx.x * run, h1), i1 = min(i0 + run, h1);
  uint64_t part = 0;
  for (int i = i0; i < i1; ++i) part += row.at(i);
  uint64_t upto = part;  // inclusive prefix over the CTA
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  for (int k = 0; k < warp; ++k) upto += scan[k];
  if (rest < upto && rest >= upto - part) {
    uint64_t left = rest - (upto - part);
    for (int i = i0; i < i1; ++i) {
      const uint64_t w = row.at(i);
      if (left < w) {
        a.next[r] = i;
        break;
      }
      left -= w;
    }
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
  if (vocab_size > 1 << 20) return fail(PFKV_ERR_UNSUPPORTED, "verify_drafts: vocabulary of %d words, at most 2^20", vocab_size);
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
  int cluster = kMaxCluster;
  while (cluster > 1 && (int64_t)batch * cluster > 2 * sms) cluster /= 2;
  while (cluster > 1 && vocab_size < 4096 * cluster) cluster /= 2;
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
  a.stretch = ((vocab_size + cluster * kWarps - 1) / (cluster * kWarps) + 31) / 32 * 32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (prob_dtype) {
    case PFKV_PROB_F32: return launch<float>(a, batch, cluster, s);
    case PFKV_PROB_BF16: return launch<__nv_bfloat16>(a, batch, cluster, s);
    default: return launch<__half>(a, batch, cluster, s);
  }
}
