// rotary.cu -- rotary positions with several axes: bf16 rows turned by their
// token's positions, alone or on the way into the paged e4m3 cache.
//
// Pair i turns by phi = position[axis_i] * f_i.  f_i / (2 pi) is kept as a
// 64-bit fraction of a turn: position * turns_i mod 2^64 is the angle's exact
// fraction of a turn for every 32-bit position, two integer multiplications in
// place of a range reduction in double precision, of which this GPU has little.
// Sine and cosine of that fraction come from a table and a short polynomial.
//
// Prompts are bounded by HBM (16,001 tokens, 64/8 heads of 128, scales per token, 624
// MB: 105 us on the device, 5.9 TB/s, 88% of a plain copy's rate; 2,039 latent tokens
// of 128 heads of 576, 605 MB: 101 us; 4,099 tokens of 48 query heads, 101 MB: 18.0
// us).  A step of 64 tokens takes 3.6 us, queries alone 2.7: the launch and the chain
// position -> angle -> turn -> store.  What the shape below gained: 168, 130, 23.3
// and 3.9 us with a piece's place worked out for every row, the angles before the
// first load and two CTAs per SM.
#include <cuda_bf16.h>
#include <math.h>

#include "pfkv_internal.h"
#include "pfkv_ptx.cuh"

namespace pfkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens a CTA takes at most
// Query rows of a thread that are in flight together, and CTAs of an SM (64 registers
// at four; rows of 128 with scales per token then spill one).  Prompt of 16,001 and
// 4,099 tokens, us, with an earlier form of the angles (sincospif): 2 rows at 4 CTAs
// 105.3 and 17.4, 3 at 4 104.5 and 18.2, 4 at 3 104.0 and 19.8, 4 at 4 111.0 and
// 20.2, 2 at 5 111.1 and 20.3.
constexpr int kBatch = 2;
constexpr int kBlocks = 4;

struct RotaryArgs {
  const uint16_t* x[3];  // q, k, v
  int64_t stride[3];     // elements between tokens
  uint16_t* q_out;
  int64_t q_out_stride;
  uint8_t* cache[2];       // [pages][Hkv][P][D]
  const float* scale[2];   // read: per tensor (scale_step 0) or per head (1)
  float* tscale[2];        // written: [pages][Hkv][P]
  const int64_t* slots;
  const int32_t* positions;  // [axes][T]
  int64_t num_slots;
  int T, Hq, Hkv, D, P, rows, scale_step, rows_per_cta, pitch, in_place;
  pfkv_rotary r;
};

// cos and sin of i / 128 of a turn, each as the nearest fp32 number and the rest.
__device__ const float4 kQuarter[32] = {
    {1.f, 0.f, 0.f, 0.f}, {0.99879545f, 6.47143805e-09f, 0.0490676761f, -1.73993431e-09f},
    {0.99518472f, 7.10966619e-09f, 0.0980171412f, -8.93393193e-10f}, {0.989176512f, -1.79974535e-09f, 0.146730468f, 6.77824552e-09f},
    {0.980785251f, 2.97394731e-08f, 0.195090324f, -1.67047143e-09f}, {0.970031261f, -8.24954771e-09f, 0.242980182f, -2.2676041e-09f},
    {0.956940353f, -1.7184508e-08f, 0.290284663f, 1.38156651e-08f}, {0.941544056f, 9.24430044e-09f, 0.336889863f, -9.62200097e-09f},
    {0.923879504f, 2.83074897e-08f, 0.382683426f, 6.22335072e-09f}, {0.903989315f, -2.1909516e-08f, 0.427555084f, 9.20176646e-09f},
    {0.881921291f, -2.70029634e-08f, 0.471396744f, -7.42525375e-09f}, {0.857728601f, 9.49825818e-09f, 0.514102757f, -1.27838593e-08f},
    {0.831469595f, 1.68702634e-08f, 0.555570245f, -1.17695214e-08f}, {0.803207517f, 1.48104178e-08f, 0.59569931f, -5.81030113e-09f},
    {0.773010433f, 2.06425526e-08f, 0.634393275f, 9.37955758e-09f}, {0.740951121f, 4.50153514e-09f, 0.671558976f, -2.13263824e-08f},
    {0.707106769f, 1.21016175e-08f, 0.707106769f, 1.21016175e-08f}, {0.671558976f, -2.13263824e-08f, 0.740951121f, 4.50153514e-09f},
    {0.634393275f, 9.37955758e-09f, 0.773010433f, 2.06425526e-08f}, {0.59569931f, -5.81030113e-09f, 0.803207517f, 1.48104178e-08f},
    {0.555570245f, -1.17695214e-08f, 0.831469595f, 1.68702634e-08f}, {0.514102757f, -1.27838593e-08f, 0.857728601f, 9.49825818e-09f},
    {0.471396744f, -7.42525375e-09f, 0.881921291f, -2.70029634e-08f}, {0.427555084f, 9.20176646e-09f, 0.903989315f, -2.1909516e-08f},
    {0.382683426f, 6.22335072e-09f, 0.923879504f, 2.83074897e-08f}, {0.336889863f, -9.62200097e-09f, 0.941544056f, 9.24430044e-09f},
    {0.290284663f, 1.38156651e-08f, 0.956940353f, -1.7184508e-08f}, {0.242980182f, -2.2676041e-09f, 0.970031261f, -8.24954771e-09f},
    {0.195090324f, -1.67047143e-09f, 0.980785251f, 2.97394731e-08f}, {0.146730468f, 6.77824552e-09f, 0.989176512f, -1.79974535e-09f},
    {0.0980171412f, -8.93393193e-10f, 0.99518472f, 7.10966619e-09f}, {0.0490676761f, -1.73993431e-09f, 0.99879545f, 6.47143805e-09f},
};

// Cosine and sine of phase / 2^64 turns: the nearest 1/128 of a turn from the table,
// which the warp's lanes hold (`entry` is this lane's), and a rest of at most 0.0246
// rad, for which three terms do (method of P. T. P. Tang, "Table-lookup algorithms for
// elementary functions and their error analysis", 1991).  By whole warps.
// Off by at most 0.65 2^-24: the last sum's rounding 0.5 (of results below 1); the
// rest's three roundings 0.074, times a table entry of at most 1; the roundings of
// sin r and of the sum before the last 0.025 each; r^5 / 120 and the rest's cut to
// 2^-39 of a turn below 0.002.  0.56 at worst of 4M angles computed so on the host.
__device__ __forceinline__ void cos_sin(uint64_t phase, const float4& entry, float* cosine, float* sine) {
  const uint32_t near = (uint32_t)((phase + (1ull << 56)) >> 57);  // of 128
  const float r = (float)(int32_t)((int64_t)(phase - ((uint64_t)near << 57)) >> 25) * 1.14290478e-11f;  // 2 pi 2^-39
  const int lane = near & 31;
  const float ch = __shfl_sync(0xFFFFFFFFu, entry.x, lane), cl = __shfl_sync(0xFFFFFFFFu, entry.y, lane);
  const float sh = __shfl_sync(0xFFFFFFFFu, entry.z, lane), sl = __shfl_sync(0xFFFFFFFFu, entry.w, lane);
  const float r2 = r * r;
  const float sr = fmaf(r * r2, -0.16666667f, r);            // sin r
  const float cr = r2 * fmaf(r2, 0.041666668f, -0.5f);       // cos r - 1
  const float c = ch + fmaf(-sh, sr, fmaf(ch, cr, cl));
  const float s = sh + fmaf(ch, sr, fmaf(sh, cr, sl));
  const bool odd = near & 32;  // quarters of a turn
  const float a = odd ? s : c, b = odd ? c : s;
  *cosine = ((near + 32) & 64) ? -a : a;
  *sine = (near & 64) ? -b : b;
}

// A piece of a row: 8 channels and 8 more, either the two halves of 8 pairs or
// 16 consecutive channels.
struct Piece {
  int lo, hi;  // first channel of each part
  bool turns;
};

__device__ __forceinline__ Piece piece_of(const pfkv_rotary& r, int j) {
  Piece p;
  const int turning = r.num_pairs >> 3;
  p.turns = j < turning;
  if (p.turns && !r.neighbours) {
    p.lo = r.first + 8 * j;
    p.hi = p.lo + r.num_pairs;
  } else if (p.turns) {
    p.lo = r.first + 16 * j;
    p.hi = p.lo + 8;
  } else {  // the channels before the turning ones, then those behind
    p.lo = 16 * (j - turning);
    if (p.lo >= r.first) p.lo += 2 * r.num_pairs;
    p.hi = p.lo + 8;
  }
  return p;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint16_t a = f32x2_to_e4m3x2(__fdiv_rn(f[4 * k], s), __fdiv_rn(f[4 * k + 1], s));
    const uint16_t b = f32x2_to_e4m3x2(__fdiv_rn(f[4 * k + 2], s), __fdiv_rn(f[4 * k + 3], s));
    w[k] = (uint32_t)a | ((uint32_t)b << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Turns the 8 pairs of a piece: x, y are its two halves, or 16 neighbours.
__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8], bool neighbours) {
  if (!neighbours) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x[i], v = y[i];
      x[i] = u * c[i] - v * s[i];
      y[i] = v * c[i] + u * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u = x[2 * i], v = x[2 * i + 1];
      x[2 * i] = u * c[i] - v * s[i];
      x[2 * i + 1] = v * c[i] + u * s[i];
      u = y[2 * i], v = y[2 * i + 1];
      y[2 * i] = u * c[i + 4] - v * s[i + 4];
      y[2 * i + 1] = v * c[i + 4] + u * s[i + 4];
    }
  }
}

// A CTA takes `tokens` consecutive tokens (kThreads / tokens threads each) and
// rows_per_cta of their rows: query heads, then keys, then values.  A thread has
// the same piece of every row that it takes, so that its place in the row and its
// 8 sines and cosines are found once; a row's pieces lie in consecutive threads
// (for kToken in a power of two of them, so that its maximum is a few shuffles).
// The first rows are on their way while the angles are worked out.  kPitch:
// threads of a row where that is known beforehand, or 0.
template <int kPitch, bool kToken>
__global__ void __launch_bounds__(kThreads, kBlocks) rotary_kernel(const __grid_constant__ RotaryArgs a, const int tokens) {
  __shared__ __align__(16) float cosine[kMaxTokens][PFKV_ROTARY_MAX_PAIRS], sine[kMaxTokens][PFKV_ROTARY_MAX_PAIRS];
  const int per_token = kThreads / tokens;
  const int which_token = threadIdx.x / per_token, tid = threadIdx.x - which_token * per_token;
  const int t = blockIdx.x * tokens + which_token;
  const int pitch = kPitch ? kPitch : a.pitch;
  const int step = per_token / pitch;  // rows of a pass
  const int r0 = tid / pitch, j = tid - r0 * pitch;
  const bool live = t < a.T && r0 < step && j < (a.D >> 4);
  const Piece p = piece_of(a.r, j);
  const int row0 = blockIdx.y * a.rows_per_cta, row1 = min(a.rows, row0 + a.rows_per_cta);
  const int64_t slot = t < a.T && a.slots ? a.slots[t] : -1;
  int64_t pos = 0;
  if (t < a.T && tid < a.r.num_pairs) pos = a.positions[(int64_t)a.r.axis[tid] * a.T + t];

  // queries: the first rows
  const int q_end = live && (p.turns || !a.in_place) ? min(row1, a.Hq) : 0;
  const uint16_t* const q = a.x[0] + t * a.stride[0];
  uint4 lo[kBatch], hi[kBatch];
  int row = row0 + r0;
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    if (row + k * step < q_end) {
      const uint16_t* const src = q + (row + k * step) * a.D;
      lo[k] = __ldcs(reinterpret_cast<const uint4*>(src + p.lo));
      hi[k] = __ldcs(reinterpret_cast<const uint4*>(src + p.hi));
    }
  }
  if (t < a.T) {
    const float4 entry = __ldg(kQuarter + (threadIdx.x & 31));
    for (int i = tid; (i & ~31) < a.r.num_pairs; i += per_token) {  // whole warps
      const bool mine = i < a.r.num_pairs;
      if (mine && i != tid) pos = a.positions[(int64_t)a.r.axis[i] * a.T + t];
      float c, s;
      cos_sin((uint64_t)pos * (mine ? a.r.turns[i] : 0), entry, &c, &s);
      if (mine) {
        cosine[which_token][i] = c;
        sine[which_token][i] = s;
      }
    }
  }
  __syncthreads();
  if (t >= a.T) return;
  float c[8], s[8];
  if (p.turns) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(&cosine[which_token][8 * j + i]);
      const float4 v = *reinterpret_cast<const float4*>(&sine[which_token][8 * j + i]);
      c[i] = u.x, c[i + 1] = u.y, c[i + 2] = u.z, c[i + 3] = u.w;
      s[i] = v.x, s[i + 1] = v.y, s[i + 2] = v.z, s[i + 3] = v.w;
    }
  }
  uint16_t* const q_out = a.q_out + t * a.q_out_stride;
  while (row < q_end) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (row + k * step < q_end) {
        uint16_t* const dst = q_out + (row + k * step) * a.D;
        if (p.turns) {
          float x[8], y[8];
          unpack8(lo[k], x);
          unpack8(hi[k], y);
          turn(x, y, c, s, a.r.neighbours);
          lo[k] = pack8(x);
          hi[k] = pack8(y);
        }
        __stcs(reinterpret_cast<uint4*>(dst + p.lo), lo[k]);
        __stcs(reinterpret_cast<uint4*>(dst + p.hi), hi[k]);
      }
    }
    row += kBatch * step;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (row + k * step < q_end) {
        const uint16_t* const src = q + (row + k * step) * a.D;
        lo[k] = __ldcs(reinterpret_cast<const uint4*>(src + p.lo));
        hi[k] = __ldcs(reinterpret_cast<const uint4*>(src + p.hi));
      }
    }
  }
  if (slot < 0 || slot >= a.num_slots || row1 <= a.Hq) return;

  // keys, then values
  const int64_t page = slot <= 0x7FFFFFFF ? (uint32_t)slot / (uint32_t)a.P : slot / a.P;
  const int64_t slot_at = page * a.Hkv * a.P + (slot - page * a.P);  // of head 0
  const int kv_end = row1 - a.Hq;
  const int kv_from = max(row0 - a.Hq, 0);
  for (int first = kv_from; first < kv_end; first += step) {  // whole warps, for the shuffles
    const int r = first + r0;
    const bool mine = live && r < kv_end;
    const int which = r >= a.Hkv ? 1 : 0, h = r - (which ? a.Hkv : 0);
    const int lo_at = which ? 16 * j : p.lo, hi_at = which ? 16 * j + 8 : p.hi;
    float x[8], y[8];
    if (mine) {
      const uint16_t* const src = a.x[1 + which] + t * a.stride[1 + which] + h * a.D;
      unpack8(__ldcs(reinterpret_cast<const uint4*>(src + lo_at)), x);
      unpack8(__ldcs(reinterpret_cast<const uint4*>(src + hi_at)), y);
      if (!which && p.turns) turn(x, y, c, s, a.r.neighbours);
    }
    float scale, m = 0.f;
    const int64_t at = slot_at + (int64_t)h * a.P;
    if constexpr (kToken) {
      if (mine)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(y[i])));
      for (int o = pitch >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      scale = __fdiv_rn(m, 448.f);
      if (mine && j == 0) a.tscale[which][at] = scale;
    } else if (mine) {
      scale = __ldg(a.scale[which] + (int64_t)h * a.scale_step);
    }
    if (mine) {
      uint2 u = make_uint2(0, 0), v = u;
      if (!kToken || scale != 0.f) u = encode8(x, scale), v = encode8(y, scale);
      uint8_t* const dst = a.cache[which] + at * a.D;
      *reinterpret_cast<uint2*>(dst + lo_at) = u;
      *reinterpret_cast<uint2*>(dst + hi_at) = v;
    }
  }
}

int check_rotary(const char* fn, const pfkv_rotary* r, int D) {
  if (!r) return fail(PFKV_ERR_INVALID_ARG, "%s: null rotary", fn);
  if (r->num_pairs < 8 || r->num_pairs > PFKV_ROTARY_MAX_PAIRS || r->num_pairs % 8 || r->first < 0 || r->first % 16 ||
      r->num_axes < 1 || r->num_axes > PFKV_ROTARY_MAX_AXES)
    return fail(PFKV_ERR_INVALID_ARG, "%s: rotary not filled by rotary_init", fn);
  for (int i = 0; i < r->num_pairs; ++i)
    if (r->axis[i] >= r->num_axes) return fail(PFKV_ERR_INVALID_ARG, "%s: rotary not filled by rotary_init", fn);
  if ((int64_t)r->first + 2 * r->num_pairs > D)
    return fail(PFKV_ERR_INVALID_ARG, "%s: channels %d..%d turn, head_dim is %d", fn, r->first,
                r->first + 2 * r->num_pairs - 1, D);
  return PFKV_OK;
}

// Token stride of [T][H][D] rows.
bool good_stride(int64_t stride, int T, int H, int D) {
  return stride >= (int64_t)H * D && stride % 8 == 0 && stride <= 0x7FFFFFFF;
}

// Whether rows of `row` and `other_row` bytes, T of each `stride` and `other_stride`
// bytes apart, have bytes in common.  With one stride (parts of the same wider rows)
// each row lies at the same place of its wider row: exact.  With two: by extents.
bool rows_meet(const void* a, int64_t stride, int64_t row, const void* b, int64_t other_stride, int64_t other_row, int T) {
  uintptr_t lo = reinterpret_cast<uintptr_t>(a), hi = reinterpret_cast<uintptr_t>(b);
  if (hi < lo) return rows_meet(b, other_stride, other_row, a, stride, row, T);
  const uint64_t apart = hi - lo;
  if (apart >= (uint64_t)(T - 1) * stride + row) return false;
  if (T == 1 || stride != other_stride) return true;
  // the first row of b begins `in` bytes behind one of a's
  const uint64_t rows = apart / stride, in = apart % stride;
  return in < (uint64_t)row || (rows + 1 < (uint64_t)T && in + other_row > (uint64_t)stride);
}

int check_q(const char* fn, const void* out, int64_t out_stride, const void* x, int64_t x_stride, int T, int H, int D,
            int* in_place) {
  if (!out || !x) return fail(PFKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(out, 16) || !aligned(x, 16)) return fail(PFKV_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (!good_stride(out_stride, T, H, D) || !good_stride(x_stride, T, H, D))
    return fail(PFKV_ERR_INVALID_ARG, "%s: token strides are multiples of 8 of at least %lld and below 2^31", fn, (long long)H * D);
  *in_place = out == x && (out_stride == x_stride || T == 1);
  const int64_t row = (int64_t)H * D * 2;
  if (!*in_place && rows_meet(out, out_stride * 2, row, x, x_stride * 2, row, T))
    return fail(PFKV_ERR_INVALID_ARG, "%s: output and input overlap", fn);
  return PFKV_OK;
}

int launch(const char* fn, RotaryArgs& a, bool token, cudaStream_t stream) {
  const int pieces = a.D / 16;
  a.pitch = pieces;
  if (token)
    for (a.pitch = 1; a.pitch < pieces;) a.pitch *= 2;
  const int sms = device_sm_count();
  if (sms <= 0) return fail(PFKV_ERR_CUDA, "%s: no device", fn);
  // A step's tokens are a CTA each, more than one where there are fewer than SMs.
  // Two tokens a CTA from four an SM on, four from eight, where a row is no wider than
  // a quarter of a token's threads (36 pieces of a latent row leave 28 of 64 idle, 4
  // of 256).  us with 1, 2 and 4 of them on 152 SMs:
  //   append, 64/8 heads of 128: 500 tokens 5.4 5.8 7.8, 608 5.9 6.2 8.3, 700 8.8 7.1
  //   9.2, 1,216 10.9 8.9 11.4, 2,432 20.3 17.7 18.8, 8,000 60 53.5 55.6, 16,001 with
  //   scales per token 120.6 105.3 105.8 (8: 113, with an earlier form of the angles)
  //   queries alone, 48 heads: 608 4.1 4.5 4.7, 1,216 7.6 7.5 7.6, 2,432 13.0 12.6
  //   11.6, 4,099 19.5 19.0 18.0, 16,001 67.2 62.7 59.2
  // One rule serves both: the append alone would do with two (2.4 us less at 1,216
  // tokens, 4% at 8,000).
  int tokens = kMaxTokens;
  while (tokens > 1 && (a.T < 2 * sms * tokens || a.pitch * 4 > kThreads / tokens)) tokens /= 2;
  int parts = 1;
  if (tokens == 1)
    while (parts * 2 * kThreads < a.rows * a.pitch && (int64_t)a.T * parts < sms) parts *= 2;
  a.rows_per_cta = (a.rows + parts - 1) / parts;
  parts = (a.rows + a.rows_per_cta - 1) / a.rows_per_cta;
  const dim3 grid((unsigned)((a.T + (int64_t)tokens - 1) / tokens), (unsigned)parts);
  if (pieces == 8) {
    if (token)
      rotary_kernel<8, true><<<grid, kThreads, 0, stream>>>(a, tokens);
    else
      rotary_kernel<8, false><<<grid, kThreads, 0, stream>>>(a, tokens);
  } else {
    if (token)
      rotary_kernel<0, true><<<grid, kThreads, 0, stream>>>(a, tokens);
    else
      rotary_kernel<0, false><<<grid, kThreads, 0, stream>>>(a, tokens);
  }
  return check_cuda(fn);
}

}  // namespace
}  // namespace pfkv

extern "C" {

int pfkv_rotary_init(pfkv_rotary* rotary, const double* frequencies, const int32_t* axes, int num_pairs, int num_axes,
                     int first, int neighbours) {
  using namespace pfkv;
  clear_error();
  if (!rotary || !frequencies) return fail(PFKV_ERR_INVALID_ARG, "rotary_init: null pointer");
  if (num_pairs < 8 || num_pairs > PFKV_ROTARY_MAX_PAIRS || num_pairs % 8)
    return fail(PFKV_ERR_UNSUPPORTED, "rotary_init: %d pairs: a multiple of 8 up to %d", num_pairs, PFKV_ROTARY_MAX_PAIRS);
  if (num_axes < 1 || num_axes > PFKV_ROTARY_MAX_AXES)
    return fail(PFKV_ERR_UNSUPPORTED, "rotary_init: %d axes: 1 to %d", num_axes, PFKV_ROTARY_MAX_AXES);
  if (first < 0 || first % 16) return fail(PFKV_ERR_UNSUPPORTED, "rotary_init: first channel %d: a multiple of 16", first);
  for (int i = 0; i < num_pairs; ++i) {
    if (!isfinite(frequencies[i])) return fail(PFKV_ERR_INVALID_ARG, "rotary_init: frequency %d is not finite", i);
    if (axes && (axes[i] < 0 || axes[i] >= num_axes))
      return fail(PFKV_ERR_INVALID_ARG, "rotary_init: axis %d of pair %d outside [0, %d)", axes[i], i, num_axes);
  }
  *rotary = pfkv_rotary{};
  rotary->first = first;
  rotary->num_pairs = num_pairs;
  rotary->neighbours = neighbours ? 1 : 0;
  rotary->num_axes = num_axes;
  for (int i = 0; i < num_pairs; ++i) {
    // the fraction of a turn, of the magnitude: a negative frequency is its exact opposite
    const double turn = fabs(frequencies[i]) / 6.283185307179586476925;
    const double part = ldexp(turn - floor(turn), 64);
    const uint64_t whole = part >= 18446744073709551616.0 ? 0 : (uint64_t)part;
    rotary->turns[i] = frequencies[i] < 0 ? 0 - whole : whole;
    rotary->axis[i] = axes ? (uint8_t)axes[i] : 0;
  }
  return PFKV_OK;
}

int pfkv_rotary_embed(void* out, int64_t out_stride, const void* x, int64_t x_stride, const int32_t* positions,
                      const pfkv_rotary* rotary, int num_tokens, int num_heads, int head_dim, pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  const char* fn = "rotary_embed";
  if (num_tokens < 0 || num_heads <= 0 || head_dim <= 0) return fail(PFKV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (head_dim % 16 || head_dim > 4096)
    return fail(PFKV_ERR_UNSUPPORTED, "%s: head_dim %d: a multiple of 16 up to 4096", fn, head_dim);
  if ((int64_t)num_heads * head_dim >= (int64_t)1 << 30) return fail(PFKV_ERR_UNSUPPORTED, "%s: rows too wide", fn);
  if (int rc = check_rotary(fn, rotary, head_dim)) return rc;
  if (num_tokens == 0) return PFKV_OK;
  RotaryArgs a = {};
  if (int rc = check_q(fn, out, out_stride, x, x_stride, num_tokens, num_heads, head_dim, &a.in_place)) return rc;
  if (!positions || !aligned(positions, 4)) return fail(PFKV_ERR_INVALID_ARG, "%s: null or misaligned positions", fn);
  a.x[0] = static_cast<const uint16_t*>(x);
  a.stride[0] = x_stride;
  a.q_out = static_cast<uint16_t*>(out);
  a.q_out_stride = out_stride;
  a.positions = positions;
  a.T = num_tokens;
  a.Hq = a.rows = num_heads;
  a.D = head_dim;
  a.P = 1;
  a.r = *rotary;
  return launch(fn, a, false, reinterpret_cast<cudaStream_t>(stream));
}

int pfkv_rotary_append_fp8(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k_new,
                           int64_t k_stride, const void* v_new, int64_t v_stride, void* k_cache, void* v_cache,
                           const int64_t* slot_mapping, const int32_t* positions, const pfkv_rotary* rotary,
                           int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                           int64_t num_pages, pfkv_scale_granularity granularity, float* k_scales, float* v_scales,
                           pfkv_stream_t stream) {
  using namespace pfkv;
  clear_error();
  const char* fn = "rotary_append_fp8";
  const bool has_q = q_out || q, has_v = v_new || v_cache || v_scales;
  if (num_tokens < 0 || (has_q && num_q_heads <= 0) || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 ||
      num_pages <= 0)
    return fail(PFKV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (head_dim % 16 || head_dim > 4096)
    return fail(PFKV_ERR_UNSUPPORTED, "%s: head_dim %d: a multiple of 16 up to 4096", fn, head_dim);
  if (((int64_t)(has_q ? num_q_heads : 0) + 2 * (int64_t)num_kv_heads) * head_dim >= (int64_t)1 << 30)
    return fail(PFKV_ERR_UNSUPPORTED, "%s: rows too wide", fn);
  if (granularity == PFKV_SCALE_BLOCK)
    return fail(PFKV_ERR_INVALID_ARG, "%s: scales per block are written by kv_append_fp8_block after rotary_embed", fn);
  if (granularity != PFKV_SCALE_TENSOR && granularity != PFKV_SCALE_HEAD && granularity != PFKV_SCALE_TOKEN)
    return fail(PFKV_ERR_INVALID_ARG, "%s: unknown granularity %d", fn, (int)granularity);
  const bool token = granularity == PFKV_SCALE_TOKEN;
  if (token && head_dim > 512) return fail(PFKV_ERR_UNSUPPORTED, "%s: per-token scales need head_dim <= 512", fn);
  if (int rc = check_rotary(fn, rotary, head_dim)) return rc;
  if (num_pages > INT64_MAX / page_size / num_kv_heads / head_dim)
    return fail(PFKV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (num_tokens == 0) return PFKV_OK;
  RotaryArgs a = {};
  if (has_q)
    if (int rc = check_q(fn, q_out, q_out_stride, q, q_stride, num_tokens, num_q_heads, head_dim, &a.in_place)) return rc;
  if (!k_new || !k_cache || !k_scales || !slot_mapping || !positions)
    return fail(PFKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (has_v && (!v_new || !v_cache || !v_scales))
    return fail(PFKV_ERR_INVALID_ARG, "%s: v_new, v_cache and v_scales must all be set or all NULL", fn);
  if (!aligned(k_new, 16) || !aligned(k_cache, 16) || !aligned(k_scales, 4) || !aligned(slot_mapping, 8) ||
      !aligned(positions, 4) || (has_v && (!aligned(v_new, 16) || !aligned(v_cache, 16) || !aligned(v_scales, 4))))
    return fail(PFKV_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (!good_stride(k_stride, num_tokens, num_kv_heads, head_dim) ||
      (has_v && !good_stride(v_stride, num_tokens, num_kv_heads, head_dim)))
    return fail(PFKV_ERR_INVALID_ARG, "%s: token strides are multiples of 8 of at least %lld and below 2^31", fn,
                (long long)num_kv_heads * head_dim);
  const int64_t q_row = (int64_t)num_q_heads * head_dim * 2, kv_row = (int64_t)num_kv_heads * head_dim * 2;
  if (has_q && (rows_meet(q_out, q_out_stride * 2, q_row, k_new, k_stride * 2, kv_row, num_tokens) ||
                (has_v && rows_meet(q_out, q_out_stride * 2, q_row, v_new, v_stride * 2, kv_row, num_tokens))))
    return fail(PFKV_ERR_INVALID_ARG, "%s: q_out overlaps k_new or v_new", fn);
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k_new);
  a.x[2] = static_cast<const uint16_t*>(v_new);
  a.stride[0] = q_stride;
  a.stride[1] = k_stride;
  a.stride[2] = v_stride;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_out_stride = q_out_stride;
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(v_cache);
  a.scale[0] = a.tscale[0] = k_scales;
  a.scale[1] = a.tscale[1] = v_scales;
  a.scale_step = granularity == PFKV_SCALE_HEAD ? 1 : 0;
  a.slots = slot_mapping;
  a.positions = positions;
  a.num_slots = num_pages * page_size;
  a.T = num_tokens;
  a.Hq = has_q ? num_q_heads : 0;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.P = page_size;
  a.rows = a.Hq + num_kv_heads * (has_v ? 2 : 1);
  a.r = *rotary;
  return launch(fn, a, token, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
