// Cross entropy of a linear output layer for sm_103a, with the gradients of the
// hidden states and the weight: the C ABI of include/linear_ce.h.
//
//   k_lce_scan         which tokens count, in order; how many
//   k_lce_gather       their hidden states side by side, in bf16; zeros for the others' gradients
//   k_lce_weight       the weight as the products read it, where it is not already
//   then for every piece of tokens
//   k_lce_logits       x = h W^T.  The ending reduces a row's 128 words to a power of two 2^I >= their
//                      largest exponential and s = sum 2^(x c - I) over the words but the target, and
//                      keeps 2^(x c - I) in fp16 (c = log2(e) / T); the logits themselves are not kept
//                      (for x c of millions: see kFar)
//   k_lce_rows         a token's I and s over the vocabulary, its lse and logp, and dx in bf16 over
//                      the exponentials: one read and one write of them
//   k_lce_grad_hidden  dx W, in parts of the vocabulary where there are few tiles
//   k_lce_join         the parts' sum
//   k_lce_grad_weight  dx^T h
//   k_lce_loss         the tokens' sum
//
// Why exponentials are kept and not computed again: the products are all but the
// whole time (2 T D V flops each), and to compute x twice is a fourth beside the
// three that have to be; keeping 16 bits of it costs 4 bytes a word and token of
// memory traffic (0.74 of 17 ms at 8192 tokens of 128256 words).
//
// Rounding.  An exponential is kept as 2^(x c - I + 15) in fp16: 2^-11 relative at
// most down to 2^-29 of the largest of its 128 words, and below that an error of
// 2^-40 of it.  A power of two moves it to the row's scale exactly.  dx is rounded
// to bf16 once; under a mean it is kept without the mean's factor, whose rounding
// would lean the same way in every token's target (bf16 gradients were up to 3.3e-3
// off for it, and are 2.0e-3 to 2.3e-3 off without; 1.7e-3 is the rounding of the
// result alone).  Given weights are in dx, and what they are all alike in leans so.
// The sum over the words without the target, R, is kept apart from the target's
// exponential E: its own dx is -R / (R + E), not 1 less a rounded q, and
// logp = -ln(1 + R / E), so a token that is nearly certain has both to the last bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <string>
#include <type_traits>

#include "adafactor_internal.h"
#include "linear_ce.h"
#include "tc_host.cuh"

namespace {

using meo::tc::Part;
using meo::tc::Shape;

constexpr int64_t kMaxTokens = int64_t{1} << 26, kMaxDim = int64_t{1} << 16, kMaxVocab = int64_t{1} << 21;
constexpr int64_t kPieceBytes = int64_t{1} << 31;   // of a piece's exponentials
constexpr int kSpan = 128;                          // words of one I and s
// The tensor cores cut off what does not fit the 24 bits of a sum, at each of its steps of 16
// values: measured, a sum of n steps comes out smaller by 0.54 n 2^-25 of itself (0.42 to 0.56, for
// terms of one sign and of both, 256 to 16384 values).  4096 values at once leave logits 4e-6 off,
// and log-probabilities 1.6e-5 of themselves.  So logits are summed in parts of 1024 values,
// 1e-6 off, and c = log2(e) / T makes up for the mean of it: 1e-7 is left on the average, and up to 1e-6 of a
// single logit.  (One token's log-probability over 4096 values is 1.4e-7 of itself off in the middle of 60, 1.2e-6
// at most; in fp32 torch operations 9e-8 and 9.7e-7.  Parts of 512 values take 5 % longer, 2.5 % parts of 1024.)
constexpr int kSumStages = 16;
constexpr double kCutOff = 0.54 / (1 << 25);
// The gradients' sums are longer, and one that grows all the way loses more (products far below it lose
// bits of their own): the gradient of a word that most of 2^21 tokens have as their target came out 7e-3
// too small in one sum, those of tokens whose target comes first of 2^19 words 1.1e-3.  So a piece has at
// most 2^16 tokens (2.0e-4), and the hidden gradient's sums go over 2^17 words at once (2.6e-4, in bf16
// an eighth of what its rounding is).  Vocabularies of more words have an ending of their own that adds
// up in registers (in one kernel with the usual one it cost every call 2.5 us, 1 % of 16 tokens' 220).
constexpr int64_t kMostRows = int64_t{1} << 16, kMostWords = int64_t{1} << 17;
constexpr int kScanThreads = 1024, kScanEach = 8;
constexpr float kLn2 = 0.6931471805599453f;
// From here on the whole number I (or 15 - I) and x c are too far apart for fp32: such a span's
// exponentials are relative to 2^(top c) itself, top its largest logit, and (top, -s) is kept
// of it in place of (I, s).
constexpr float kFar = 4194304.f;
constexpr int kIgnored = -1, kBad = -2;

struct Rows {
  const void* p;
  int64_t sb, ss;
};

struct CeArgs {
  const void* h;
  int32_t h_bf16, g_bf16;
  int64_t hsb, hss, gsb, gss;
  void* g;                   // the hidden states' gradient; NULL: none
  Rows y;
  int32_t y64;
  int64_t ignore;
  Rows w;                    // NULL: the mean
  int32_t tokens, seq, dim, vocab;
  int32_t ldh, lde, spans;   // of the gathered hidden states, of the exponentials; spans of a row
  int32_t first, rows;       // the piece: its first row, rows that it has room for
  float c_hi, c_lo, inv_t, z_loss, scale;
  int32_t* count;            // tokens that count
  int32_t* status;
  int32_t* token;            // [rows] which token a row is
  int32_t* target;           // [rows]
  __nv_bfloat16* hc;         // [rows][ldh]
  float* xt;                 // [rows of a piece]: the target's logit
  float2* stat;              // [rows of a piece][spans]
  unsigned short* e;         // [rows of a piece][lde]; NULL: no gradient
  float* part;               // [rows] w (z_loss lse^2 - logp)
  float* loss;
  float* logp;
  float* lse;
};

__device__ __forceinline__ int64_t place(int t, int seq, int64_t sb, int64_t ss) {
  const int b = t / seq;
  return b * sb + (t - b * seq) * ss;
}
__device__ __forceinline__ int target_of(const CeArgs& a, int t) {
  const int64_t at = place(t, a.seq, a.y.sb, a.y.ss);
  const int64_t y = a.y64 ? static_cast<const int64_t*>(a.y.p)[at] : static_cast<const int32_t*>(a.y.p)[at];
  return y == a.ignore ? kIgnored : y < 0 || y >= a.vocab ? kBad : static_cast<int>(y);
}

// ---- tokens ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kScanThreads) k_lce_scan(const CeArgs a) {
  meo::tc::next_may_begin();
  __shared__ int warps[32];
  __shared__ int total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kScanThreads * kScanEach) {
    int y[kScanEach], n = 0;
    const int64_t mine = t0 + threadIdx.x * kScanEach;
#pragma unroll
    for (int i = 0; i < kScanEach; ++i) {
      y[i] = mine + i < a.tokens ? target_of(a, static_cast<int>(mine + i)) : kIgnored;
      n += y[i] != kIgnored;
    }
    int up = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (lane == 31) warps[warp] = up;
    __syncthreads();
    if (warp == 0) {
      int v = warps[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      warps[lane] = v;
      if (lane == 31) total = v;
    }
    __syncthreads();
    int at = base + (warp ? warps[warp - 1] : 0) + up - n;
#pragma unroll
    for (int i = 0; i < kScanEach; ++i)
      if (y[i] != kIgnored) {
        a.token[at] = static_cast<int>(mine + i);
        a.target[at++] = y[i];
      }
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    *a.count = base;
    *a.status = 0;
  }
}

__device__ __forceinline__ uint32_t pack(float x, float y) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&two);
}

// Which token row i is, and how many count, by looking at all targets: for few tokens in place of
// k_lce_scan, whose launch takes longer.
__device__ __forceinline__ int find_token(const CeArgs& a, int i, int* n) {
  __shared__ int warps[4], found[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int t0 = 0; t0 < a.tokens; t0 += 128) {
    const int t = t0 + static_cast<int>(threadIdx.x), y = t < a.tokens ? target_of(a, t) : kIgnored;
    const unsigned votes = __ballot_sync(0xffffffffu, y != kIgnored);
    if (lane == 0) warps[warp] = __popc(votes);
    __syncthreads();
    int at = base + __popc(votes & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += warps[w];
    if (y != kIgnored && at == i) {
      found[0] = t;
      found[1] = y;
    }
    base += warps[0] + warps[1] + warps[2] + warps[3];
    __syncthreads();
  }
  *n = base;
  if (i >= base) return 0;
  if (threadIdx.x == 0) {
    a.token[i] = found[0];
    a.target[i] = found[1];
  }
  return found[0];
}
constexpr int kFewTokens = 512;

// Row i of the gathered hidden states, up to a multiple of 64 rows (zeros beyond the
// last token), and what an ignored token i is answered.
__global__ void __launch_bounds__(128) k_lce_gather(const CeArgs a) {
  meo::tc::next_may_begin();
  meo::tc::previous_done();
  const int i = blockIdx.x;
  int n, token = 0;
  if (a.tokens <= kFewTokens) {
    token = find_token(a, i, &n);
    if (i == 0 && threadIdx.x == 0) {
      *a.count = n;
      *a.status = 0;
    }
  } else {
    n = *a.count;
    if (i < n) token = a.token[i];
  }
  if (i < ((n + 63) & ~63)) {
    __nv_bfloat16* const to = a.hc + static_cast<int64_t>(i) * a.ldh;
    if (i < n) {
      const int64_t at = place(token, a.seq, a.hsb, a.hss);
      if (a.h_bf16) {
        const __nv_bfloat16* const from = static_cast<const __nv_bfloat16*>(a.h) + at;
        int d = 0;
        if (reinterpret_cast<uintptr_t>(from) % 16 == 0) {
          d = a.dim & ~7;
          for (int k = threadIdx.x; k < a.dim >> 3; k += 128)
            reinterpret_cast<uint4*>(to)[k] = reinterpret_cast<const uint4*>(from)[k];
        }
        for (int k = d + threadIdx.x; k < a.dim; k += 128) to[k] = from[k];
      } else {
        const float* const from = static_cast<const float*>(a.h) + at;
        for (int k = threadIdx.x; k < a.dim; k += 128) to[k] = __float2bfloat16_rn(from[k]);
      }
      for (int k = a.dim + threadIdx.x; k < a.ldh; k += 128) to[k] = __float2bfloat16_rn(0.f);
    } else {
      for (int k = threadIdx.x; k < a.ldh; k += 128) to[k] = __float2bfloat16_rn(0.f);
    }
  }
  if (i < a.tokens && target_of(a, i) == kIgnored) {
    if (threadIdx.x == 0) {
      if (a.logp != nullptr) a.logp[i] = 0.f;
      if (a.lse != nullptr) a.lse[i] = 0.f;
    }
    if (a.g != nullptr) {
      const int64_t at = place(i, a.seq, a.gsb, a.gss);
      for (int k = threadIdx.x; k < a.dim; k += 128) {
        if (a.g_bf16)
          static_cast<__nv_bfloat16*>(a.g)[at + k] = __float2bfloat16_rn(0.f);
        else
          static_cast<float*>(a.g)[at + k] = 0.f;
      }
    }
  }
}

// The weight in bf16 with rows of a multiple of 8 values, 8 values a thread.  Rows whose values lie at
// any place are read value by value, eight of a thread's under way together: 85456 x 949 in bf16 59 us
// (5.5 TB/s; 154 with one at a time), 32000 x 4096 in fp32 118 (6.7 TB/s).
__global__ void __launch_bounds__(256) k_lce_weight(const void* w, int32_t bf16, int64_t stride, int32_t vocab, int32_t dim, int32_t ld,
                                                    __nv_bfloat16* to) {
  meo::tc::next_may_begin();
  meo::tc::previous_done();
  const int across = ld >> 3;
  const int64_t vecs = static_cast<int64_t>(vocab) * across;
  const bool wide = bf16 == 0 && stride % 4 == 0 && reinterpret_cast<uintptr_t>(w) % 16 == 0;
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < vecs; i += gridDim.x * 256) {
    // (a division of 64 bits takes as long as the copy)
    const int64_t v = i >> 32 == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(across) : i / across;
    const int k = static_cast<int>(i - v * across) * 8, left = dim - k;
    const int64_t at = v * stride + k;
    float x[8];
    if (wide && left >= 8) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(w) + at));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(w) + at) + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else if (bf16 != 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < left ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[at + e]) : 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < left ? static_cast<const float*>(w)[at + e] : 0.f;
    }
    reinterpret_cast<uint4*>(to)[i] = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
  }
}

// ---- logits to exponentials --------------------------------------------------------------
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool KEEP>
struct LogitsEnd {
  static constexpr int kChunk = kSumStages;
  struct Args {
    float c_hi, c_lo;
    const int32_t* target;   // of the piece
    float* xt;
    float2* stat;
    unsigned short* e;
    int32_t lde, spans;
  };
  // the columns of a group are one span: 128 words
  static __device__ __forceinline__ void whole(const Args& a, const Part& p, float (&v)[kSpan]) {
    if (p.col >= p.n) return;
    const bool mine = p.row < p.m;
    const int at = mine ? a.target[p.row] - p.col : -1, left = p.n - p.col;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      if (i >= left) v[i] = -INFINITY;
      top = fmaxf(top, v[i]);
    }
    if (at >= 0 && at < kSpan) {
#pragma unroll
      for (int i = 0; i < kSpan; ++i)
        if (i == at) a.xt[p.row] = v[i];
    }
    // (nothing but -inf or NaN leaves top at -inf: the sum is NaN or 0 then)
    const bool none = !(top > -INFINITY);
    const float I = ceilf(fmaf(top, a.c_hi, top * a.c_lo));   // (-inf: no words)
    const bool far = !none && fabsf(I) >= kFar;
    if (far) {
#pragma unroll
      for (int i = 0; i < kSpan; ++i) v[i] -= top;
    }
    const float shift = far || none ? 15.f : 15.f - I;
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kSpan; c += 32) {
      float some = 0.f;
#pragma unroll
      for (int i = c; i < c + 32; ++i) {
        // (-inf stays -inf: c_lo is above 0)
        v[i] = i < left ? exp2_approx(fmaf(v[i], a.c_lo, fmaf(v[i], a.c_hi, shift))) : 0.f;
        some += v[i];
      }
      if (at >= c && at < c + 32) {
        some = 0.f;
#pragma unroll
        for (int i = c; i < c + 32; ++i)
          if (i != at) some += v[i];
      }
      sum += some;
      if (KEEP && c < left) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t k[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const __half2 two = __floats2half2_rn(v[c + 8 * i + 2 * q], v[c + 8 * i + 2 * q + 1]);
            k[q] = *reinterpret_cast<const uint32_t*>(&two);
          }
          w[i] = make_uint4(k[0], k[1], k[2], k[3]);
        }
        p.ex.to_memory(w);
        p.ex.put(a.e + static_cast<int64_t>(p.row0()) * a.lde + p.col + c, static_cast<int64_t>(a.lde) * 2, p.m - p.row0(),
                 (a.lde - p.col - c) * 2, w);
      }
    }
    if (mine) a.stat[static_cast<int64_t>(p.row) * a.spans + p.col / kSpan] = far ? make_float2(top, -sum) : make_float2(I, sum);
  }
};

// ---- a token's softmax, and dx ---------------------------------------------------------------
__device__ __forceinline__ float power_of_two(float d) {   // 2^d for a whole d <= 0
  return d < -126.f ? 0.f : __int_as_float((static_cast<int>(d) + 127) << 23);
}

// What a row's exponentials are relative to: 2^top, or with far spans (kFar) maybe 2^(t c).
struct Reference {
  float top, t;
  bool any, far;        // there are far spans; t counts
  __device__ __forceinline__ float times(const CeArgs& a, float x, float less) const { return fmaf(x, a.c_lo, fmaf(x, a.c_hi, -less)); }
  // A span's 2^I, or 2^(top c), over the row's.
  __device__ __forceinline__ float scale(const CeArgs& a, const float2& s) const {
    if (!any) return power_of_two(s.x - top);
    if (!signbit(s.y)) return far ? exp2f(-times(a, t, s.x)) : power_of_two(s.x - top);
    return exp2f(far ? times(a, s.x - t, 0.f) : times(a, s.x, top));
  }
};

// A row a CTA: of 1024 threads where there are few rows (16 rows of 32000 words 5 us less).
template <int kRowThreads>
__global__ void __launch_bounds__(kRowThreads) k_lce_rows(const CeArgs a) {
  __shared__ float s_max[kRowThreads / 32], s_far[kRowThreads / 32], s_sum[kRowThreads / 32];
  meo::tc::next_may_begin();
  meo::tc::previous_done();
  const int r = blockIdx.x;
  const int n = *a.count, live = min(a.rows, n - a.first);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4* const e = a.e != nullptr ? reinterpret_cast<uint4*>(a.e + static_cast<int64_t>(r) * a.lde) : nullptr;
  const int vecs = a.lde >> 3;
  if (r >= live) {
    // rows up to a multiple of 64 count as zeros in the weight's gradient
    if (live > 0 && r < ((live + 63) & ~63) && e != nullptr)
      for (int i = threadIdx.x; i < vecs; i += kRowThreads) e[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const float2* const stat = a.stat + static_cast<int64_t>(r) * a.spans;
  Reference ref{-INFINITY, -INFINITY, false, false};
  for (int i = threadIdx.x; i < a.spans; i += kRowThreads) {
    const float2 s = stat[i];
    float& most = signbit(s.y) ? ref.t : ref.top;
    most = fmaxf(most, s.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ref.top = fmaxf(ref.top, __shfl_xor_sync(0xffffffffu, ref.top, o));
    ref.t = fmaxf(ref.t, __shfl_xor_sync(0xffffffffu, ref.t, o));
  }
  if (lane == 0) {
    s_max[warp] = ref.top;
    s_far[warp] = ref.t;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) {
    ref.top = fmaxf(ref.top, s_max[w]);
    ref.t = fmaxf(ref.t, s_far[w]);
  }
  ref.any = ref.t > -INFINITY;
  ref.far = ref.any && ref.times(a, ref.t, 0.f) >= ref.top;
  float sum = 0.f;
  for (int i = threadIdx.x; i < a.spans; i += kRowThreads) {
    const float2 s = stat[i];
    sum = fmaf(fabsf(s.y), ref.scale(a, s), sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) sum += s_sum[w];

  const int i = a.first + r, t = a.token[i], y = a.target[i];
  const float nan = __int_as_float(0x7fc00000);
  // rest: the words without the target; own: the target (both over the row's reference)
  const float rest = sum * 0x1p-15f;
  float own = 0.f, far = 0.f;
  if (y >= 0) {
    const float x = a.xt[r];
    far = ref.far ? ref.times(a, x - ref.t, 0.f) : ref.times(a, x, ref.top);
    own = exp2f(far);
  }
  const float all = rest + own;
  const float log_s = log2f(all);
  // (no word above -inf: no distribution)
  const float lse = !(all > 0.f) ? nan : ref.far ? fmaf(kLn2 * ref.t, a.c_hi, kLn2 * log_s) : kLn2 * (ref.top + log_s);
  const float logp = y < 0 ? nan : own > rest ? -log1pf(rest / own) : kLn2 * (far - log_s);
  const float w = a.w.p != nullptr ? static_cast<const float*>(a.w.p)[place(t, a.seq, a.w.sb, a.w.ss)] : 1.f / static_cast<float>(n);
  if (threadIdx.x == 0) {
    a.part[i] = w * (a.z_loss * lse * lse - logp);
    if (a.logp != nullptr) a.logp[t] = logp;
    if (a.lse != nullptr) a.lse[t] = lse;
  }
  if (e == nullptr) return;
  // (the mean's factor is the endings': see Factor)
  const float d = a.w.p != nullptr ? w * a.scale * a.inv_t : 1.f, z = 2.f * a.z_loss * lse;
  // (a target outside the vocabulary makes the whole row NaN)
  const float factor = y >= 0 ? d * (1.f + z) / (all * 32768.f) : nan;
  const float at_target = d * (z * own - rest) / all;
  for (int v = threadIdx.x; v < vecs; v += kRowThreads) {
    const float f = factor * (ref.any ? ref.scale(a, stat[v >> 4]) : power_of_two(stat[v >> 4].x - ref.top));
    const uint4 q = e[v];
    const uint32_t in[4] = {q.x, q.y, q.z, q.w};
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&in[k]));
      const int j = 8 * v + 2 * k;
      out[k] = pack(j == y ? at_target : x.x * f, j + 1 == y ? at_target : x.y * f);
    }
    e[v] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ---- gradients --------------------------------------------------------------------------------
// What the products of dx still have to be multiplied by: under a mean, scale / (T count).
struct Factor {
  const int32_t* count;      // NULL: nothing
  float scale;
  __device__ __forceinline__ float value() const { return count == nullptr ? 1.f : scale / static_cast<float>(max(1, *count)); }
};

// Writes the warp's 32 rows of 32 values of a result, fp32 or bf16: row i at out + row(i), of
// which `left` values are there; load: adds what is there first.
template <class RowAt>
__device__ __forceinline__ void store32(const Part& p, void* out, bool bf16, bool wide, bool load, RowAt&& row_at, int left, float (&v)[32]) {
  const meo::tc::Exchange& x = p.ex;
  const int rows = p.m - p.row0();
  if (bf16 && !load) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_uint4(pack(v[8 * i], v[8 * i + 1]), pack(v[8 * i + 2], v[8 * i + 3]), pack(v[8 * i + 4], v[8 * i + 5]),
                        pack(v[8 * i + 6], v[8 * i + 7]));
    x.to_memory(w);
    const int j = x.place() / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (x.row(i) >= rows || j >= left) continue;
      __nv_bfloat16* const q = static_cast<__nv_bfloat16*>(out) + row_at(i) + j;
      if (wide && j + 8 <= left) {
        *reinterpret_cast<uint4*>(q) = w[i];
      } else {
        const __nv_bfloat16* const k = reinterpret_cast<const __nv_bfloat16*>(&w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (j + e < left) q[e] = k[e];
      }
    }
    return;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_uint4(__float_as_uint(v[16 * half + 4 * i]), __float_as_uint(v[16 * half + 4 * i + 1]),
                        __float_as_uint(v[16 * half + 4 * i + 2]), __float_as_uint(v[16 * half + 4 * i + 3]));
    x.to_memory(w);
    const int j = 16 * half + x.place() / 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (x.row(i) >= rows || j >= left) continue;
      float r[4] = {__uint_as_float(w[i].x), __uint_as_float(w[i].y), __uint_as_float(w[i].z), __uint_as_float(w[i].w)};
      if (bf16) {   // added to what is there
        __nv_bfloat16* const q = static_cast<__nv_bfloat16*>(out) + row_at(i) + j;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < left) q[e] = __float2bfloat16_rn(r[e] + __bfloat162float(q[e]));
        continue;
      }
      float* const q = static_cast<float*>(out) + row_at(i) + j;
      if (wide && j + 4 <= left) {
        if (load) {
          const float4 o = *reinterpret_cast<const float4*>(q);
          r[0] += o.x, r[1] += o.y, r[2] += o.z, r[3] += o.w;
        }
        *reinterpret_cast<float4*>(q) = make_float4(r[0], r[1], r[2], r[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < left) q[e] = r[e] + (load ? q[e] : 0.f);
      }
    }
  }
}

struct HiddenArgs {
  const int32_t* token;     // of the piece
  void* out;
  int64_t sb, ss;
  int32_t seq, bf16, wide;
  float* parts;             // where sums are in several parts: [splits][rows that count][dim]
  Factor factor;
};
// LONG: sums over more than kMostWords words.
template <bool LONG>
struct HiddenEnd {
  static constexpr int kChunk = LONG ? static_cast<int>(kMostWords / meo::tc::kBlockK) : 0;
  using Args = HiddenArgs;
  // col32(c, v): 32 columns of the sums
  template <class Columns>
  static __device__ __forceinline__ void store(const Args& a, const Part& p, Columns&& col32) {
    const float f = a.factor.value();
    const bool parts = p.splits > 1;   // then summed by k_lce_join
    int64_t at[4];   // of the rows that this lane writes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = p.row0() + p.ex.row(i);
      at[i] = r >= p.m ? 0 : parts ? (static_cast<int64_t>(p.tile.split) * p.m + r) * p.n : place(a.token[r], a.seq, a.sb, a.ss);
    }
#pragma unroll 1
    for (int c = 0; c < p.cols && p.col + c < p.n; c += 32) {
      float v[32];
      col32(c, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= f;
      const int j = p.col + c;
      if (parts)
        store32(p, a.parts, false, p.n % 4 == 0, false, [&](int i) { return at[i] + j; }, p.n - j, v);
      else
        store32(p, a.out, a.bf16, a.wide, false, [&](int i) { return at[i] + j; }, p.n - j, v);
    }
  }
  static __device__ __forceinline__ void part(const Args& a, const Part& p) {
    store(a, p, [&](int c, float (&v)[32]) { p.load(c, v); });
  }
  static __device__ __forceinline__ void whole(const Args& a, const Part& p, float (&sum)[kSpan]) {
    store(a, p, [&](int c, float (&v)[32]) {
#pragma unroll
      for (int k = 0; k < kSpan; k += 32)
        if (c == k) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = sum[k + i];
        }
    });
  }
};

// A token's hidden gradient from its parts, in their order.
__global__ void __launch_bounds__(256) k_lce_join(int32_t dim, int32_t blocks, int32_t clusters, int64_t room, const int32_t* count,
                                                  int32_t first, int32_t most, const HiddenArgs o) {
  meo::tc::next_may_begin();
  meo::tc::previous_done();
  const int rows = meo::tc::live(count, first, most);
  const int splits = meo::tc::splits_of(rows, dim, blocks, 256, 256, clusters, room);
  if (splits == 1) return;
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t at = place(o.token[r], o.seq, o.sb, o.ss);
    const float* const parts = o.parts + static_cast<int64_t>(r) * dim;
    const int64_t part = static_cast<int64_t>(rows) * dim;
    if (dim % 4 == 0 && o.wide) {
      for (int k = 4 * (blockIdx.y * 256 + threadIdx.x); k < dim; k += 4 * gridDim.y * 256) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
          const float4 x = __ldcs(reinterpret_cast<const float4*>(parts + s * part + k));
          v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
        }
        if (o.bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o.out) + at + k) = make_uint2(pack(v.x, v.y), pack(v.z, v.w));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(o.out) + at + k) = v;
      }
      continue;
    }
    for (int k = blockIdx.y * 256 + threadIdx.x; k < dim; k += gridDim.y * 256) {
      float v = 0.f;
      for (int s = 0; s < splits; ++s) v += __ldcs(parts + s * part + k);
      if (o.bf16)
        static_cast<__nv_bfloat16*>(o.out)[at + k] = __float2bfloat16_rn(v);
      else
        static_cast<float*>(o.out)[at + k] = v;
    }
  }
}

struct WeightEnd {
  static constexpr int kChunk = 0;
  struct Args {
    void* out;
    int64_t stride;
    int32_t bf16, wide;
    float* sum;                // [vocab][dim] over the pieces; NULL: there is one, or the result is fp32
    int32_t load_sum, load_out, last;
    Factor factor;
  };
  static __device__ __forceinline__ void part(const Args& a, const Part& p) {
    if (p.zero && !a.last && (a.sum != nullptr ? a.load_sum : a.load_out)) return;   // nothing to add
    const float f = a.factor.value();
    const auto row_at = [&](int i) { return (p.row0() + p.ex.row(i)) * a.stride; };
    if (a.sum == nullptr && a.bf16 && a.wide && !a.load_out && p.col + p.cols <= p.n) {
      // the usual case: few tokens leave little time for a tile
      const int64_t at[4] = {row_at(0), row_at(1), row_at(2), row_at(3)};
#pragma unroll 1
      for (int c = 0; c < p.cols; c += 64) {
        float v[32], w[32];
        p.load64(c, v, w);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float(&x)[32] = half == 0 ? v : w;
          uint4 q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            q[i] = make_uint4(pack(x[8 * i] * f, x[8 * i + 1] * f), pack(x[8 * i + 2] * f, x[8 * i + 3] * f),
                              pack(x[8 * i + 4] * f, x[8 * i + 5] * f), pack(x[8 * i + 6] * f, x[8 * i + 7] * f));
          p.ex.to_memory(q);
          __nv_bfloat16* const to = static_cast<__nv_bfloat16*>(a.out) + p.col + c + 32 * half + p.ex.place() / 2;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p.row0() + p.ex.row(i) < p.m) *reinterpret_cast<uint4*>(to + at[i]) = q[i];
        }
      }
      return;
    }
#pragma unroll 1
    for (int c = 0; c < p.cols && p.col + c < p.n; c += 32) {
      float v[32];
      p.load(c, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= f;
      const int j = p.col + c, left = p.n - j;
      if (a.sum != nullptr) {
        const auto sum_at = [&](int i) { return static_cast<int64_t>(p.row0() + p.ex.row(i)) * p.n + j; };
        if (!a.last) {
          store32(p, a.sum, false, p.n % 4 == 0, a.load_sum, sum_at, left, v);
          continue;
        }
        if (p.row < p.m) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < left) v[i] += a.sum[static_cast<int64_t>(p.row) * p.n + j + i];
        }
      }
      store32(p, a.out, a.bf16, a.wide, a.load_out, [&](int i) { return row_at(i) + j; }, left, v);
    }
  }
};

// An fp32 sum that carries what its additions round off.
struct Sum {
  float s = 0.f, rest = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
    rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
  }
  __device__ __forceinline__ void add(const Sum& o) {
    add(o.s);
    rest = __fadd_rn(rest, o.rest);
  }
  __device__ __forceinline__ float total() const { return fabsf(s) == INFINITY ? s : s + rest; }
};

__global__ void __launch_bounds__(1024) k_lce_loss(const CeArgs a) {
  __shared__ Sum warps[32];
  meo::tc::previous_done();
  const int n = *a.count;
  Sum s;
  for (int i = threadIdx.x; i < n; i += 1024) s.add(a.part[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum other;
    other.s = __shfl_down_sync(0xffffffffu, s.s, o);
    other.rest = __shfl_down_sync(0xffffffffu, s.rest, o);
    s.add(other);
  }
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    Sum all;
    for (int w = 0; w < 32; ++w) all.add(warps[w]);
    *a.loss = *a.status != 0 ? __int_as_float(0x7fc00000) : all.total();
  }
}

// ---- host side ------------------------------------------------------------------------------
adaf_status fail(adaf_status st, const std::string& msg) { return meo::set_last_error(st, ("linear_ce: " + msg).c_str()); }
adaf_status invalid(const std::string& msg) { return fail(ADAF_ERR_INVALID_ARGUMENT, msg); }
adaf_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(ADAF_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(a) == 0; }
int64_t size_of(int32_t dtype) { return dtype == ADAF_BFLOAT16 ? 2 : 4; }
bool known(int32_t dtype) { return dtype == ADAF_BFLOAT16 || dtype == ADAF_FLOAT32; }

const char* const kKernelNames[] = {"k_lce_scan", "k_lce_gather", "k_lce_weight",      "k_lce_logits", "k_lce_rows", "k_lce_grad_hidden",
                                    "k_lce_join", "k_lce_grad_weight", "k_lce_loss"};
constexpr int kNumKernels = 9;
enum Slot { kSlotScan, kSlotGather, kSlotWeight, kSlotLogits, kSlotRows, kSlotGradHidden, kSlotJoin, kSlotGradWeight, kSlotLoss };
meo::tc::Profile g_profile;
thread_local bool t_stall = false;

constexpr int64_t kMaxStride = int64_t{1} << 38;

// [p, end) of a tensor's bytes.
struct Extent {
  uintptr_t from, to;
  bool meets(const Extent& o) const { return from < o.to && o.from < to; }
};
Extent extent(const linear_ce_hidden& h) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(h.p);
  return {p, p + static_cast<uintptr_t>(((h.batch - 1) * h.stride_b + (h.seq - 1) * h.stride_s + h.dim) * size_of(h.dtype))};
}
Extent extent(const linear_ce_weight& w, int64_t dim) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(w.p);
  return {p, p + static_cast<uintptr_t>(((w.vocab - 1) * w.stride_v + dim) * size_of(w.dtype))};
}

adaf_status check_sizes(const linear_ce_hidden* h, const linear_ce_weight* w, const linear_ce_hidden* gh, const linear_ce_weight* gw) {
  if (h == nullptr || w == nullptr) return invalid("hidden or weight is NULL");
  if (!known(h->dtype)) return invalid("hidden: unknown dtype");
  if (!known(w->dtype)) return invalid("weight: unknown dtype");
  if (h->batch < 0 || h->seq < 0) return invalid("hidden: negative batch or seq");
  if (h->dim < 1) return invalid("hidden: dim must be at least 1");
  if (w->vocab < 1) return invalid("weight: vocab must be at least 1");
  if (h->dim > kMaxDim || w->vocab > kMaxVocab) return fail(ADAF_ERR_UNSUPPORTED, "dim above 2^16 or vocab above 2^21");
  if (h->batch > kMaxTokens || h->seq > kMaxTokens || h->batch * h->seq > kMaxTokens) return fail(ADAF_ERR_UNSUPPORTED, "more than 2^26 tokens");
  if (w->stride_v < 0 || (w->vocab > 1 && w->stride_v < h->dim)) return invalid("weight: rows overlap (stride)");
  if (w->stride_v > kMaxStride) return invalid("weight: strides must be 0 to 2^38");
  if (gh != nullptr) {
    if (!known(gh->dtype)) return invalid("grad_hidden: unknown dtype");
    if (gh->batch != h->batch || gh->seq != h->seq || gh->dim != h->dim) return invalid("grad_hidden: not the hidden states' size");
  }
  if (gw != nullptr) {
    if (!known(gw->dtype)) return invalid("grad_weight: unknown dtype");
    if (gw->vocab != w->vocab) return invalid("grad_weight: not the weight's size");
  }
  return ADAF_OK;
}

// How a call is cut, and where things are in the workspace.
struct Plan {
  int64_t tokens, room, rows, pieces;   // room: rows of the gathered hidden states; rows: of a piece
  int64_t ldh, lde, ldw, spans;
  int64_t split_room;                   // values of the parts of the hidden gradient's sums
  bool packed;                          // the weight is copied
  size_t token, target, part, hc, xt, stat, e, w, parts, sum, bytes;
};

Plan plan(const linear_ce_hidden& h, const linear_ce_weight& w, const linear_ce_hidden* gh, const linear_ce_weight* gw) {
  Plan P{};
  const bool grad = gh != nullptr || gw != nullptr;
  P.tokens = h.batch * h.seq;
  P.room = round_up(P.tokens, 64);
  P.ldh = round_up(h.dim, 8);
  P.lde = round_up(w.vocab, 64);
  P.spans = (w.vocab + kSpan - 1) / kSpan;
  P.rows = std::min({P.room, kMostRows, std::max<int64_t>(256, kPieceBytes / (P.lde * 2) / 256 * 256)});
  P.pieces = P.rows > 0 ? (P.tokens + P.rows - 1) / P.rows : 0;   // (no tokens, no rows)
  // (a single row's stride says nothing)
  P.packed = w.dtype != ADAF_BFLOAT16 || !aligned(w.p, 16) || (w.vocab > 1 && w.stride_v % 8 != 0);
  P.ldw = P.packed || w.vocab == 1 ? P.ldh : w.stride_v;
  // up to 16 parts, of 256 MB together
  P.split_room = std::min(P.rows * h.dim * 16, int64_t{1} << 26);
  size_t o = 256;
  auto take = [&](int64_t bytes) {
    const size_t at = o;
    o = static_cast<size_t>(round_up(static_cast<int64_t>(o) + bytes, 256));
    return at;
  };
  P.token = take(P.tokens * 4);
  P.target = take(P.tokens * 4);
  P.part = take(P.tokens * 4);
  P.hc = take(P.room * P.ldh * 2);
  P.xt = take(P.rows * 4);
  P.stat = take(P.rows * P.spans * 8);
  if (grad) P.e = take(P.rows * P.lde * 2);
  if (P.packed) P.w = take(w.vocab * P.ldw * 2);
  if (gh != nullptr) P.parts = take(P.split_room * 4);
  if (gw != nullptr && P.pieces > 1 && gw->dtype == ADAF_BFLOAT16) P.sum = take(w.vocab * h.dim * 4);
  P.bytes = o;
  return P;
}

#define LCE_TRY(expr, what)                           \
  do {                                                \
    const cudaError_t e_ = (expr);                    \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)

}  // namespace

extern "C" {

adaf_status linear_ce_workspace_size(const linear_ce_hidden* hidden, const linear_ce_weight* weight, const linear_ce_hidden* grad_hidden,
                                     const linear_ce_weight* grad_weight, size_t* bytes) {
  if (bytes == nullptr) return invalid("bytes is NULL");
  const adaf_status st = check_sizes(hidden, weight, grad_hidden, grad_weight);
  if (st != ADAF_OK) return st;
  *bytes = plan(*hidden, *weight, grad_hidden, grad_weight).bytes;
  return ADAF_OK;
}

adaf_status linear_ce(const linear_ce_hidden* hidden, const linear_ce_weight* weight, const loss_targets* targets,
                      const linear_ce_args* args, const linear_ce_hidden* grad_hidden, const linear_ce_weight* grad_weight, float* loss,
                      float* logp, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const linear_ce_hidden* const gh = grad_hidden != nullptr && grad_hidden->p != nullptr ? grad_hidden : nullptr;
  const linear_ce_weight* const gw = grad_weight != nullptr && grad_weight->p != nullptr ? grad_weight : nullptr;
  const adaf_status st = check_sizes(hidden, weight, gh, gw);
  if (st != ADAF_OK) return st;
  if (targets == nullptr || args == nullptr) return invalid("targets or args is NULL");
  const linear_ce_hidden& h = *hidden;
  const linear_ce_weight& w = *weight;
  const int64_t tokens = h.batch * h.seq;
  // strides of rows that reach no further than 2^46 values, so that no place overflows
  auto bad_stride = [](int64_t s) { return s < 0 || s > kMaxStride; };
  auto too_far = [&](int64_t sb, int64_t ss) {
    constexpr int64_t kReach = int64_t{1} << 46;
    return (h.batch > 1 && sb > kReach / (h.batch - 1)) || (h.seq > 1 && ss > kReach / (h.seq - 1));
  };
  if (bad_stride(h.stride_b) || bad_stride(h.stride_s) || too_far(h.stride_b, h.stride_s)) return invalid("hidden: strides must be 0 to 2^38, and reach 2^46 values");
  if (tokens > 0 && h.p == nullptr) return invalid("hidden is NULL");
  if (w.p == nullptr) return invalid("weight is NULL");
  if (!aligned(h.p, size_of(h.dtype))) return invalid("hidden is not element-aligned");
  if (!aligned(w.p, size_of(w.dtype))) return invalid("weight is not element-aligned");
  if (targets->dtype != LOSS_INT32 && targets->dtype != LOSS_INT64) return invalid("targets: unknown dtype");
  if (tokens > 0 && targets->rows.p == nullptr) return invalid("targets is NULL");
  if (!aligned(targets->rows.p, targets->dtype == LOSS_INT64 ? 8 : 4)) return invalid("targets is not element-aligned");
  if (bad_stride(targets->rows.stride_b) || bad_stride(targets->rows.stride_s) || too_far(targets->rows.stride_b, targets->rows.stride_s))
    return invalid("targets: strides must be 0 to 2^38, and reach 2^46 values");
  if (!aligned(args->weights.p, 4)) return invalid("weights is not element-aligned");
  if (args->weights.p != nullptr && (bad_stride(args->weights.stride_b) || bad_stride(args->weights.stride_s) ||
                                     too_far(args->weights.stride_b, args->weights.stride_s)))
    return invalid("weights: strides must be 0 to 2^38, and reach 2^46 values");
  const double inv_t = 1.0 / args->temperature;
  if (!(args->temperature > 0.0) || !std::isfinite(args->temperature) || !std::isfinite(static_cast<float>(inv_t * 1.5)) ||
      static_cast<float>(inv_t) < FLT_MIN)
    return invalid("temperature must be positive, and 1 / temperature a normal fp32 number");
  if (!(args->z_loss >= 0.0) || !std::isfinite(static_cast<float>(args->z_loss))) return invalid("z_loss must be >= 0");
  if (!std::isfinite(static_cast<float>(args->grad_scale))) return invalid("grad_scale must be finite");
  if (loss == nullptr) return invalid("loss is NULL");
  if (!aligned(loss, 4) || !aligned(logp, 4) || !aligned(lse, 4)) return invalid("loss, logp or lse is not element-aligned");
  if (gh != nullptr && tokens > 0) {
    if (bad_stride(gh->stride_b) || bad_stride(gh->stride_s) || too_far(gh->stride_b, gh->stride_s))
      return invalid("grad_hidden: strides must be 0 to 2^38, and reach 2^46 values");
    if (!aligned(gh->p, size_of(gh->dtype))) return invalid("grad_hidden is not element-aligned");
    if ((gh->seq > 1 && gh->stride_s < gh->dim) || (gh->batch > 1 && gh->stride_b < (gh->seq - 1) * gh->stride_s + gh->dim))
      return invalid("grad_hidden: rows overlap");
    const bool same = gh->p == h.p && gh->dtype == h.dtype && (h.batch == 1 || gh->stride_b == h.stride_b) &&
                      (h.seq == 1 || gh->stride_s == h.stride_s);
    if (!same && extent(*gh).meets(extent(h))) return invalid("grad_hidden overlaps the hidden states, and is not in their place");
    if (extent(*gh).meets(extent(w, h.dim))) return invalid("grad_hidden overlaps the weight");
  }
  if (gw != nullptr) {
    if (!aligned(gw->p, size_of(gw->dtype))) return invalid("grad_weight is not element-aligned");
    if (bad_stride(gw->stride_v) || (gw->vocab > 1 && gw->stride_v < h.dim)) return invalid("grad_weight: rows overlap (stride)");
    if (extent(*gw, h.dim).meets(extent(w, h.dim))) return invalid("grad_weight overlaps the weight");
    if (tokens > 0 && extent(*gw, h.dim).meets(extent(h))) return invalid("grad_weight overlaps the hidden states");
    if (tokens > 0 && gh != nullptr && extent(*gw, h.dim).meets(extent(*gh))) return invalid("grad_weight overlaps grad_hidden");
  }
  const Plan P = plan(h, w, gh, gw);
  if (workspace == nullptr || !aligned(workspace, 256)) return invalid("workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < P.bytes) return fail(ADAF_ERR_WORKSPACE_TOO_SMALL, "workspace needs " + std::to_string(P.bytes) + " bytes");

  using namespace meo::tc;
  unsigned char* const ws = static_cast<unsigned char*>(workspace);
  cudaStream_t const s = static_cast<cudaStream_t>(stream);
  const bool grad = gh != nullptr || gw != nullptr;
  CeArgs a{};
  a.h = h.p;
  a.h_bf16 = h.dtype == ADAF_BFLOAT16;
  a.hsb = h.stride_b;
  a.hss = h.stride_s;
  if (gh != nullptr) {
    a.g = gh->p;
    a.g_bf16 = gh->dtype == ADAF_BFLOAT16;
    a.gsb = gh->stride_b;
    a.gss = gh->stride_s;
  }
  a.y = {targets->rows.p, targets->rows.stride_b, targets->rows.stride_s};
  a.y64 = targets->dtype == LOSS_INT64;
  a.ignore = targets->ignore_index;
  a.w = {args->weights.p, args->weights.stride_b, args->weights.stride_s};
  a.tokens = static_cast<int32_t>(tokens);
  a.seq = static_cast<int32_t>(std::max<int64_t>(1, h.seq));
  a.dim = static_cast<int32_t>(h.dim);
  a.vocab = static_cast<int32_t>(w.vocab);
  a.ldh = static_cast<int32_t>(P.ldh);
  a.lde = static_cast<int32_t>(P.lde);
  a.spans = static_cast<int32_t>(P.spans);
  a.rows = static_cast<int32_t>(P.rows);
  const double c = 1.4426950408889634 * inv_t * (1.0 + kCutOff * static_cast<double>(std::min<int64_t>((h.dim + 15) / 16, kSumStages * 4)));
  // c = c_hi + c_lo, rounded down: with c_lo above 0 a logit of -inf is -inf in both products
  a.c_hi = static_cast<float>(c);
  if (static_cast<double>(a.c_hi) >= c) a.c_hi = std::nextafter(a.c_hi, 0.f);
  a.c_lo = static_cast<float>(c - static_cast<double>(a.c_hi));
  a.inv_t = static_cast<float>(inv_t);
  a.z_loss = static_cast<float>(args->z_loss);
  a.scale = static_cast<float>(args->grad_scale);
  a.count = reinterpret_cast<int32_t*>(ws);
  a.status = a.count + 1;
  a.token = reinterpret_cast<int32_t*>(ws + P.token);
  a.target = reinterpret_cast<int32_t*>(ws + P.target);
  a.part = reinterpret_cast<float*>(ws + P.part);
  a.hc = reinterpret_cast<__nv_bfloat16*>(ws + P.hc);
  a.xt = reinterpret_cast<float*>(ws + P.xt);
  a.stat = reinterpret_cast<float2*>(ws + P.stat);
  a.e = grad ? reinterpret_cast<unsigned short*>(ws + P.e) : nullptr;
  a.loss = loss;
  a.logp = logp;
  a.lse = lse;

  int device = 0, sms = 0;
  LCE_TRY(sm_count(&device, &sms), "current device");
  // (the call's first launch begins when the stream's work before it is done; the others early)
  const bool few = tokens > 0 && tokens <= kFewTokens;
  if (!few) LCE_TRY(g_profile.run(kSlotScan, s, [&] { k_lce_scan<<<1, kScanThreads, 0, s>>>(a); return cudaGetLastError(); }), "k_lce_scan");
  if (P.room > 0)
    LCE_TRY(g_profile.run(kSlotGather, s, [&] {
      if (!few) return launch_early(k_lce_gather, dim3(static_cast<unsigned>(P.room)), 128, s, a);
      k_lce_gather<<<static_cast<unsigned>(P.room), 128, 0, s>>>(a);
      return cudaGetLastError();
    }), "k_lce_gather");
  const void* wp = w.p;
  if (P.packed && tokens > 0) {
    wp = ws + P.w;
    LCE_TRY(g_profile.run(kSlotWeight, s, [&] {
      return launch_early(k_lce_weight, dim3(static_cast<unsigned>(std::min<int64_t>((w.vocab * (P.ldw >> 3) + 255) / 256, 8 * sms))), 256, s, w.p,
                          static_cast<int32_t>(w.dtype == ADAF_BFLOAT16), w.stride_v, a.vocab, a.dim, static_cast<int32_t>(P.ldw),
                          reinterpret_cast<__nv_bfloat16*>(ws + P.w));
    }), "k_lce_weight");
  }
  const Factor factor{a.w.p != nullptr ? nullptr : a.count, a.scale * a.inv_t};
  const int nt_d = static_cast<int>((h.dim + 255) / 256);
  // without tokens one piece remains, which writes the weight's gradient
  for (int64_t piece = 0; piece < std::max<int64_t>(P.pieces, gw != nullptr ? 1 : 0); ++piece) {
    a.first = static_cast<int32_t>(piece * P.rows);
    const int64_t rows = std::min(P.rows, std::max<int64_t>(tokens - a.first, 0));
    __nv_bfloat16* const hc = a.hc + static_cast<int64_t>(a.first) * P.ldh;
    const int64_t room = std::max<int64_t>(P.room - a.first, 64), e_rows = std::max<int64_t>(P.rows, 64);
    Shape shape{};
    shape.splits = 1;
    shape.first = a.first;
    shape.status = a.status;
    shape.stall = t_stall ? 1 : 0;
    CUtensorMap h_k, w_k, e_k, w_n, e_m, h_n;
    bool ok = true;
    if (rows > 0) {
      ok = make_map(&h_k, hc, true, room, h.dim, P.ldh, 1, room * P.ldh, kBoxK) &&
           make_map(&w_k, wp, true, w.vocab, h.dim, P.ldw, 1, w.vocab * P.ldw, kBoxK);
      if (!ok) return fail(ADAF_ERR_CUDA, "cuTensorMapEncodeTiled failed");
      Shape x = shape;
      x.m = static_cast<int32_t>(rows);
      x.n = a.vocab;
      x.k = a.dim;
      x.group = 32;
      x.m_live = a.count;
      const auto logits = [&](auto keep) {
        using End = LogitsEnd<decltype(keep)::value>;
        const typename End::Args end{a.c_hi, a.c_lo, a.target + a.first, a.xt, a.stat, a.e, a.lde, a.spans};
        return g_profile.run(kSlotLogits, s, [&] {
          if (rows <= 128) return launch_product<1, 256, 4, false, false, End>(h_k, w_k, x, end, s);
          return launch_product<2, 256, 6, false, false, End>(h_k, w_k, x, end, s);
        });
      };
      const cudaError_t e = grad ? logits(std::true_type{}) : logits(std::false_type{});
      LCE_TRY(e, "k_lce_logits");
      LCE_TRY(g_profile.run(kSlotRows, s, [&] {
        const dim3 grid(static_cast<unsigned>(grad ? round_up(rows, 64) : rows));
        return rows <= 2 * sms ? launch_early(k_lce_rows<1024>, grid, 1024, s, a) : launch_early(k_lce_rows<256>, grid, 256, s, a);
      }), "k_lce_rows");
    }
    if (gh != nullptr && rows > 0) {
      ok = make_map(&e_k, a.e, true, e_rows, w.vocab, P.lde, 1, e_rows * P.lde, kBoxK) &&
           make_map(&w_n, wp, true, w.vocab, h.dim, P.ldw, 1, w.vocab * P.ldw, kBoxMN);
      if (!ok) return fail(ADAF_ERR_CUDA, "cuTensorMapEncodeTiled failed");
      const int64_t es = size_of(gh->dtype);
      const bool wide = aligned(gh->p, 16) && (h.batch == 1 || gh->stride_b * es % 16 == 0) && (h.seq == 1 || gh->stride_s * es % 16 == 0);
      const HiddenArgs end{a.token + a.first, gh->p, gh->stride_b, gh->stride_s, a.seq, a.g_bf16, wide,
                                reinterpret_cast<float*>(ws + P.parts), factor};
      Shape x = shape;
      x.m = static_cast<int32_t>(rows);
      x.n = a.dim;
      x.k = a.vocab;
      x.splits = 0;
      x.split_room = P.split_room;
      x.group = 8;
      x.m_live = a.count;
      LCE_TRY(g_profile.run(kSlotGradHidden, s, [&] {
        if (w.vocab > kMostWords) return launch_product<2, 256, 6, false, true, HiddenEnd<true>>(e_k, w_n, x, end, s);
        return launch_product<2, 256, 6, false, true, HiddenEnd<false>>(e_k, w_n, x, end, s);
      }), "k_lce_grad_hidden");
      const dim3 join(static_cast<unsigned>(std::min<int64_t>(rows, 8 * sms)),
                      static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((h.dim + 1023) / 1024, 8 * sms / rows))));
      LCE_TRY(g_profile.run(kSlotJoin, s, [&] {
        return launch_early(k_lce_join, join, 256, s, a.dim,
                            static_cast<int32_t>((w.vocab + kBlockK - 1) / kBlockK), static_cast<int32_t>(sms / 2), P.split_room,
                            static_cast<const int32_t*>(a.count), a.first, static_cast<int32_t>(rows), end);
      }), "k_lce_join");
    }
    if (gw != nullptr) {
      ok = make_map(&e_m, P.e != 0 ? static_cast<void*>(a.e) : ws, true, e_rows, w.vocab, P.lde, 1, e_rows * P.lde, kBoxMN) &&
           make_map(&h_n, hc, true, room, h.dim, P.ldh, 1, room * P.ldh, kBoxMN);
      if (!ok) return fail(ADAF_ERR_CUDA, "cuTensorMapEncodeTiled failed");
      const int64_t es = size_of(gw->dtype);
      const bool wide = aligned(gw->p, 16) && gw->stride_v * es % 16 == 0;
      const bool last = piece + 1 >= P.pieces, more = P.pieces > 1 && gw->dtype == ADAF_FLOAT32;
      // over several pieces: an fp32 result is summed in place, a bf16 one beside it
      const WeightEnd::Args end{gw->p, gw->stride_v, gw->dtype == ADAF_BFLOAT16, wide,
                                P.sum != 0 ? reinterpret_cast<float*>(ws + P.sum) : nullptr, piece > 0,
                                gw->accumulate != 0 || (more && piece > 0), last, factor};
      Shape x = shape;
      x.m = a.vocab;
      x.n = a.dim;
      x.k = static_cast<int32_t>(rows);
      x.group = std::max(1, sms / 2 / nt_d);
      x.k_live = a.count;
      LCE_TRY(g_profile.run(kSlotGradWeight, s, [&] { return launch_product<2, 256, 6, true, true, WeightEnd>(e_m, h_n, x, end, s); }),
              "k_lce_grad_weight");
    }
  }
  LCE_TRY(g_profile.run(kSlotLoss, s, [&] { return launch_early(k_lce_loss, dim3(1), 1024, s, a); }), "k_lce_loss");
  return ADAF_OK;
}

void linear_ce_debug_stall_copies(int32_t on) { t_stall = on != 0; }

adaf_status linear_ce_profile_enable(int32_t on) {
  g_profile.on = on != 0;
  return ADAF_OK;
}
adaf_status linear_ce_profile_read(double* ms, int64_t* launches, int32_t nk) {
  const cudaError_t e = g_profile.read(ms, launches, nk);
  return e == cudaSuccess ? ADAF_OK : cuda_fail(e, "profile event");
}
int32_t linear_ce_num_kernels(void) { return kNumKernels; }
const char* linear_ce_kernel_name(int32_t k) { return k >= 0 && k < kNumKernels ? kKernelNames[k] : ""; }

}  // extern "C"
