// Losses over a vocabulary for sm_103a: the C ABI of include/losses.h.
//
// Every operator is a pass over the rows of the logits x[token, vocab] with a
// softmax in it.  A row is reduced to m = max x and s = sum exp((x - m) / T),
// a few scalars follow from those (the token's loss and its derivative), and
// the gradient row is a multiple of exp((x - m) / T) plus a correction at the
// target or at the teacher's entries.
//
//   k_loss_count    number of counted tokens, the denominator of the mean
//   k_loss_row      one row: m, s, the operator's scalars, the gradient row
//   k_loss_short    the same where a few warps keep a row
//   k_loss_forward  m, s and the target's log-probability of a row
//   k_loss_grad     gradient rows from kept m, s and the tokens' coefficients
//   k_loss_pair     a pair's sums over tokens, its loss and its coefficients
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "adafactor_internal.h"
#include "losses.h"

namespace {

constexpr int kMaxWarps = 8;       // of a CTA of k_loss_row that sum
// Lists of so many entries are made by two warps of a CTA in turn.  By one, two
// warps 4096 rows of 128256 bf16 values take, with 64 entries 420, 428 us, 256
// 517, 509, 320 598, 551, 500 803, 662, 1000 1412, 957; rows of 32000 with 256
// 150, 150 us, 384 181, 169.
constexpr int kTwoListers = 320;
constexpr int kGradThreads = 256;
constexpr int kPairThreads = 256;
constexpr int kCountThreads = 1024;
constexpr int kGradVecs = 8;       // vectors of a thread of k_loss_grad
constexpr int kMaxCluster = 8;
constexpr int kKeep = 4;           // chunks of a row that a warp keeps
constexpr int kNoValue = -(1 << 30);  // a target that no value of a row is
constexpr float kLn2 = 0.6931471805599453f;
constexpr int64_t kMaxVocab = int64_t{1} << 21;
constexpr int64_t kMaxTokens = int64_t{1} << 30;

__host__ __device__ constexpr int div_up(int x, int y) { return (x + y - 1) / y; }

enum Op : int { kLogprobs, kPolicy, kDistill };

// ---- sums over tokens ------------------------------------------------------------
// An fp32 sum that carries what its additions round off: as good as an fp64
// one, whose additions and divisions run at a few per cent of the rate here
// (the kernels that end a call took 14 to 19 us with them, 3 to 5 without).
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
  // Over the lanes of a warp, in a fixed order (equal in all lanes).
  __device__ __forceinline__ void over_warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Sum p;
      p.s = __shfl_xor_sync(0xffffffffu, s, o);
      p.rest = __shfl_xor_sync(0xffffffffu, rest, o);
      add(p);
    }
  }
  __device__ __forceinline__ float total() const { return fabsf(s) == INFINITY ? s : s + rest; }
};

// 1 / T as the sum of two fp32 numbers: one alone is off by up to 2^-24 of it, and
// every ln q would lean by that times z[y] - max z the same way, which sums over
// tokens collect.  Both are positive, so that an infinity stays one.
//
// log2(e) / T of the terms is one number.  For it the mean of ln q is off by up to
// 4e-7 (over 48 temperatures by 1e-7, as in fp32 torch operations), at T = 1 by
// 3e-8 to 7e-8, where the exponential's own mean error of -5e-8 goes the other
// way; a ln q is rounded to 5e-7.  A second multiply-add a term leaves a fifth of
// it over the temperatures, twice as much at T = 1, and costs the policy loss 2.5 %.
struct PerT {
  float hi, lo;
};
__device__ __forceinline__ float over_t(float v, const PerT& t) { return fmaf(v, t.hi, v * t.lo); }

struct Rows {
  const void* p;
  int64_t sb, ss;
};

// Arguments of every kernel of this file.
struct LossArgs {
  const void* x;
  void* g;                        // NULL: no gradient
  int64_t xsb, xss, gsb, gss;
  uintptr_t x_begin, x_end;       // the bytes from the logits' first value to their last
  int32_t seq, tokens, vocab;
  float c, inv_t, gscale;         // log2(e) / T, 1 / T, scale of the gradient
  PerT per_t;
  Rows y;
  int32_t ydt;
  int64_t ignore;
  float* loss;
  float* logp;
  float* token_loss;
  float2* stats;                  // [tokens]: m, s
  int* count;                     // counted tokens; NULL: k_loss_row counts them itself
  Sum* part;                      // [clusters]: sum of w l, or of l
  unsigned* ticket;
  int32_t vecs_per_cta;           // k_loss_row, k_loss_forward: vectors of a row for a CTA
  int32_t slots;                  // k_loss_row: places of a CTA's ring, a round each
  int32_t stall;                  // k_loss_row: make no copies (a test)
  int32_t tiles;                  // k_loss_grad: CTAs of a row
  // policy
  Rows adv, old, ref, weights;
  float lo, hi, kl;
  // backward and preference
  Rows dlogp;
  const float* coef;              // [tokens]
  float* coef_out;
  const void* offsets;
  int32_t odt, kind, average;
  int64_t pairs;
  float beta, smooth, margin;
  float* pair_loss;
  float* rewards;
  float* pair_part;               // [pairs]
  // distill
  const void* ids;
  const void* tv;
  int32_t idt, tdt, top_k;
  int64_t isb, iss, tsb, tss;
  Rows lse, mask;
};

// ---- loads -------------------------------------------------------------------
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float& o, float v) { o = v; }
__device__ __forceinline__ void narrow(__nv_bfloat16& o, float v) { o = __float2bfloat16_rn(v); }

__device__ __forceinline__ int64_t load_index(const void* p, int dt, int64_t e) {
  return dt == LOSS_INT64 ? static_cast<const int64_t*>(p)[e] : static_cast<const int32_t*>(p)[e];
}
__device__ __forceinline__ float row_value(const Rows& r, int b, int s) {
  return static_cast<const float*>(r.p)[b * r.sb + s * r.ss];
}
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ bool counted(const LossArgs& a, int op, int b, int s) {
  if (op == kDistill)
    return a.mask.p == nullptr || static_cast<const uint8_t*>(a.mask.p)[b * a.mask.sb + s * a.mask.ss] != 0;
  return load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss) != a.ignore;
}

// ---- terms -----------------------------------------------------------------------
// The terms of a sum with the largest value m are 2^(x c - R), c = log2(e) / T
// and R = m c rounded: one fused multiply-add and one exponential each.  What R
// is off m c by, residue(), is put right where parts of other m are brought
// together and where ln s leaves the kernel.  Where R is so large that the
// residue is no longer small (large logits or low temperatures; masks at the
// type's lowest value, where R is not even finite) the exponent is (x - m) c, in
// two roundings.  A part of -inf alone has terms 0 with R = 0.
struct Ref {
  float m, R;
  __device__ __forceinline__ Ref(float m_, float c) {
    m = m_;
    R = m_ == -INFINITY ? 0.f : __fmul_rn(m_, c);
  }
  __device__ __forceinline__ bool far() const { return fabsf(R) > kFar; }
  __device__ __forceinline__ float exponent(float x, float c) const { return far() ? (x - m) * c : fmaf(x, c, -R); }
  // m c - R
  __device__ __forceinline__ float residue(float c) const { return far() || m == -INFINITY ? 0.f : fmaf(m, c, -R); }
  // What the sum of a part with the largest value m2 <= m is multiplied by.
  __device__ __forceinline__ float factor(float m2, float c) const {
    const float R2 = __fmul_rn(m2, c);
    if (!far() && (R2 >= -kFar || R2 < R - 512.f)) return ex2(__fsub_rn(R2, R));  // (0 where the part is far below)
    return far_factor(m2, m, R, c);
  }
  static __device__ __noinline__ float far_factor(float m2, float m, float R, float c) {
    const float R2 = m2 == -INFINITY ? 0.f : __fmul_rn(m2, c);
    const float off = fabsf(R) > kFar ? 0.f : fmaf(m, c, -R);
    const float off2 = fabsf(R2) > kFar || m2 == -INFINITY ? 0.f : fmaf(m2, c, -R2);
    return ex2((m2 - m) * c + off - off2);
  }
  static constexpr float kFar = 65536.f;
};

// ---- vectors of a row ----------------------------------------------------------
// A row is read as aligned 16-byte vectors.  Vector i of a row that starts
// `lead` values after a 16-byte boundary holds its values i kN - lead ..  The
// first and the last may hold bytes that are not the row's; -inf stands for
// their values.
template <typename T> constexpr int kN = 16 / static_cast<int>(sizeof(T));
template <typename T> constexpr uint32_t kNegInf = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
constexpr int kBatch = 4;           // vectors of a lane in a warp's chunk of a row
constexpr int kForwardBatch = 4;    // vectors in flight in k_loss_forward, twice

template <typename T>
struct Row {
  uintptr_t base;     // the first vector
  int lead, n, vecs;  // values before the row in its first vector, values, vectors
  __device__ __forceinline__ Row(const T* p, int vocab) : n(vocab) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    base = at & ~uintptr_t{15};
    lead = static_cast<int>((at & 15) / sizeof(T));
    vecs = (lead + n + kN<T> - 1) / kN<T>;
  }
  __device__ __forceinline__ const T* value(int j) const { return reinterpret_cast<const T*>(base) + lead + j; }
  __device__ __forceinline__ bool ragged(int i) const { return (i == 0 && lead != 0) || (i == vecs - 1 && i * kN<T> + kN<T> > lead + n); }
  // Vectors [first_whole, past_whole) hold nothing but the row's values.
  __device__ __forceinline__ int first_whole() const { return lead != 0; }
  __device__ __forceinline__ int past_whole() const { return (lead + n) / kN<T>; }
};

__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

// Value j of a vector, replaced.
template <typename T>
__device__ __forceinline__ void put(uint4& w, int j, uint32_t bits) {
  uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (sizeof(T) == 4) {
      if (j == k) q[k] = bits;
    } else {
      if (j == 2 * k) q[k] = (q[k] & 0xffff0000u) | bits;
      if (j == 2 * k + 1) q[k] = (q[k] & 0xffffu) | (bits << 16);
    }
  }
  w = make_uint4(q[0], q[1], q[2], q[3]);
}
// Value j of a vector.
template <typename T>
__device__ __forceinline__ float get(const uint4& w, int j) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kN<T>; ++k)
    if (j == k) v = sizeof(T) == 4 ? __uint_as_float(q[k & 3]) : __uint_as_float(k & 1 ? q[k >> 1 & 3] & 0xffff0000u : q[k >> 1 & 3] << 16);
  return v;
}
// -inf outside the row.
template <typename T>
__device__ __forceinline__ void trim(uint4& w, const Row<T>& r, int i) {
#pragma unroll
  for (int j = 0; j < kN<T>; ++j) {
    const int e = i * kN<T> - r.lead + j;
    if (e < 0 || e >= r.n) put<T>(w, j, kNegInf<T> & (sizeof(T) == 2 ? 0xffffu : 0xffffffffu));
  }
}
// -inf for the values whose bit is set.
template <typename T>
__device__ __forceinline__ void leave_out(uint4& w, uint32_t on) {
#pragma unroll
  for (int j = 0; j < kN<T>; ++j)
    if (on >> j & 1) put<T>(w, j, kNegInf<T> & (sizeof(T) == 2 ? 0xffffu : 0xffffffffu));
}
__device__ __forceinline__ uint4 no_values(uint32_t neg_inf) { return make_uint4(neg_inf, neg_inf, neg_inf, neg_inf); }

// Vector i < last of the row from memory.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const Row<T>& r, int i, int last) {
  uint4 w = no_values(kNegInf<T>);
  if (i < last) {
    if (!r.ragged(i)) {
      w = __ldcs(reinterpret_cast<const uint4*>(r.base) + i);
    } else {
#pragma unroll
      for (int j = 0; j < kN<T>; ++j) {
        const int e = i * kN<T> - r.lead + j;
        if (e >= 0 && e < r.n) put<T>(w, j, bits_of(*r.value(e)));
      }
    }
  }
  return w;
}
// A warp's batch: vectors i + k NT of lane i - first.  Whether all of them lie
// in [lo, hi): then nothing is looked at vector by vector.
template <int NT, int N = kBatch>
__device__ __forceinline__ bool batch_in(int first, int lo, int hi) { return first >= lo && first + 31 + (N - 1) * NT < hi; }
template <typename T, int NT, int N>
__device__ __forceinline__ void load_batch(uint4 (&w)[N], const Row<T>& r, int i, int last) {
  if (batch_in<NT, N>(i - (threadIdx.x & 31), r.first_whole(), min(r.past_whole(), last))) {
    const uint4* p = reinterpret_cast<const uint4*>(r.base) + i;
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = __ldcs(p + k * NT);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = load_vec(r, i + k * NT, last);
  }
}

__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }
// Two values of a vector.
template <typename T>
__device__ __forceinline__ float2 pair_at(const uint4& w, int j) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
  if (sizeof(T) == 4) return make_float2(__uint_as_float(q[(2 * j) & 3]), __uint_as_float(q[(2 * j + 1) & 3]));
  return make_float2(__uint_as_float(q[j] << 16), __uint_as_float(q[j] & 0xffff0000u));
}
template <bool FAR>
__device__ __forceinline__ float2 terms(float2 x, const Ref& ref, float c) {
  const float2 z = FAR ? __fmul2_rn(__fadd2_rn(x, twice(-ref.m)), twice(c)) : __ffma2_rn(x, twice(c), twice(-ref.R));
  return make_float2(ex2(z.x), ex2(z.y));
}

// Largest value of a batch (NaN is left out: it shows in the sum).
template <typename T, int N>
__device__ __forceinline__ float batch_max(const uint4 (&w)[N]) {
  if (sizeof(T) == 2) {
    __nv_bfloat162 a;
    memcpy(&a, &w[0].x, 4);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t q[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        __nv_bfloat162 b;
        memcpy(&b, &q[t], 4);
        a = __hmax2(a, b);
      }
    }
    return fmaxf(__low2float(a), __high2float(a));
  }
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; ++k)
    m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(w[k].x), __uint_as_float(w[k].y)),
                       fmaxf(__uint_as_float(w[k].z), __uint_as_float(w[k].w))));
  return m;
}

// A thread's part of a row: the largest value and the sum of the terms.
template <typename T>
struct Part {
  float m = -INFINITY, s = 0.f;
  template <bool FAR, int N>
  __device__ __forceinline__ void sum(const uint4 (&w)[N], const Ref& ref, float c) {
    float2 acc = make_float2(0.f, 0.f), acc2 = acc;
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
      for (int j = 0; j < kN<T> / 2; j += 2) {
        acc = __fadd2_rn(acc, terms<FAR>(pair_at<T>(w[k], j), ref, c));
        acc2 = __fadd2_rn(acc2, terms<FAR>(pair_at<T>(w[k], j + 1), ref, c));
      }
    }
    s += (acc.x + acc.y) + (acc2.x + acc2.y);
  }
  template <int N>
  __device__ __forceinline__ void add(const uint4 (&w)[N], float c) {
    const float m2 = batch_max<T, N>(w);
    if (m2 > m) {
      s *= Ref(m2, c).factor(m, c);
      m = m2;
    }
    const Ref ref(m, c);
    if (ref.far()) sum<true>(w, ref, c);
    else sum<false>(w, ref, c);
  }
};

// Stores of a gradient row, from vectors in the logits' phase.
template <typename T>
struct GradRow {
  T* g;
  int n, lead, shift;  // values before the row in its first 16 bytes; that minus the logits' lead, mod kN
  __device__ __forceinline__ GradRow(T* p, int vocab, int x_lead) : g(p), n(vocab) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    shift = (lead - x_lead) & (kN<T> - 1);
  }
  __device__ __forceinline__ void value(const uint4& w, int e0, int j) const {
    const int e = e0 + j;
    if (e < 0 || e >= n) return;
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
    if (sizeof(T) == 4) {
      reinterpret_cast<uint32_t*>(g)[e] = q[j & 3];
    } else {
      reinterpret_cast<uint16_t*>(g)[e] = static_cast<uint16_t>(q[(j >> 1) & 3] >> (16 * (j & 1)));
    }
  }
  // Vector of values e0 .. e0 + kN of the row; `in` false: not this thread's.
  // Every lane of the warp calls, lanes holding consecutive vectors.
  __device__ __forceinline__ void store(const uint4& w, int e0, bool in) const {
    if (shift == 0) {
      if (!in) return;
      if (e0 >= 0 && e0 + kN<T> <= n) {
        __stcs(reinterpret_cast<uint4*>(g + e0), w);
      } else {
#pragma unroll
        for (int j = 0; j < kN<T>; ++j) value(w, e0, j);
      }
      return;
    }
    // The gradient's aligned vectors straddle two of these: each lane joins
    // its tail to the head of the next lane's and stores that; a warp's first
    // head and last tail go value by value.
    const int lane = threadIdx.x & 31, tail = kN<T> - shift;  // first value of the aligned vector that starts here
    uint32_t q[8] = {w.x, w.y, w.z, w.w, 0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < 4; ++t) q[4 + t] = __shfl_down_sync(0xffffffffu, q[t], 1);
    const bool next_in = __shfl_down_sync(0xffffffffu, static_cast<int>(in), 1) != 0;
    const bool joint = in && next_in && lane < 31 && e0 + tail >= 0 && e0 + tail + kN<T> <= n;
    const bool before = __shfl_up_sync(0xffffffffu, static_cast<int>(joint), 1) != 0 && lane > 0;
    if (joint) {
      const int bytes = tail * static_cast<int>(sizeof(T));
      if (bytes & 8) {
#pragma unroll
        for (int t = 0; t < 6; ++t) q[t] = q[t + 2];
      }
      if (bytes & 4) {
#pragma unroll
        for (int t = 0; t < 5; ++t) q[t] = q[t + 1];
      }
      const uint32_t by = 8 * (bytes & 3);
      const uint4 o = make_uint4(__funnelshift_r(q[0], q[1], by), __funnelshift_r(q[1], q[2], by),
                                 __funnelshift_r(q[2], q[3], by), __funnelshift_r(q[3], q[4], by));
      __stcs(reinterpret_cast<uint4*>(g + e0 + tail), o);
    }
    if (in) {
#pragma unroll
      for (int j = 0; j < kN<T>; ++j) {
        if (j < tail ? !before : !joint) value(w, e0, j);
      }
    }
  }
  // The part of the row that CTA `rank` of `ranks` has, as zeros.
  __device__ __forceinline__ void zero(int rank, int ranks, int threads, int thread) const {
    const int vecs = (lead + n + kN<T> - 1) / kN<T>, per = (vecs + ranks - 1) / ranks;
    const int last = min(vecs, (rank + 1) * per);
    for (int i = rank * per + thread; i < last; i += threads) {
      const int e0 = i * kN<T> - lead;
      if (e0 >= 0 && e0 + kN<T> <= n) {
        __stcs(reinterpret_cast<uint4*>(g + e0), make_uint4(0, 0, 0, 0));
      } else {
#pragma unroll
        for (int j = 0; j < kN<T>; ++j) value(make_uint4(0, 0, 0, 0), e0, j);
      }
    }
  }
};

__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  uint32_t r;
  memcpy(&r, &b, 4);
  return r;
}
// scale 2^(x c - R) of a vector, rounded to its type.
template <typename T, bool FAR>
__device__ __forceinline__ uint4 scaled_terms(const uint4& w, const Ref& ref, float c, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < kN<T> / 2; ++j) {
    const float2 v = __fmul2_rn(terms<FAR>(pair_at<T>(w, j), ref, c), twice(scale));
    if (sizeof(T) == 4) {
      o[(2 * j) & 3] = __float_as_uint(v.x);
      o[(2 * j + 1) & 3] = __float_as_uint(v.y);
    } else {
      o[j] = pack2(v);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
template <typename T>
__device__ __forceinline__ uint32_t rounded_bits(float v) {
  T t;
  narrow(t, v);
  return bits_of(t);
}
// A vector of the gradient from the logits' vector i: scale 2^(x c - R), and
// at value y that plus `more`.  Every lane of the warp calls.
template <typename T>
__device__ __forceinline__ void store_grad(const uint4& w, const Row<T>& r, const GradRow<T>& g, int i, bool in, const Ref& ref,
                                           float c, float scale, int y, float more) {
  const int e0 = i * kN<T> - r.lead;
  uint4 o = ref.far() ? scaled_terms<T, true>(w, ref, c, scale) : scaled_terms<T, false>(w, ref, c, scale);
  const unsigned j = static_cast<unsigned>(y - e0);
  if (j < static_cast<unsigned>(kN<T>))
    put<T>(o, static_cast<int>(j), rounded_bits<T>(scale * ex2(ref.exponent(get<T>(w, static_cast<int>(j)), c)) + more));
  g.store(o, e0, in);
}

// The gradient's vectors of a batch, of vectors i + k NT < last; every lane of
// the warp calls.  `plain`: whole vectors in the logits' phase without the
// target.
template <typename T, int NT, int N>
__device__ __forceinline__ void store_batch(const uint4 (&w)[N], const Row<T>& r, const GradRow<T>& g, int i, int last,
                                            bool plain, const Ref& ref, float c, float scale, int y, int y_vec, float more) {
  uint4* p = reinterpret_cast<uint4*>(g.g + (i * kN<T> - r.lead));
  if (plain) {
#pragma unroll
    for (int k = 0; k < N; ++k) __stcs(p + k * NT, scaled_terms<T, false>(w[k], ref, c, scale));
    return;
  }
  const int first = i - (threadIdx.x & 31), lo = r.first_whole(), hi = min(r.past_whole(), last);
  const bool near = g.shift == 0 && !ref.far();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int f = first + k * NT;
    if (near && batch_in<NT, 1>(f, lo, hi) && static_cast<unsigned>(y_vec - f) >= 32u)
      __stcs(p + k * NT, scaled_terms<T, false>(w[k], ref, c, scale));
    else if (f < last)
      store_grad(w[k], r, g, i + k * NT, i + k * NT < last, ref, c, scale, y, more);
  }
}

// ---- clusters --------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_remote(const float4* mine, uint32_t rank, float4 v) {
  const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(there), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
// Waits for the kernel before this one (launched so that they overlap).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// ---- counted tokens ------------------------------------------------------------
// Also clears the ticket of the sum over tokens.
__global__ void __launch_bounds__(kCountThreads) k_loss_count(const __grid_constant__ LossArgs a, int op) {
  __shared__ int parts[kCountThreads / 32];
  let_next_start();
  if (threadIdx.x == 0) *a.ticket = 0;
  int n = 0;
#pragma unroll 8
  for (uint32_t t = threadIdx.x; t < static_cast<uint32_t>(a.tokens); t += kCountThreads)
    n += counted(a, op, static_cast<int>(t / static_cast<uint32_t>(a.seq)), static_cast<int>(t % static_cast<uint32_t>(a.seq)));
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x < 32) {
    n = __reduce_add_sync(0xffffffffu, parts[threadIdx.x]);
    if (threadIdx.x == 0) {
      *a.count = n;
      if (a.tokens == 0) *a.loss = 0.f;
    }
  }
}

// ---- the operators' scalars -----------------------------------------------------
struct PolicyIn {
  float adv, old, ref;
};
// Loss of a token and its derivative with respect to logp.
struct Token {
  float loss, d;
};
__device__ __forceinline__ Token policy_token(const LossArgs& a, float logp, const PolicyIn& in) {
  // Without old_logp the ratio is 1, for a word of probability 0 too (NaN stays).
  const float r = a.old.p != nullptr ? expf(logp - in.old) : isnan(logp) ? logp : 1.f;
  const float raw = r * in.adv;
  const float cut = fminf(fmaxf(r, a.lo), a.hi) * in.adv;
  Token t;
  const bool free = raw <= cut || isnan(raw);
  t.loss = free ? -raw : -cut;
  t.d = free ? -raw : 0.f;
  if (a.kl != 0.f) {
    const float far = in.ref - logp;
    const float e = expm1f(far);
    t.loss += a.kl * (far == INFINITY ? far : e - far);  // (a word of probability 0: not inf - inf)
    t.d -= a.kl * e;
  }
  return t;
}

// ---- barriers and copies in shared memory -----------------------------------------
__device__ __forceinline__ uint32_t shared_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void init_barrier(uint64_t* bar, int arrivals) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_at(bar)), "r"(arrivals) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_at(bar)) : "memory");
}
// A bulk copy, and its bytes to be counted by `bar`.  `stall`: they are expected
// and the copy not made (a test of the waits).
__device__ __forceinline__ void copy_bulk(void* to, const void* from, uint32_t bytes, uint64_t* bar, bool stall) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_at(bar)), "r"(bytes) : "memory");
  if (bytes != 0 && !stall)
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(shared_at(to)),
                 "l"(from), "r"(bytes), "r"(shared_at(bar))
                 : "memory");
}
// Orders what a thread has read (or has waited for others to read) before a bulk
// copy that it makes to the same place: barriers alone order them with ordinary
// stores, not with a copy, which goes by another way.
__device__ __forceinline__ void reads_before_copies() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(shared_at(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}
// Waits for a phase; false, in the whole warp, after meo::kWaitCycles.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
  bool ok = phase_done(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    while (!(ok = phase_done(bar, parity)))
      if (clock64() - t0 > meo::kWaitCycles) break;
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_at(bar)), "r"(bytes) : "memory");
}
// 16 bytes to the same place in another CTA of the cluster, counted by its
// barrier there.  Unlike the cluster's own barrier this waits for no store to
// global memory before it.
__device__ __forceinline__ void send(const float4* mine, uint32_t rank, float4 v, uint64_t* bar) {
  uint32_t to, there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(shared_at(mine)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(shared_at(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)), "r"(there)
               : "memory");
}
constexpr int kChunk = 32 * kBatch;  // vectors of a warp's batch: consecutive ones, lane by lane

// A teacher's list, as one warp makes it for a row.
using Bits = uint32_t;
static_assert(sizeof(Bits) == kBatch, "a byte for each vector of a lane: list_bytes() counts on it");
struct List {
  Bits* bits;      // [chunks of the CTA's part][lanes]: a byte a vector, a bit a value
  int32_t* id;     // [top_k]
  float* p;        // [top_k]: the teacher's probabilities
  float* x;        // [top_k]: the logits (of all in rank 0, of the CTA's own elsewhere)
  float* head;     // sum p, rest, NaN where the list is bad (else 0); of the CTA's own: the largest of x, sum of terms
};
__host__ __device__ constexpr int list_bytes(int slice, int top_k) {
  return (slice + 15) / 16 * 16 + 12 * ((top_k + 3) / 4 * 4) + 32;
}
__device__ __forceinline__ List list_at(unsigned char* p, int slice, int top_k) {
  List l;
  const int kpad = (top_k + 3) / 4 * 4;
  l.bits = reinterpret_cast<Bits*>(p);
  l.id = reinterpret_cast<int32_t*>(p + (slice + 15) / 16 * 16);
  l.p = reinterpret_cast<float*>(l.id + kpad);
  l.x = l.p + kpad;
  l.head = l.x + kpad;
  return l;
}

template <typename T>
__device__ __forceinline__ void make_list(const LossArgs& a, const List& l, const Row<T>& r, int b, int s, int v0, int v1,
                                          int slice, bool all) {
  const int lane = threadIdx.x & 31;
  const float lse = a.lse.p == nullptr ? 0.f : row_value(a.lse, b, s);
  const int64_t ids = b * a.isb + s * a.iss, values = b * a.tsb + s * a.tss;
  for (int i = lane; i < slice / 16; i += 32) reinterpret_cast<uint4*>(l.bits)[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();
  float top = -INFINITY, most = -INFINITY;
  int entries = 0, wrong = 0;
  // Four entries of a lane at a time: their loads, and then those of their
  // logits, are under way together.
  constexpr int kAtOnce = 4;
  for (int k0 = lane; k0 < a.top_k; k0 += 32 * kAtOnce) {
    int64_t i[kAtOnce];
    float v[kAtOnce], x[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int k = k0 + 32 * u;
      i[u] = -1;
      v[u] = -INFINITY;
      if (k < a.top_k) {
        i[u] = load_index(a.ids, a.idt, ids + k);
        v[u] = a.tdt == ADAF_BFLOAT16 ? widen(static_cast<const __nv_bfloat16*>(a.tv)[values + k])
                                      : static_cast<const float*>(a.tv)[values + k];
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      x[u] = 0.f;
      if (i[u] >= 0 && i[u] < a.vocab) {
        const int at = (static_cast<int>(i[u]) + r.lead) / kN<T> - v0;
        if (all || (at >= 0 && at < v1 - v0)) x[u] = widen(*r.value(static_cast<int>(i[u])));
      } else {
        wrong |= i[u] != -1;
        i[u] = -1;
        v[u] = -INFINITY;
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int k = k0 + 32 * u;
      if (k >= a.top_k) continue;
      if (i[u] >= 0) {
        ++entries;
        top = fmaxf(top, v[u]);
        const int e = static_cast<int>(i[u]) + r.lead, at = e / kN<T> - v0;
        if (at >= 0 && at < v1 - v0) {
          most = fmaxf(most, x[u]);
          const uint32_t bit = 1u << (at % kChunk / 32 * 8 + e % kN<T>);
          if (atomicOr(l.bits + at / kChunk * 32 + at % 32, bit) & bit) wrong = 1;
        }
      }
      l.id[k] = static_cast<int>(i[u]);
      l.p[k] = v[u];
      l.x[k] = x[u];
    }
  }
  top = warp_max(top);
  most = warp_max(most);
  entries = __reduce_add_sync(0xffffffffu, entries);
  const bool bad = __any_sync(0xffffffffu, wrong);
  const float sh = top == -INFINITY ? 0.f : top;
  const Ref ref(most, a.c);
  float sum = 0.f, own = 0.f;
  for (int k = lane; k < a.top_k; k += 32) {
    const int at = (l.id[k] + r.lead) / kN<T> - v0;
    if (l.id[k] >= 0 && at >= 0 && at < v1 - v0) own += ex2(ref.exponent(l.x[k], a.c));
    // renormalised: exp((t - max) / T) / sum; with lse: exp(t / T - lse)
    const float p = l.id[k] < 0 ? 0.f : a.lse.p == nullptr ? ex2((l.p[k] - sh) * a.c) : expf(over_t(l.p[k], a.per_t) - lse);
    l.p[k] = p;
    sum += p;
  }
  sum = warp_sum(sum);
  own = warp_sum(own);
  float sum_p = sum, rest = 0.f;
  if (a.lse.p == nullptr) {
    sum_p = sum == 0.f ? 0.f : sum == sum ? 1.f : sum;
    const float by = sum == 0.f ? 0.f : 1.f / sum;
    for (int k = lane; k < a.top_k; k += 32) l.p[k] *= by;
  } else if (sum != sum) {
    rest = sum;
  } else if (entries < a.vocab) {
    rest = fmaxf(0.f, 1.f - sum);
  }
  if (lane == 0) {
    l.head[0] = sum_p;
    l.head[1] = rest;
    l.head[2] = bad ? NAN : 0.f;
    l.head[3] = most;
    l.head[4] = own;
  }
}

// What the gradient needs: scale 2^(x c - R) with R of m, `more` at the target;
// for a list, with R of m_on, lead (on 2^(x c - R) - p) at its words.
struct RowScale {
  float m, scale, more, m_on, lead, on;
};
// A token's own values.
struct Values {
  int row, y;
  bool live;
  PolicyIn in;
  float weight, x_at;
};
// A row with a list has two sums.  That of the words not listed is relative to
// the largest of them: their shares among themselves are needed too, and beside
// the listed words they may all be too small for fp32 (logits 88 T below).
// (Rows that need no such care on a path of their own: 415 us for 417 of 4096 x
// 128256 bf16 values, with one sum and no care 408.)
struct ListSums {
  Ref off, whole;              // of the words not listed, of all
  float factor, off_sum, sum;  // from `off` to `whole`; the two sums
};
// The row's scalars from its sum.  The policy's loss is done with them.
__device__ __forceinline__ RowScale policy_scale(const LossArgs& a, const Values& v, const Ref& ref, float sum, float wrong, float w,
                                                 float& logp, float& loss) {
  RowScale out{ref.m, 0.f, 0.f, 0.f, 0.f, 0.f};
  logp = v.y < 0 ? NAN : over_t(v.x_at - ref.m, a.per_t) - logf(sum) + ref.residue(a.c) * kLn2 + wrong;
  const Token t = policy_token(a, logp, v.in);
  loss = t.loss;
  out.more = w * a.gscale * a.inv_t * t.d;
  out.scale = __fdividef(-out.more, sum);
  return out;
}
// Off the list q (P + u) - u share, share = q / (sum of such q); on it q (P + u) - p.
__device__ __forceinline__ RowScale list_scale(const LossArgs& a, const List& list, const ListSums& s, float wrong, float w) {
  RowScale out{s.off.m, 0.f, 0.f, s.whole.m, 0.f, 0.f};
  const float rest = list.head[1];
  out.lead = w * a.gscale / a.inv_t + wrong;
  out.on = (list.head[0] + rest) / s.sum;
  out.scale = out.lead * (out.on * s.factor - (rest > 0.f ? rest / s.off_sum : 0.f));
  return out;
}
// By a whole warp.
__device__ __forceinline__ float list_loss(const LossArgs& a, const List& list, const ListSums& s, float wrong) {
  const Ref& ref = s.whole;
  const float log_s = logf(s.sum), rest = list.head[1], d = ref.residue(a.c) * kLn2;
  float loss = 0.f;
  for (int k = threadIdx.x & 31; k < a.top_k; k += 32) {
    const float p = list.p[k];
    if (p != 0.f) loss += p * (logf(p) - (over_t(list.x[k] - ref.m, a.per_t) + d - log_s));
  }
  loss = warp_sum(loss);
  if (rest > 0.f) {
    // The unlisted words' part of the row: one logarithm where fp32 holds it
    // (the sum of four is rounded at their size, which showed in the loss).
    const float part = s.off_sum * s.factor / s.sum;
    loss += rest * (logf(rest) - (part > 1e-30f ? logf(part) : over_t(s.off.m - ref.m, a.per_t) +
                                                                 (logf(s.off_sum) - s.off.residue(a.c) * kLn2) - (log_s - d)));
  }
  return loss / (a.inv_t * a.inv_t) + wrong;
}
// The loss from `n` parts, by the warp that adds the last: in a fixed order.
__device__ __forceinline__ void add_part(const LossArgs& a, int part, int n, const Sum& share, int n_counted) {
  const int lane = threadIdx.x & 31;
  int last = 0;
  if (lane == 0) {
    a.part[part] = share;
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == static_cast<unsigned>(n - 1);
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  Sum sum;
  for (int k = lane; k < n; k += 32) {
    const float2 o = __ldcg(reinterpret_cast<const float2*>(a.part) + k);
    Sum p;
    p.s = o.x;
    p.rest = o.y;
    sum.add(p);
  }
  sum.over_warp();
  if (lane == 0) {
    const float c = a.weights.p == nullptr ? static_cast<float>(n_counted) : 1.f;
    *a.loss = c > 0.f ? sum.total() / c : 0.f;
    if (a.count == nullptr) *a.ticket = 0;  // for the stream's next call
  }
}
// Counted tokens, by a warp that has them from no other kernel.
__device__ __forceinline__ int count_tokens(const LossArgs& a, int op) {
  int n = 0;
#pragma unroll 4
  for (int t = threadIdx.x & 31; t < a.tokens; t += 32) n += counted(a, op, t / a.seq, t % a.seq);
  return __reduce_add_sync(0xffffffffu, n);
}

// ---- rows: the sum and the gradient in one read ---------------------------------
// A row of the walk, as the managing warp tells it to the others.
struct RowInfo {
  uintptr_t x, g;           // the first value of the logits' and of the gradient's row
  int32_t live;             // 0: there is no further row
  int32_t y;                // the target, kNoValue without one
  int32_t ignored, n_ignored;  // rows before it (every `stride`) whose gradient is 0
};
// The rows first, first + stride, .. of a cluster, 32 at a time: a lane looks
// one up, and its per-token values with it, so that none of them is waited for
// row by row.
template <typename T, int OP>
struct Walk {
  const LossArgs& a;
  int stride, base, off = 32;      // row of lane 0 one window back; next lane to look at
  unsigned live = 0, valid = 0;
  int64_t target = 0;
  PolicyIn in{0.f, 0.f, 0.f};
  float weight = 0.f, x_at = 0.f;
  __device__ __forceinline__ Walk(const LossArgs& args, int first, int step) : a(args), stride(step), base(first - 32 * step) {}
  // `values`: look the token's values up too, and write the results of ignored tokens (`writes`)
  __device__ __forceinline__ void window(bool values, bool writes) {
    const int lane = threadIdx.x & 31;
    base += 32 * stride;
    off = 0;
    const int64_t row64 = base + static_cast<int64_t>(lane) * stride;
    const bool is = row64 < a.tokens;
    bool counts = false;
    if (is) {
      const int row = static_cast<int>(row64), b = row / a.seq, s = row % a.seq;
      if (OP == kDistill) {
        counts = counted(a, OP, b, s);
      } else {
        target = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
        counts = target != a.ignore;
      }
      if (values && counts) {
        if (OP == kPolicy) {
          in.adv = row_value(a.adv, b, s);
          if (a.old.p != nullptr) in.old = row_value(a.old, b, s);
          if (a.kl != 0.f) in.ref = row_value(a.ref, b, s);
          if (target >= 0 && target < a.vocab) x_at = widen((static_cast<const T*>(a.x) + b * a.xsb + s * a.xss)[target]);
        }
        if (a.weights.p != nullptr) weight = row_value(a.weights, b, s);
      }
      if (writes && !counts) {
        if (a.logp != nullptr) a.logp[row] = 0.f;
        if (a.token_loss != nullptr) a.token_loss[row] = 0.f;
      }
    }
    valid = __ballot_sync(0xffffffffu, is);
    live = __ballot_sync(0xffffffffu, counts);
  }
  // The lane that has the next counted row, -1 at the end; `ignored`: first and
  // number of the rows passed over.
  __device__ __forceinline__ int next(bool values, bool writes, int& ignored, int& n_ignored) {
    n_ignored = 0;
    while (true) {
      if (off == 32) {
        if (base + 32 * static_cast<int64_t>(stride) >= a.tokens) return -1;
        window(values, writes);
      }
      const unsigned left = live >> off;
      const int skip = left != 0 ? __ffs(static_cast<int>(left)) - 1 : __popc(valid >> off);
      if (skip > 0 && n_ignored == 0) ignored = base + off * stride;
      n_ignored += skip;
      if (left != 0) {
        off += skip + 1;
        return off - 1;
      }
      off = 32;
    }
  }
};

// Clusters of CTAs walk the rows; a CTA has a run of a row's vectors and its
// warps share that in rounds of a chunk each.  One warp copies rounds into a
// ring in shared memory as places come free (bulk copies, so that the next row
// is on its way while this one is worked on).  The warps add up their terms,
// and, when the cluster's parts of the row are together, make the gradient from
// the same copies.  Another warp manages: it looks the rows up ahead of the
// others, joins the parts and works out the row's scalars, so that these cost
// the others nothing (16 warps doing so themselves took 2300 cycles to begin a
// row and 2500 from its sum to its gradient, of 13,500 in all).  For lists
// there are one or two more (LISTERS), which make those up to two rows ahead.
// LONG: rows that no cluster keeps are read twice, from global memory.
//
// Bound by memory where rows are many: 8192 x 128256 bf16 values take 652 us,
// 6.44 TB/s or 0.95 of the copy rate (ring of 6 x 16 KB a CTA, two CTAs an SM,
// four CTAs a row); 3000 x 50256 fp32 195 us, 0.91; 4096 x 32000 bf16 95 us,
// 0.82.  What it took: one CTA of 16 warps an SM 716 us; the parts exchanged
// under the cluster's own barrier, whose release waits for every store before
// it, 748; registers in place of the ring 1075.  With a list of 64 entries 4096
// rows take 418 us, 0.74 (the policy loss 334), with 8 entries 389, with 1000
// 963: reading the listed words' logits and writing their gradients takes
// sectors of their own, and long lists are bound by the warps that make them.
// 100 rows take 23 us, bound by one row's way through the warps (11 us).
template <typename T, int OP, bool LONG, int LISTERS = OP == kDistill ? 1 : 0>
__global__ void __launch_bounds__((kMaxWarps + 2 + LISTERS) * 32, 2)
    k_loss_row(const __grid_constant__ LossArgs a) {
  extern __shared__ __align__(16) unsigned char shared[];
  __shared__ RowInfo info[3];
  __shared__ RowScale scales[2];
  __shared__ uint64_t together[2], info_full[3], scale_full[2], list_full[2], list_free[2], written;
  constexpr bool kLists = OP == kDistill;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = (blockDim.x >> 5) - 2 - LISTERS;  // that sum
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int first = static_cast<int>(blockIdx.x) / ranks, stride = static_cast<int>(gridDim.x) / ranks;
  const int v0 = rank * a.vecs_per_cta, slots = a.slots;
  const int round = warps * kChunk;                                  // vectors
  uint4* const ring = reinterpret_cast<uint4*>(shared);              // [slots][round]
  float4* const parts = reinterpret_cast<float4*>(shared) + slots * round;  // [2][warps of the cluster]
  uint64_t* const full = reinterpret_cast<uint64_t*>(parts + 2 * warps * ranks);  // [slots]
  uint64_t* const empty = full + slots;                              // [slots]
  unsigned char* const lists = reinterpret_cast<unsigned char*>(empty + slots);
  const int slice = a.vecs_per_cta, list_size = list_bytes(slice, a.top_k);
  // Bytes that a row's parts are; the manager expects the next but one row's
  // as soon as a row's are there, and only then its scalars let anybody go on.
  const uint32_t row_bytes = 16 * warps * ranks;
  if (threadIdx.x == 0) {
    for (int k = 0; k < 2; ++k) {
      init_barrier(together + k, ranks > 1 ? 1 : warps);
      if (ranks > 1) expect_bytes(together + k, row_bytes);
      init_barrier(scale_full + k, 1);
      init_barrier(list_full + k, 1);
      init_barrier(list_free + k, warps + 1);
    }
    for (int k = 0; k < 3; ++k) init_barrier(info_full + k, 1);
    init_barrier(&written, warps);
  }
  if (threadIdx.x < slots) {
    init_barrier(full + threadIdx.x, 1);
    init_barrier(empty + threadIdx.x, warps);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();
  if (ranks > 1) {  // shared memory of the others may be written once they have all begun
    cluster_arrive();
    cluster_wait();
  }
  bool dead = false;  // a wait ran out: no more waiting, the loss is NaN
  // The granule of 16 bytes at a row's end may hold bytes of its neighbour; at
  // the tensor's own ends it may reach outside, and is then read value by value.
  auto copied_from = [&](const Row<T>& r) { return r.base < a.x_begin ? 1 : 0; };
  auto copied_to = [&](const Row<T>& r) { return r.base + 16 * static_cast<int64_t>(r.vecs) > a.x_end ? r.vecs - 1 : r.vecs; };

  if (warp == warps + 1) {
    // The warp that copies.
    if (!LONG) {
      Walk<T, OP> walk(a, first, stride);
      int place = 0, none, n_none, copies = 0;
      uint32_t parity = 1;  // of the place's last reading; the first waits return at once
      for (int at = walk.next(false, false, none, n_none); at >= 0 && !dead; at = walk.next(false, false, none, n_none)) {
        const int row = walk.base + at * stride, b = row / a.seq, s = row % a.seq;
        const Row<T> r(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss, a.vocab);
        const int v1 = min(r.vecs, v0 + a.vecs_per_cta), lo = copied_from(r), hi = min(copied_to(r), v1);
        for (int i = v0; i < v1; i += round) {
          if (!wait_phase(empty + place, parity)) {
            dead = true;
            break;
          }
          if (lane == 0) {
            reads_before_copies();
            const int i0 = max(i, lo), n = min(i + round, hi) - i0;
            copy_bulk(ring + place * round + (i0 - i), reinterpret_cast<const uint4*>(r.base) + i0, n > 0 ? 16 * n : 0, full + place,
                      a.stall != 0);
          }
          ++copies;
          if (++place == slots) {
            place = 0;
            parity ^= 1;
          }
        }
      }
      // The last copies land before the CTA's memory is given up.
      for (int k = min(copies, slots); k > 0; --k) {
        if (--place < 0) {
          place = slots - 1;
          parity ^= 1;
        }
        if (!wait_phase(full + place, parity ^ 1)) break;
      }
    }
  } else if (kLists && warp >= warps + 2) {
    // A warp that makes lists, up to two rows ahead: every row's, or of two such
    // warps every other row's.
    Walk<T, OP> walk(a, first, stride);
    int q = 0, none, n_none;
    for (int at = walk.next(false, false, none, n_none); at >= 0; at = walk.next(false, false, none, n_none), ++q) {
      if (LISTERS == 2 && (q & 1) != warp - warps - 2) continue;
      const int row = walk.base + at * stride, b = row / a.seq, s = row % a.seq;
      const Row<T> r(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss, a.vocab);
      if (q >= 2 && !wait_phase(list_free + (q & 1), (q - 2) >> 1 & 1)) break;
      make_list(a, list_at(lists + (q & 1) * list_size, slice, a.top_k), r, b, s, v0, min(r.vecs, v0 + a.vecs_per_cta), slice,
                rank == 0);
      __syncwarp();
      if (lane == 0) arrive(list_full + (q & 1));
    }
  } else if (warp == warps) {
    // The manager.
    Walk<T, OP> walk(a, first, stride);
    int told = 0;
    auto tell_next = [&] {
      RowInfo i;
      Values v;
      int ignored = 0;
      const int at = walk.next(true, rank == 0, ignored, i.n_ignored);
      const int from = max(at, 0);
      v.live = at >= 0;
      v.row = walk.base + from * stride;
      const int64_t target = __shfl_sync(0xffffffffu, walk.target, from);
      v.y = !kLists && target >= 0 && target < a.vocab ? static_cast<int>(target) : kNoValue;
      v.in.adv = __shfl_sync(0xffffffffu, walk.in.adv, from);
      v.in.old = __shfl_sync(0xffffffffu, walk.in.old, from);
      v.in.ref = __shfl_sync(0xffffffffu, walk.in.ref, from);
      v.weight = __shfl_sync(0xffffffffu, walk.weight, from);
      v.x_at = __shfl_sync(0xffffffffu, walk.x_at, from);
      const int b = v.row / a.seq, s = v.row % a.seq;
      i.x = reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss);
      i.g = a.g == nullptr ? 0 : reinterpret_cast<uintptr_t>(static_cast<T*>(a.g) + b * a.gsb + s * a.gss);
      i.live = v.live;
      i.y = v.y;
      i.ignored = ignored;
      if (lane == 0) {
        info[told % 3] = i;
        arrive(info_full + told % 3);
      }
      ++told;
      return v;
    };
    Values v = tell_next(), v1 = v;
    if (v.live) v1 = tell_next();
    Sum share;  // of the cluster's rows in the loss
    int n_counted = 0;
    bool waited = false;
    if (a.count == nullptr) {
      n_counted = count_tokens(a, OP);
      waited = true;
    }
    // The counting kernel's result and its clearing of the ticket.
    auto wait_for_count = [&] {
      if (waited) return;
      wait_for_previous();
      waited = true;
      n_counted = *a.count;
    };
    for (int q = 0; v.live; ++q) {
      const List list = list_at(lists + (q & 1) * list_size, slice, a.top_k);
      if (kLists && !wait_phase(list_full + (q & 1), q >> 1 & 1)) dead = true;
      if (dead || !wait_phase(together + (q & 1), q >> 1 & 1)) dead = true;
      if (dead) break;
      const float4* const here = parts + (q & 1) * warps * ranks;
      const int all = warps * ranks;
      const float4 none = make_float4(-INFINITY, 0.f, -INFINITY, 0.f), mine = lane < all ? here[lane] : none;
      float m = mine.x, m_whole = fmaxf(mine.x, mine.z);
      for (int k = lane + 32; k < all; k += 32) {
        const float4 o = here[k];
        m = fmaxf(m, o.x);
        m_whole = fmaxf(m_whole, fmaxf(o.x, o.z));
      }
      const Ref ref(warp_max(m), a.c), whole(kLists ? warp_max(m_whole) : ref.m, a.c);
      float sum = mine.y * ref.factor(mine.x, a.c), top = kLists ? mine.w * whole.factor(mine.z, a.c) : 0.f;
      for (int k = lane + 32; k < all; k += 32) {
        const float4 o = here[k];
        sum += o.y * ref.factor(o.x, a.c);
        if (kLists) top += o.w * whole.factor(o.z, a.c);
      }
      const float f = kLists ? whole.factor(ref.m, a.c) : 1.f;
      sum = warp_sum(sum);
      if (kLists) top = warp_sum(top);
      // A row without a distribution, and a bad list, whose sum is NaN.
      const float wrong = fabsf(whole.m) == INFINITY || isnan(top) ? NAN : 0.f;
      __syncwarp();
      if (ranks > 1 && lane == 0) expect_bytes(together + (q & 1), row_bytes);

      wait_for_count();
      const float w = a.weights.p != nullptr ? v.weight : 1.f / static_cast<float>(n_counted);
      float logp = 0.f, loss = 0.f;
      const ListSums both{ref, whole, f, sum, sum * f + top};
      const RowScale out = kLists ? list_scale(a, list, both, wrong, w) : policy_scale(a, v, ref, sum, wrong, w, logp, loss);
      if (lane == 0) {
        scales[q & 1] = out;
        arrive(scale_full + (q & 1));
      }
      __syncwarp();
      // The others make the gradient from here on.
      if (kLists && rank == 0) loss = list_loss(a, list, both, wrong);
      if (rank == 0) {
        if (lane == 0 && a.logp != nullptr) a.logp[v.row] = logp;
        if (lane == 0 && a.token_loss != nullptr) a.token_loss[v.row] = loss;
        share.add(a.weights.p != nullptr ? w * loss : loss);
      }
      if (kLists) {
        __syncwarp();
        if (lane == 0) arrive(list_free + (q & 1));
      }
      v = v1;
      if (v.live) v1 = tell_next();
    }
    if (dead) share.s = NAN;

    // The clusters' shares: the last to come sums them all, in order.
    if (rank == 0) {
      wait_for_count();
      add_part(a, first, stride, share, n_counted);
    }
  } else {
    // A warp that sums: in a round, chunk `mine` + k round.
    const int mine = v0 + warp * kChunk;
    const bool gradient = a.g != nullptr;
    int told = 0, told_parity = 0;
    // The ring's place of the row's first round and the parity of its barrier.
    int base = 0;
    uint32_t parity = 0;
    for (int q = 0;; ++q) {
      if (!wait_phase(info_full + told, told_parity)) break;
      const RowInfo now = info[told];
      if (++told == 3) {
        told = 0;
        told_parity ^= 1;
      }
      if (gradient && now.n_ignored > 0) {
        for (int k = 0; k < now.n_ignored; ++k) {
          const int row = now.ignored + k * stride, b = row / a.seq, s = row % a.seq;
          GradRow<T>(static_cast<T*>(a.g) + b * a.gsb + s * a.gss, a.vocab, 0).zero(rank, ranks, 32 * warps, threadIdx.x);
        }
      }
      if (!now.live) break;
      const Row<T> r(reinterpret_cast<const T*>(now.x), a.vocab);
      const List list = list_at(lists + (q & 1) * list_size, slice, a.top_k);
      if (kLists && !wait_phase(list_full + (q & 1), q >> 1 & 1)) break;

      // The warp's terms.
      const int v1 = min(r.vecs, v0 + a.vecs_per_cta), lo = r.first_whole(), hi = min(r.past_whole(), v1);
      Part<T> part;
      int place = base;
      uint32_t phase = parity;
      for (int i = mine + lane, i0 = v0; i0 < v1; i += round, i0 += round) {
        const uint4* const from = ring + place * round + warp * kChunk + lane;
        if (!LONG && !wait_phase(full + place, phase)) {
          dead = true;
          break;
        }
        // The listed words are left out here: their terms are summed apart, and
        // their gradients written after the others'.
        const int chunk = (i - lane - v0) / kChunk;
        const Bits on = kLists && i - lane < v1 ? list.bits[chunk * 32 + lane] : 0;
        if (batch_in<32>(i - lane, lo, hi)) {
          uint4 w[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) w[k] = LONG ? __ldcs(reinterpret_cast<const uint4*>(r.base) + i + k * 32) : from[k * 32];
          if (kLists && on != 0) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) leave_out<T>(w[k], on >> (8 * k));
          }
          part.add(w, a.c);
        } else {
#pragma unroll 1
          for (int k = 0; k < kBatch && i - lane + k * 32 < v1; ++k) {
            const int e = i + k * 32;
            uint4 w[1] = {no_values(kNegInf<T>)};
            if (LONG || e < copied_from(r) || e >= copied_to(r)) {
              w[0] = load_vec(r, e, v1);
            } else if (e < v1) {
              w[0] = from[k * 32];
              if (r.ragged(e)) trim(w[0], r, e);
            }
            if (kLists) leave_out<T>(w[0], on >> (8 * k));
            part.add(w, a.c);
          }
        }
        if (!LONG) {
          if (!gradient) {
            reads_before_copies();  // (no store waits for them here)
            __syncwarp();
            if (lane == 0) arrive(empty + place);
          }
          if (++place == slots) {
            place = 0;
            phase ^= 1;
          }
        }
      }
      if (dead) break;

      // The warp's part, to every CTA of the cluster: the largest value and the
      // sum, and in the first warp's those of the CTA's listed words.
      float4 p;
      p.x = warp_max(part.m);
      p.z = -INFINITY;
      p.w = 0.f;
      if (kLists && warp == 0) {
        p.z = list.head[3];
        p.w = list.head[4] + list.head[2];
      }
      p.y = warp_sum(part.s * Ref(p.x, a.c).factor(part.m, a.c));
      float4* const here = parts + (q & 1) * warps * ranks;
      if (ranks > 1) {
        if (lane < ranks) send(here + rank * warps + warp, lane, p, together + (q & 1));
      } else if (lane == 0) {
        here[warp] = p;
        arrive(together + (q & 1));
      }
      if (!wait_phase(scale_full + (q & 1), q >> 1 & 1)) break;
      const RowScale by = scales[q & 1];
      const Ref ref(by.m, a.c);

      if (gradient) {
        const GradRow<T> g(reinterpret_cast<T*>(now.g), a.vocab, r.lead);
        const bool near = g.shift == 0 && !ref.far();
        const int y_vec = now.y >= 0 ? (now.y + r.lead) / kN<T> : kNoValue;
        place = base;
        for (int i = mine + lane, i0 = v0; i0 < v1; i += round, i0 += round) {
          uint4 v[kBatch];
          const bool plain = batch_in<32>(i - lane, lo, hi);
          if (LONG) {
            load_batch<T, 32>(v, r, i, v1);
          } else {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) v[k] = ring[place * round + warp * kChunk + k * 32 + lane];  // past the slice: not stored
            if (!plain) {
#pragma unroll
              for (int k = 0; k < kBatch; ++k) {
                const int e = i + k * 32;
                if (e < v1 && (e < copied_from(r) || e >= copied_to(r))) v[k] = load_vec(r, e, v1);
              }
            }
          }
          store_batch<T, 32>(v, r, g, i, v1, plain && near && static_cast<unsigned>(y_vec - (i - lane)) >= kChunk, ref, a.c,
                             by.scale, now.y, y_vec, by.more);
          if (!LONG) {
            // The place is given back when the stores have taken what was read
            // from it.  Given back once its reads were merely begun, it was
            // seen overwritten by the next row's copy before the last of them
            // where stores to global memory held them up.  8192 x 128256 bf16
            // values take 658 us with either, 670 with a fence by every warp
            // here, 679 with one before the stores.
            __syncwarp();
            if (lane == 0) arrive(empty + place);
            if (++place == slots) place = 0;
          }
        }
        if (kLists) {
          // The listed words' values replace those written above, once all
          // warps have (each looking for its own among the ids instead: 3 % more
          // time with 64 ids, 16 % with 256; the warp that makes the lists
          // writing them: 4 % more).
          __syncwarp();
          if (lane == 0) arrive(&written);
          if (!wait_phase(&written, q & 1)) break;
          const Ref on(by.m_on, a.c);
          for (int k = threadIdx.x; k < a.top_k; k += 32 * warps) {
            const int i = list.id[k], v = (i + r.lead) / kN<T>;
            if (i >= 0 && v >= v0 && v < v1)
              narrow(g.g[i], by.lead * (by.on * ex2(on.exponent(list.x[k], a.c)) - list.p[k]));
          }
        }
      }
      if (kLists) {
        __syncwarp();
        if (lane == 0) arrive(list_free + (q & 1));
      }
      if (!LONG) {
        base += max(0, v1 - v0 + round - 1) / round;
        if (base >= slots) {
          base -= slots;
          parity ^= 1;
        }
      }
    }
  }
  if (ranks > 1) {  // nobody leaves while others may write here
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
}

// ---- short rows -------------------------------------------------------------------
// TEAM warps have a row and keep it in registers.  Nothing is handed to other
// warps but the team's parts: 16384 rows of 1000 bf16 values take 33 us, 70 in
// k_loss_row, whose rows pass through three warps and two barriers; 4096 rows
// of 8192 37 us for 45.  Teams of eight no longer gain: 4096 rows of 12000 63 us
// for 59, with a teacher's 64 entries of 16000 88 us for 73.
constexpr int kShortVecs = 8;     // of a lane
constexpr int kShortWarps = 8;    // of a CTA
constexpr int kMaxTeam = 4;
template <typename T, int OP, int TEAM>
__global__ void __launch_bounds__(32 * kShortWarps, 2) k_loss_short(const __grid_constant__ LossArgs a) {
  extern __shared__ __align__(16) unsigned char shared[];
  __shared__ Sum shares[kShortWarps];
  __shared__ float2 parts[2][kShortWarps];
  constexpr bool kLists = OP == kDistill;
  constexpr int kOwn = 32 * kShortVecs, kSlice = kOwn * TEAM, kTeams = kShortWarps / TEAM;
  static_assert(kOwn % kChunk == 0, "a list's bits are by chunks");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / TEAM, member = warp % TEAM;
  auto team_sync = [&] {
    if (TEAM == 1) __syncwarp();
    else asm volatile("barrier.sync.aligned %0, %1;" ::"r"(1 + team), "n"(32 * TEAM) : "memory");
  };
  const List list = list_at(shared + team * (kLists ? list_bytes(kSlice, a.top_k) : 0), kSlice, a.top_k);
  int n_counted = 0;
  bool waited = false;
  if (a.count == nullptr) {
    n_counted = count_tokens(a, OP);
    waited = true;
  }
  auto wait_for_count = [&] {
    if (waited) return;
    wait_for_previous();
    waited = true;
    n_counted = *a.count;
  };
  Sum share;
  int q = 0;
  for (int row = static_cast<int>(blockIdx.x) * kTeams + team; row < a.tokens; row += gridDim.x * kTeams) {
    const int b = row / a.seq, s = row % a.seq;
    const Row<T> r(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss, a.vocab);
    const GradRow<T> g(a.g == nullptr ? nullptr : static_cast<T*>(a.g) + b * a.gsb + s * a.gss, a.vocab, r.lead);
    const int first = member * kOwn + lane;
    // Read before it is known whether the row counts: one wait, not two.  (What
    // is read of a row that does not is left alone.)
    uint4 w[kShortVecs];
    load_batch<T, 32>(w, r, first, r.vecs);
    Values v{row, kNoValue, true, {0.f, 0.f, 0.f}, 0.f, 0.f};
    bool live;
    if (kLists) {
      live = counted(a, OP, b, s);
    } else {
      const int64_t target = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
      live = target != a.ignore;
      if (live && target >= 0 && target < a.vocab) {
        v.y = static_cast<int>(target);
        v.x_at = widen(*r.value(v.y));
      }
    }
    if (!live) {
      if (a.g != nullptr) g.zero(member, TEAM, 32, lane);
      if (member == 0 && lane == 0) {
        if (a.logp != nullptr) a.logp[row] = 0.f;
        if (a.token_loss != nullptr) a.token_loss[row] = 0.f;
      }
      continue;
    }
    if (OP == kPolicy) {
      v.in.adv = row_value(a.adv, b, s);
      if (a.old.p != nullptr) v.in.old = row_value(a.old, b, s);
      if (a.kl != 0.f) v.in.ref = row_value(a.ref, b, s);
    }
    if (a.weights.p != nullptr) v.weight = row_value(a.weights, b, s);
    if (kLists) {
      team_sync();  // the list before has been read
      if (member == 0) make_list(a, list, r, b, s, 0, r.vecs, kSlice, true);
      team_sync();
#pragma unroll
      for (int k = 0; k < kShortVecs; ++k)
        leave_out<T>(w[k], list.bits[(member * (kOwn / kChunk) + k / kBatch) * 32 + lane] >> (k % kBatch * 8));
    }
    Part<T> part;
    part.add(w, a.c);
    // (the target's logit, and a list's, are read before anything is written)
    float m = warp_max(part.m);
    float sum = warp_sum(part.s * Ref(m, a.c).factor(part.m, a.c));
    if (TEAM > 1) {
      if (lane == 0) parts[q & 1][warp] = make_float2(m, sum);
      team_sync();
      const float2* const here = parts[q & 1] + team * TEAM;
      for (int k = 0; k < TEAM; ++k) m = fmaxf(m, here[k].x);
      sum = 0.f;
      for (int k = 0; k < TEAM; ++k) sum += here[k].y * Ref(m, a.c).factor(here[k].x, a.c);
    }
    ++q;
    const Ref ref(m, a.c);
    const Ref whole(kLists ? fmaxf(m, list.head[3]) : m, a.c);
    const float f = kLists ? whole.factor(m, a.c) : 1.f;
    const ListSums both{ref, whole, f, sum, kLists ? sum * f + list.head[4] * whole.factor(list.head[3], a.c) : sum};
    const float wrong = (kLists ? list.head[2] : 0.f) + (fabsf(whole.m) == INFINITY ? NAN : 0.f);
    wait_for_count();
    const float weight = a.weights.p != nullptr ? v.weight : 1.f / static_cast<float>(n_counted);
    float logp = 0.f, loss = 0.f;
    const RowScale by = kLists ? list_scale(a, list, both, wrong, weight) : policy_scale(a, v, ref, sum, wrong, weight, logp, loss);
    if (a.g != nullptr) {
      const int y_vec = v.y >= 0 ? (v.y + r.lead) / kN<T> : kNoValue;
      const bool plain = batch_in<32, kShortVecs>(first - lane, r.first_whole(), r.past_whole()) && g.shift == 0 && !ref.far() &&
                         static_cast<unsigned>(y_vec - (first - lane)) >= kOwn;
      store_batch<T, 32>(w, r, g, first, r.vecs, plain, ref, a.c, by.scale, v.y, y_vec, by.more);
      if (kLists) {
        __syncwarp();  // the listed words' values replace those that this warp wrote
        for (int k = lane; k < a.top_k; k += 32) {
          const int i = list.id[k];
          if (i >= 0 && (i + r.lead) / kN<T> / kOwn == member)
            narrow(g.g[i], by.lead * (by.on * ex2(whole.exponent(list.x[k], a.c)) - list.p[k]));
        }
      }
    }
    if (member != 0) continue;
    if (kLists) loss = list_loss(a, list, both, wrong);
    if (lane == 0 && a.logp != nullptr) a.logp[row] = logp;
    if (lane == 0 && a.token_loss != nullptr) a.token_loss[row] = loss;
    share.add(a.weights.p != nullptr ? weight * loss : loss);
  }
  if (lane == 0) shares[warp] = share;
  __syncthreads();
  if (warp != 0) return;
  wait_for_count();
  Sum all;
  for (int k = 0; k < kShortWarps; ++k) {
    const Sum p = shares[k];
    all.add(p);
  }
  add_part(a, blockIdx.x, gridDim.x, all, n_counted);
}

// ---- log-probabilities --------------------------------------------------------
// A row is read once and nothing of it is kept: a CTA (or, for a few rows, a
// cluster) has one, a thread loads a batch while it adds up the one before.
// 8192 x 128256 bf16 values (6144 rows counted) take 234 us, 0.99 of the copy
// rate; in k_loss_row's first form, all of a row in registers before its sum
// began, 418.
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_loss_forward(const __grid_constant__ LossArgs a) {
  extern __shared__ __align__(16) unsigned char shared[];
  float4* parts = reinterpret_cast<float4*>(shared);  // [warps of the cluster]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int warps = NT / 32;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int row = static_cast<int>(blockIdx.x) / ranks, b = row / a.seq, s = row % a.seq;
  // k_loss_pair may begin as these CTAs end; its ticket is cleared here
  let_next_start();
  if (a.ticket != nullptr && blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  const bool writes = rank == 0 && warp == 0;
  const int64_t target = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
  if (writes && lane == 0 && a.coef_out != nullptr) a.coef_out[row] = 0.f;
  if (target == a.ignore) {
    if (writes && lane == 0) {
      a.logp[row] = 0.f;
      if (a.stats != nullptr) a.stats[row] = make_float2(0.f, 0.f);
    }
    return;
  }
  if (ranks > 1) cluster_arrive();
  const Row<T> r(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss, a.vocab);
  const int v0 = rank * a.vecs_per_cta, v1 = min(r.vecs, v0 + a.vecs_per_cta);
  const bool inside = target >= 0 && target < a.vocab;
  const float x_at = writes && inside ? widen(*r.value(static_cast<int>(target))) : NAN;
  Part<T> part;
  uint4 w[kForwardBatch], w1[kForwardBatch];
  load_batch<T, NT>(w, r, v0 + tid, v1);
  for (int i = v0 + tid; i - lane < v1; i += kForwardBatch * NT) {
    load_batch<T, NT>(w1, r, i + kForwardBatch * NT, v1);
    part.add(w, a.c);
#pragma unroll
    for (int k = 0; k < kForwardBatch; ++k) w[k] = w1[k];
  }
  float4 p;
  p.x = warp_max(part.m);
  p.y = warp_sum(part.s * Ref(p.x, a.c).factor(part.m, a.c));
  p.z = p.w = 0.f;
  if (ranks > 1) {
    cluster_wait();
    if (lane == 0) store_remote(parts + rank * warps + warp, 0, p);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  } else {
    if (lane == 0) parts[warp] = p;
    __syncthreads();
  }
  if (!writes) return;
  float m = -INFINITY, sum = 0.f;
  for (int k = lane; k < warps * ranks; k += 32) m = fmaxf(m, parts[k].x);
  const Ref ref(warp_max(m), a.c);
  for (int k = lane; k < warps * ranks; k += 32) sum += parts[k].y * ref.factor(parts[k].x, a.c);
  sum = warp_sum(sum);
  const float wrong = fabsf(ref.m) == INFINITY ? NAN : 0.f;  // a row without a distribution
  if (lane == 0) {
    a.logp[row] = over_t(x_at - ref.m, a.per_t) - logf(sum) + ref.residue(a.c) * kLn2 + wrong;
    if (a.stats != nullptr) a.stats[row] = make_float2(ref.m, sum + wrong);
  }
}

// ---- gradient rows from kept statistics ------------------------------------------
// A CTA has a tile of a row; the last rows come first: of what the forward
// pass read they are the ones most likely still in L2.  4096 x 32000 bf16
// values take 77 us and 999 x 50257 fp32 59 us, the copy rate; with a gradient
// whose rows start at other 16-byte phases than the logits' 71 us.
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_loss_grad(const __grid_constant__ LossArgs a) {
  const int row = a.tokens - 1 - static_cast<int>(blockIdx.x / a.tiles), tile = blockIdx.x % a.tiles;
  const int b = row / a.seq, s = row % a.seq;
  const Row<T> r(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss, a.vocab);
  const GradRow<T> g(static_cast<T*>(a.g) + b * a.gsb + s * a.gss, a.vocab, r.lead);
  const int64_t target = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
  if (a.coef != nullptr) wait_for_previous();
  if (target == a.ignore) {
    g.zero(tile, a.tiles, NT, threadIdx.x);
    return;
  }
  const int first = tile * kGradVecs * NT + threadIdx.x;
  const int last = min(r.vecs, (tile + 1) * kGradVecs * NT);
  uint4 w[kGradVecs];
  load_batch<T, NT>(w, r, first, last);
  const float2 st = a.stats[row];
  const float d = (a.coef != nullptr ? a.coef[row] : row_value(a.dlogp, b, s)) * a.gscale * a.inv_t;
  const bool inside = target >= 0 && target < a.vocab;
  const float scale = inside ? -d / st.y : NAN;
  const Ref ref(st.x, a.c);
  const int y = inside ? static_cast<int>(target) : kNoValue;
  const int y_vec = inside ? (y + r.lead) / kN<T> : kNoValue;
  const int lane_first = first - (threadIdx.x & 31), to_y = y_vec - lane_first;
  const bool plain = batch_in<NT, kGradVecs>(lane_first, r.first_whole(), min(r.past_whole(), last)) && g.shift == 0 &&
                     !ref.far() && !(to_y >= 0 && to_y < kGradVecs * NT && to_y % NT < 32);
  store_batch<T, NT>(w, r, g, first, last, plain, ref, a.c, scale, y, y_vec, d);
}

// ---- a pair's loss ---------------------------------------------------------------
__global__ void __launch_bounds__(kPairThreads) k_loss_pair(const __grid_constant__ LossArgs a) {
  __shared__ Sum sums[2][kPairThreads / 32];
  __shared__ int counts[2][kPairThreads / 32], last;
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t pair = blockIdx.x;
  int64_t from[2], to[2];
  bool ok = true;
  for (int h = 0; h < 2; ++h) {
    const int64_t q = pair + h * a.pairs;
    if (a.offsets != nullptr) {
      from[h] = load_index(a.offsets, a.odt, q);
      to[h] = load_index(a.offsets, a.odt, q + 1);
      if (from[h] < 0 || to[h] < from[h] || to[h] > a.tokens) {
        ok = false;
        from[h] = to[h] = 0;
      }
    } else {
      from[h] = q * a.seq;
      to[h] = from[h] + a.seq;
    }
    Sum sum;
    int n = 0;
#pragma unroll 4
    for (uint32_t t = static_cast<uint32_t>(from[h]) + threadIdx.x; t < static_cast<uint32_t>(to[h]); t += kPairThreads) {
      const int b = static_cast<int>(t / static_cast<uint32_t>(a.seq)), s = static_cast<int>(t % static_cast<uint32_t>(a.seq));
      if (!counted(a, kLogprobs, b, s)) continue;
      sum.add(a.logp[t]);
      if (a.ref.p != nullptr) sum.add(-row_value(a.ref, b, s));
      ++n;
    }
    sum.over_warp();
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      sums[h][warp] = sum;
      counts[h][warp] = n;
    }
  }
  __syncthreads();
  float D[2], n[2];
  for (int h = 0; h < 2; ++h) {
    Sum sum;
    int count = 0;
    for (int w = 0; w < kPairThreads / 32; ++w) {
      const Sum p = sums[h][w];
      sum.add(p);
      count += counts[h][w];
    }
    n[h] = static_cast<float>(count);
    D[h] = a.average ? (count > 0 ? sum.total() / n[h] : 0.f) : sum.total();
  }
  const float h = D[0] - D[1];
  float loss, dh;  // and its derivative with respect to h
  if (a.kind == LOSS_PREFERENCE_SIGMOID) {
    const float z = a.beta * h - a.margin, e = expf(-fabsf(z)), l = log1pf(e);
    const float neg = l + fmaxf(-z, 0.f), pos = l + fmaxf(z, 0.f);  // -ln s(z), -ln s(-z)
    const float big = 1.f / (1.f + e), small = e / (1.f + e);
    // (pos is infinite where the rejected side has probability 0: with e = 0 it is no term)
    loss = (1.f - a.smooth) * neg + (a.smooth != 0.f ? a.smooth * pos : 0.f);
    dh = a.beta * (z >= 0.f ? a.smooth * big - (1.f - a.smooth) * small : a.smooth * small - (1.f - a.smooth) * big);
  } else if (a.kind == LOSS_PREFERENCE_HINGE) {
    const float z = 1.f + a.margin - a.beta * h;
    loss = z > 0.f || isnan(z) ? z : 0.f;
    dh = z > 0.f ? -a.beta : isnan(z) ? z : 0.f;
  } else {
    const float z = h - 1.f / (2.f * a.beta) - a.margin;
    loss = z * z;
    dh = 2.f * z;
  }
  if (!ok) loss = dh = NAN;
  if (threadIdx.x == 0) {
    if (a.pair_loss != nullptr) a.pair_loss[pair] = loss;
    a.pair_part[pair] = loss;
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == static_cast<unsigned>(a.pairs - 1);
    if (a.rewards != nullptr) {
      a.rewards[pair] = ok ? a.beta * D[0] : NAN;
      a.rewards[pair + a.pairs] = ok ? a.beta * D[1] : NAN;
    }
  }
  for (int q = 0; q < 2; ++q) {
    float c = (q == 0 ? dh : -dh) / static_cast<float>(a.pairs);
    if (a.average) c = n[q] > 0.f ? c / n[q] : 0.f;
    for (int64_t t = from[q] + threadIdx.x; t < to[q]; t += kPairThreads) a.coef_out[t] = c;
  }
  __syncthreads();
  if (!last || warp != 0) return;
  // the last pair to come sums them all, in order
  __threadfence();
  Sum v;
  for (int64_t k = lane; k < a.pairs; k += 32) v.add(__ldcg(a.pair_part + k));
  v.over_warp();
  if (lane == 0) *a.loss = v.total() / static_cast<float>(a.pairs);
}

// ---- host side -----------------------------------------------------------------
adaf_status fail(adaf_status st, const std::string& msg) { return meo::set_last_error(st, ("loss: " + msg).c_str()); }
adaf_status invalid(const std::string& msg) { return fail(ADAF_ERR_INVALID_ARGUMENT, msg); }
adaf_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ADAF_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t dtype_size(int32_t dt) { return dt == ADAF_BFLOAT16 ? 2 : 4; }
size_t index_size(int32_t dt) { return dt == LOSS_INT64 ? 8 : 4; }

// Strides whose offsets stay below 2^59, so that no address sum overflows.
bool strides_ok(int64_t batch, int64_t seq, int64_t sb, int64_t ss) {
  if (sb < 0 || ss < 0) return false;
  const int64_t most = int64_t{1} << 58;
  return (batch <= 1 || sb <= most / (batch - 1)) && (seq <= 1 || ss <= most / (seq - 1));
}

adaf_status check_rows(const loss_logits& x, const loss_rows& r, const char* name, size_t align, bool optional) {
  if (r.p == nullptr) return optional ? ADAF_OK : invalid(std::string(name) + " is NULL");
  if (!aligned(r.p, align)) return invalid(std::string(name) + " is not element-aligned");
  if (!strides_ok(x.batch, x.seq, r.stride_b, r.stride_s)) return invalid(std::string(name) + ": bad strides");
  return ADAF_OK;
}

adaf_status check_logits(const loss_logits* x) {
  if (x == nullptr) return invalid("logits is NULL");
  if (x->dtype != ADAF_FLOAT32 && x->dtype != ADAF_BFLOAT16) return invalid("logits: unknown dtype");
  if (x->batch < 0 || x->seq < 0) return invalid("logits: batch or seq < 0");
  if (x->vocab < 1) return invalid("logits: vocab must be >= 1");
  if (x->vocab > kMaxVocab) return fail(ADAF_ERR_UNSUPPORTED, "logits: vocab must be at most 2^21");
  if (x->batch > kMaxTokens || x->seq > kMaxTokens || x->batch * x->seq > kMaxTokens)
    return fail(ADAF_ERR_UNSUPPORTED, "logits: batch * seq must be at most 2^30");
  if (!(x->temperature > 0.0) || !std::isfinite(x->temperature))
    return invalid("invalid temperature (needs 0 < temperature < inf)");
  const double inv = 1.0 / x->temperature;
  if (!(inv >= 1e-30) || !(inv <= 1e30)) return invalid("invalid temperature (needs 1e-30 .. 1e30)");
  if (!strides_ok(x->batch, x->seq, x->stride_b, x->stride_s)) return invalid("logits: bad strides");
  if (x->batch * x->seq > 0) {
    if (x->p == nullptr) return invalid("logits is NULL");
    if (!aligned(x->p, dtype_size(x->dtype))) return invalid("logits is not element-aligned");
  }
  return ADAF_OK;
}

adaf_status check_targets(const loss_logits& x, const loss_targets* y) {
  if (y == nullptr) return invalid("targets is NULL");
  if (y->dtype != LOSS_INT32 && y->dtype != LOSS_INT64) return invalid("targets: unknown dtype");
  if (x.batch * x.seq == 0) return ADAF_OK;
  return check_rows(x, y->rows, "targets", index_size(y->dtype), false);
}

// First and one past the last byte of the rows.
void extent(const void* p, int64_t batch, int64_t seq, int64_t sb, int64_t ss, int64_t vocab, size_t es, uintptr_t* lo,
            uintptr_t* hi) {
  const int64_t last = (batch - 1) * sb + (seq - 1) * ss + vocab;
  *lo = reinterpret_cast<uintptr_t>(p);
  *hi = *lo + static_cast<uintptr_t>(last) * es;
}

adaf_status check_grad(const loss_logits& x, const loss_grad* g, bool optional) {
  if (g == nullptr || g->p == nullptr) {
    if (optional || x.batch * x.seq == 0) return ADAF_OK;
    return invalid("grad is NULL");
  }
  if (!std::isfinite(g->scale)) return invalid("grad: scale must be finite");
  if (x.batch * x.seq == 0) return ADAF_OK;
  const size_t es = dtype_size(x.dtype);
  if (!aligned(g->p, es)) return invalid("grad is not element-aligned");
  if (!strides_ok(x.batch, x.seq, g->stride_b, g->stride_s)) return invalid("grad: bad strides");
  // Rows apart: the inner of the two dims steps over a row, the outer over
  // all that the inner one covers.
  const int64_t sb = x.batch > 1 ? g->stride_b : -1, ss = x.seq > 1 ? g->stride_s : -1;
  const bool b_outer = (ss < 0 || ss >= x.vocab) && (sb < 0 || sb >= (x.seq - 1) * std::max<int64_t>(ss, 0) + x.vocab);
  const bool s_outer =
      (sb < 0 || sb >= x.vocab) && (ss < 0 || ss >= (x.batch - 1) * std::max<int64_t>(sb, 0) + x.vocab);
  if (!b_outer && !s_outer) return invalid("grad: rows overlap");
  const bool same = g->p == x.p && (x.batch == 1 || g->stride_b == x.stride_b) && (x.seq == 1 || g->stride_s == x.stride_s);
  if (!same) {
    uintptr_t xl, xh, gl, gh;
    extent(x.p, x.batch, x.seq, x.stride_b, x.stride_s, x.vocab, es, &xl, &xh);
    extent(g->p, x.batch, x.seq, g->stride_b, g->stride_s, x.vocab, es, &gl, &gh);
    if (xl < gh && gl < xh) return invalid("grad overlaps the logits without being the same rows");
  }
  return ADAF_OK;
}

struct Layout {
  size_t off_part = 0, off_stats = 0, off_logp = 0, off_coef = 0, off_pair = 0, bytes = 0;
};
constexpr int kMaxClusters = 1 << 13;  // of k_loss_row: at most the CTAs that a GPU holds
adaf_status layout(int64_t tokens, int64_t pairs, Layout* L) {
  if (tokens < 0 || pairs < 0) return invalid("tokens or pairs < 0");
  if (tokens > kMaxTokens || pairs > kMaxTokens / 2)
    return fail(ADAF_ERR_UNSUPPORTED, "at most 2^30 tokens and 2^29 pairs");
  size_t o = 256;  // the count of tokens, the ticket at byte 8
  const size_t n = static_cast<size_t>(tokens);
  if (pairs == 0) {
    L->off_part = o;
    o = round_up(o + sizeof(Sum) * std::min<size_t>(n, kMaxClusters), 256);
  } else {
    L->off_stats = o; o = round_up(o + sizeof(float2) * n, 256);
    L->off_logp = o;  o = round_up(o + sizeof(float) * n, 256);
    L->off_coef = o;  o = round_up(o + sizeof(float) * n, 256);
    L->off_pair = o;  o = round_up(o + sizeof(float) * static_cast<size_t>(pairs), 256);
  }
  L->bytes = o;
  return ADAF_OK;
}
adaf_status check_workspace(const void* ws, size_t bytes, const Layout& L) {
  if (ws == nullptr || !aligned(ws, 256)) return invalid("workspace is NULL or not 256-byte aligned");
  if (bytes < L.bytes)
    return fail(ADAF_ERR_WORKSPACE_TOO_SMALL, "workspace needs " + std::to_string(L.bytes) + " bytes");
  return ADAF_OK;
}

Rows rows_of(const loss_rows& r) { return Rows{r.p, r.stride_b, r.stride_s}; }

LossArgs base_args(const loss_logits& x, const loss_targets* y, const loss_grad* g) {
  LossArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = x.p;
  a.xsb = x.stride_b;
  a.xss = x.stride_s;
  if (x.batch * x.seq > 0) extent(x.p, x.batch, x.seq, x.stride_b, x.stride_s, x.vocab, dtype_size(x.dtype), &a.x_begin, &a.x_end);
  a.seq = static_cast<int32_t>(x.seq);
  a.tokens = static_cast<int32_t>(x.batch * x.seq);
  a.vocab = static_cast<int32_t>(x.vocab);
  a.c = static_cast<float>(1.4426950408889634 / x.temperature);
  const double per_t = 1.0 / x.temperature;
  a.inv_t = a.per_t.hi = static_cast<float>(per_t);
  if (per_t - a.per_t.hi < per_t * 0x1p-30) a.per_t.hi = std::nextafterf(a.per_t.hi, 0.f);
  a.per_t.lo = static_cast<float>(per_t - a.per_t.hi);
  if (g != nullptr && g->p != nullptr) {
    a.g = g->p;
    a.gsb = g->stride_b;
    a.gss = g->stride_s;
    a.gscale = static_cast<float>(g->scale);
  }
  if (y != nullptr) {
    a.y = rows_of(y->rows);
    a.ydt = y->dtype;
    a.ignore = y->ignore_index;
  }
  return a;
}

const char* const kKernelNames[] = {"k_loss_count", "k_loss_row", "k_loss_short", "k_loss_forward", "k_loss_grad", "k_loss_pair"};
enum Slot { kSlotCount = 0, kSlotRow, kSlotShort, kSlotForward, kSlotGrad, kSlotPair, kNumKernels };
struct ProfRecord {
  int slot;
  cudaEvent_t start, stop;
};
std::mutex g_mu;
bool g_profile = false;
thread_local bool t_stall = false;
std::vector<ProfRecord> g_prof;

// Launches a kernel of this file; under profiling between two events.
// `overlap`: the kernel may begin while the one before it ends (it waits for
// that one itself, where it needs its results).
template <typename... Args>
adaf_status launch(int slot, void (*kernel)(LossArgs, Args...), int64_t grid, int threads, int shared, int cluster,
                   bool overlap, cudaStream_t s, const LossArgs& a, Args... args) {
  bool prof;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    prof = g_profile;
  }
  ProfRecord rec{slot, nullptr, nullptr};
  cudaError_t e = cudaSuccess;
  if (prof) {
    if ((e = cudaEventCreate(&rec.start)) != cudaSuccess || (e = cudaEventCreate(&rec.stop)) != cudaSuccess ||
        (e = cudaEventRecord(rec.start, s)) != cudaSuccess)
      return cuda_fail(e, "profile event");
  }
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(shared);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    ++cfg.numAttrs;
  }
  if (overlap) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  if ((e = cudaLaunchKernelEx(&cfg, kernel, a, args...)) != cudaSuccess) {
    cudaGetLastError();
    return cuda_fail(e, kKernelNames[slot]);
  }
  if (prof) {
    if ((e = cudaEventRecord(rec.stop, s)) != cudaSuccess) return cuda_fail(e, "profile event");
    std::lock_guard<std::mutex> lock(g_mu);
    g_prof.push_back(rec);
  }
  return ADAF_OK;
}

// Vectors of a row, at any alignment that the rows have.
int row_vecs(const LossArgs& a, int32_t dtype) {
  const int es = static_cast<int>(dtype_size(dtype)), per = 16 / es;
  const bool even = a.x_begin % 16 == 0 && a.xsb * es % 16 == 0 && a.xss * es % 16 == 0;
  return div_up(a.vocab + (even ? 0 : per - 1), per);
}

// How a row is cut: CTAs, warps of each that sum, vectors of a CTA, places of
// its ring, a round each (0: the row is read twice).
struct Cut {
  int cluster, warps, vecs_per_cta, slots, shared;
};
constexpr int kSharedBytes = 227 << 10;  // of an SM; a CTA takes 1 KB more than it asks for

Cut cut_row(int64_t tokens, int vecs, bool lists, int top_k, int sms) {
  const int chunks = div_up(vecs, kChunk);
  Cut c;
  // `keep`: chunks of a row for a warp
  auto set = [&](int cluster, int keep) {
    const int mine = div_up(chunks, cluster);
    c.cluster = cluster;
    c.vecs_per_cta = mine * kChunk;
    c.warps = std::min(kMaxWarps, div_up(mine, keep));
    const int n = div_up(mine, c.warps);
    c.shared = 2 * c.warps * cluster * static_cast<int>(sizeof(float4)) + (lists ? 2 * list_bytes(c.vecs_per_cta, top_k) : 0);
    const int place = c.warps * kChunk * 16 + 16;  // and its two barriers
    for (int ctas = 2 * kMaxWarps / c.warps; ctas >= 1; ctas /= 2) {  // long lists: fewer CTAs of an SM
      const int room = kSharedBytes / ctas - 1024 - 512 - c.shared;
      c.slots = std::min(2 * n, std::max(0, room / place));
      // places for a row and more; beside long lists for one row: a second CTA
      // that makes lists is worth more (4096 x 128256, 1000 entries, one such warp
      // in each: 1451 us, 2486 with one CTA an SM)
      if (c.slots > n || (lists && c.slots == n)) break;
    }
    if (c.slots < n) c.slots = 0;
    c.shared += c.slots * place;
  };
  int cluster = 1;
  set(1, kKeep);
  while (cluster < kMaxCluster && c.vecs_per_cta > kMaxWarps * kKeep * kChunk) set(cluster *= 2, kKeep);
  while (cluster < kMaxCluster && tokens * cluster < sms && c.vecs_per_cta > kChunk) set(cluster *= 2, 1);
  return c;
}

struct Device {
  int sms = 0;
  unsigned* tickets = nullptr;           // g_tickets on this device
  std::map<unsigned long long, int> streams;  // of the streams that have one, by the stream's id
  std::map<std::pair<const void*, int64_t>, int> clusters;  // that run at a time, by kernel and cut
};
std::map<int, Device> g_devices;
// The current device's, with g_mu held.
Device* current_device(cudaError_t* e) {
  int device = 0;
  if ((*e = cudaGetDevice(&device)) != cudaSuccess) return nullptr;
  Device& dev = g_devices[device];
  if (dev.sms == 0 && (*e = cudaDeviceGetAttribute(&dev.sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess)
    return nullptr;
  return &dev;
}

template <int OP>
adaf_status launch_rows(LossArgs a, int32_t dtype, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  int sms = 0;
  std::unique_lock<std::mutex> lock(g_mu);
  Device* const dev = current_device(&e);
  if (dev == nullptr) return cuda_fail(e, "current device");
  sms = dev->sms;
  const int vecs = row_vecs(a, dtype);
  const bool bf16 = dtype == ADAF_BFLOAT16;
  if (vecs <= 32 * kShortVecs * kMaxTeam) {
    lock.unlock();
    int team = 1;
    while (32 * kShortVecs * team < vecs) team *= 2;
    const int teams = kShortWarps / team;
    const int shared = OP == kDistill ? teams * list_bytes(32 * kShortVecs * team, a.top_k) : 0;
    void (*const kernel)(LossArgs) = team == 1   ? (bf16 ? k_loss_short<__nv_bfloat16, OP, 1> : k_loss_short<float, OP, 1>)
                                     : team == 2 ? (bf16 ? k_loss_short<__nv_bfloat16, OP, 2> : k_loss_short<float, OP, 2>)
                                                 : (bf16 ? k_loss_short<__nv_bfloat16, OP, 4> : k_loss_short<float, OP, 4>);
    if (shared > (48 << 10) - 512 &&
        (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes - 1024)) != cudaSuccess)
      return cuda_fail(e, "cudaFuncSetAttribute");
    const int grid = std::min(div_up(a.tokens, teams), 2 * sms);
    return launch(kSlotShort, kernel, grid, 32 * kShortWarps, shared, 1, a.count != nullptr, s, a);
  }
  const Cut cut = cut_row(a.tokens, vecs, OP == kDistill, a.top_k, sms);
  const bool twice_read = cut.slots == 0;
  constexpr int kFew = OP == kDistill ? 1 : 0, kMany = 2 * kFew;
  const int listers = kFew == 1 && !twice_read && a.top_k >= kTwoListers ? 2 : kFew;
  void (*const kernel)(LossArgs) =
      twice_read    ? (bf16 ? k_loss_row<__nv_bfloat16, OP, true> : k_loss_row<float, OP, true>)
      : listers < 2 ? (bf16 ? k_loss_row<__nv_bfloat16, OP, false> : k_loss_row<float, OP, false>)
                    : (bf16 ? k_loss_row<__nv_bfloat16, OP, false, kMany> : k_loss_row<float, OP, false, kMany>);
  const int threads = 32 * (cut.warps + 2 + listers);
  int& most = dev->clusters[{reinterpret_cast<const void*>(kernel),
                            (static_cast<int64_t>(cut.shared) << 16) + (cut.warps << 4) + cut.cluster}];
  if (most == 0) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes - 1024)) != cudaSuccess)
      return cuda_fail(e, "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(cut.cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(cut.shared);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {static_cast<unsigned>(cut.cluster), 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess)
      return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
    if (n < 1) return fail(ADAF_ERR_CUDA, "no cluster of k_loss_row fits on the device");
    most = std::min(n, kMaxClusters);
  }
  const int64_t clusters = std::min<int64_t>(a.tokens, most);
  lock.unlock();
  a.vecs_per_cta = cut.vecs_per_cta;
  a.slots = cut.slots;
  a.stall = t_stall ? 1 : 0;
  return launch(kSlotRow, kernel, clusters * cut.cluster, threads, cut.shared, cut.cluster, a.count != nullptr, s, a);
}
adaf_status launch_forward(LossArgs a, int32_t dtype, cudaStream_t s) {
  const int vecs = row_vecs(a, dtype);
  int sms = 0;
  {
    cudaError_t e = cudaSuccess;
    std::lock_guard<std::mutex> lock(g_mu);
    const Device* const dev = current_device(&e);
    if (dev == nullptr) return cuda_fail(e, "current device");
    sms = dev->sms;
  }
  int64_t cluster = 1;
  // Few rows are cut among a cluster's CTAs.  (Cutting them where that would
  // only fill the last wave of CTAs better costs more than it gives: 999 rows
  // of 50257 fp32 values 38 us whole, 47 cut in two.)
  while (cluster < kMaxCluster && a.tokens * cluster < 2 * sms && div_up(vecs, static_cast<int>(cluster)) > 512) cluster *= 2;
  a.vecs_per_cta = div_up(vecs, static_cast<int>(cluster));
  // Small CTAs keep the SMs' loads apart in time, and with many rows their ends
  // too; few rows want more threads each.  In CTAs of 32, 128, 256, 512:
  //   16384 x 1000 bf16       18, 39 us
  //   4096 x 8192             13, 17
  //   8192 x 128256          299, 295, 299, 304
  //   600 x 128256                 29,  25,  27
  //   100 x 128256 (4 CTAs)   21, 9.4, 7.7, 10.8
  const int64_t ctas = a.tokens * cluster;
  const int threads = a.vecs_per_cta <= 1024 ? (ctas >= 16 * sms ? 32 : 128) : ctas >= 8 * sms ? 128 : 256;
  const int shared = threads / 32 * static_cast<int>(cluster * sizeof(float4));
  const bool bf16 = dtype == ADAF_BFLOAT16;
  void (*const kernel)(LossArgs) =
      threads == 256   ? (bf16 ? k_loss_forward<__nv_bfloat16, 256> : k_loss_forward<float, 256>)
      : threads == 128 ? (bf16 ? k_loss_forward<__nv_bfloat16, 128> : k_loss_forward<float, 128>)
                       : (bf16 ? k_loss_forward<__nv_bfloat16, 32> : k_loss_forward<float, 32>);
  return launch(kSlotForward, kernel, a.tokens * cluster, threads, shared, static_cast<int>(cluster), false, s, a);
}
adaf_status launch_grad(LossArgs a, int32_t dtype, cudaStream_t s) {
  // A tile is 256 threads' or, for rows that fill no such tile, a warp's:
  // 16384 rows of 1000 bf16 values take 61 us in CTAs of 256 threads.
  const int vecs = row_vecs(a, dtype), threads = vecs <= 4 * 32 * kGradVecs ? 32 : kGradThreads;
  const bool bf16 = dtype == ADAF_BFLOAT16;
  a.tiles = div_up(vecs, threads * kGradVecs);
  const int64_t grid = static_cast<int64_t>(a.tokens) * a.tiles;
  if (grid > INT32_MAX) return fail(ADAF_ERR_UNSUPPORTED, "gradient of more than 2^31 tiles");
  void (*const kernel)(LossArgs) =
      threads == 32 ? (bf16 ? k_loss_grad<__nv_bfloat16, 32> : k_loss_grad<float, 32>)
                    : (bf16 ? k_loss_grad<__nv_bfloat16, kGradThreads> : k_loss_grad<float, kGradThreads>);
  return launch(kSlotGrad, kernel, grid, threads, 0, 1, a.coef != nullptr, s, a);
}
// A call for a few tokens is one launch: the managing warps count the tokens
// themselves, and the ticket is one that the library keeps for the stream (the
// last CTA leaves it at 0; calls on one stream follow one another).  A call of
// 400 tokens of 500 words takes 21.8 us so, 24.0 us with k_loss_count before
// it, host time for the most part; beyond some hundred tokens a warp's counting
// would hold the first row up.  A stream is known by its id, which no other gets:
// its handle may be another's once it is destroyed, while its last call still
// runs.  Streams beyond the first 1024 and captured calls, which may be replayed
// on any stream, take the workspace's ticket.
constexpr int kFewTokens = 512;
constexpr int kTickets = 1024;
__device__ unsigned g_tickets[kTickets];

unsigned* stream_ticket(cudaStream_t s) {
  if (s == cudaStreamPerThread) return nullptr;  // a handle for many streams
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capturing) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  int device = 0;
  unsigned long long id = 0;
  if (capturing != cudaStreamCaptureStatusNone) return nullptr;
  if (cudaGetDevice(&device) != cudaSuccess || cudaStreamGetId(s, &id) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  Device& dev = g_devices[device];
  if (dev.tickets == nullptr && cudaGetSymbolAddress(reinterpret_cast<void**>(&dev.tickets), g_tickets) != cudaSuccess) {
    cudaGetLastError();
    dev.tickets = nullptr;
    return nullptr;
  }
  const auto at = dev.streams.find(id);
  if (at != dev.streams.end()) return dev.tickets + at->second;
  const int slot = static_cast<int>(dev.streams.size());
  if (slot >= kTickets) return nullptr;
  dev.streams[id] = slot;
  return dev.tickets + slot;
}

adaf_status launch_mean(LossArgs a, int op, int32_t dtype, cudaStream_t s) {
  unsigned* const ticket = a.tokens > 0 && a.tokens <= kFewTokens ? stream_ticket(s) : nullptr;
  if (ticket != nullptr) {
    a.ticket = ticket;
    a.count = nullptr;
  } else {
    const adaf_status st = launch(kSlotCount, k_loss_count, 1, kCountThreads, 0, 1, false, s, a, op);
    if (st != ADAF_OK || a.tokens == 0) return st;
  }
  return op == kPolicy ? launch_rows<kPolicy>(a, dtype, s) : launch_rows<kDistill>(a, dtype, s);
}

#define LOSS_CHECK(expr)                 \
  do {                                   \
    const adaf_status st_ = (expr);      \
    if (st_ != ADAF_OK) return st_;      \
  } while (0)

adaf_status check_out(const float* p, const char* name, bool optional) {
  if (p == nullptr) return optional ? ADAF_OK : invalid(std::string(name) + " is NULL");
  return aligned(p, 4) ? ADAF_OK : invalid(std::string(name) + " is not element-aligned");
}

}  // namespace

extern "C" {

adaf_status loss_workspace_size(int64_t tokens, int64_t pairs, size_t* bytes) {
  if (bytes == nullptr) return invalid("bytes is NULL");
  Layout L;
  LOSS_CHECK(layout(tokens, pairs, &L));
  *bytes = L.bytes;
  return ADAF_OK;
}

adaf_status loss_token_logprobs(const loss_logits* x, const loss_targets* y, float* logp, float* stats, void* stream) {
  LOSS_CHECK(check_logits(x));
  LOSS_CHECK(check_targets(*x, y));
  if (x->batch * x->seq == 0) return ADAF_OK;
  LOSS_CHECK(check_out(logp, "logp", false));
  if (stats != nullptr && !aligned(stats, 8)) return invalid("stats is not 8-byte aligned");
  LossArgs a = base_args(*x, y, nullptr);
  a.logp = logp;
  a.stats = reinterpret_cast<float2*>(stats);
  return launch_forward(a, x->dtype, static_cast<cudaStream_t>(stream));
}

adaf_status loss_token_logprobs_backward(const loss_logits* x, const loss_targets* y, const float* stats,
                                         const loss_rows* grad_logp, const loss_grad* grad, void* stream) {
  LOSS_CHECK(check_logits(x));
  LOSS_CHECK(check_targets(*x, y));
  LOSS_CHECK(check_grad(*x, grad, false));
  if (x->batch * x->seq == 0) return ADAF_OK;
  if (stats == nullptr || !aligned(stats, 8)) return invalid("stats is NULL or not 8-byte aligned");
  if (grad_logp == nullptr) return invalid("grad_logp is NULL");
  LOSS_CHECK(check_rows(*x, *grad_logp, "grad_logp", 4, false));
  LossArgs a = base_args(*x, y, grad);
  a.stats = reinterpret_cast<float2*>(const_cast<float*>(stats));
  a.dlogp = rows_of(*grad_logp);
  return launch_grad(a, x->dtype, static_cast<cudaStream_t>(stream));
}

adaf_status loss_policy(const loss_logits* x, const loss_targets* y, const loss_policy_args* args,
                        const loss_grad* grad, float* loss, float* logp, float* token_loss, void* workspace,
                        size_t workspace_bytes, void* stream) {
  LOSS_CHECK(check_logits(x));
  LOSS_CHECK(check_targets(*x, y));
  if (args == nullptr) return invalid("args is NULL");
  if (!std::isfinite(args->clip_low) || args->clip_low < 0.0 || args->clip_low > 1.0)
    return invalid("invalid clip_low (needs 0 <= clip_low <= 1)");
  if (!std::isfinite(args->clip_high) || args->clip_high < 0.0) return invalid("invalid clip_high (needs clip_high >= 0)");
  if (!std::isfinite(args->kl_coef) || args->kl_coef < 0.0) return invalid("invalid kl_coef (needs kl_coef >= 0)");
  if (x->batch * x->seq > 0) {
    LOSS_CHECK(check_rows(*x, args->advantages, "advantages", 4, false));
    LOSS_CHECK(check_rows(*x, args->old_logp, "old_logp", 4, true));
    if (args->ref_logp.p == nullptr && args->kl_coef != 0.0) return invalid("kl_coef needs ref_logp");
    LOSS_CHECK(check_rows(*x, args->ref_logp, "ref_logp", 4, true));
    LOSS_CHECK(check_rows(*x, args->weights, "weights", 4, true));
  }
  LOSS_CHECK(check_grad(*x, grad, true));
  LOSS_CHECK(check_out(loss, "loss", false));
  LOSS_CHECK(check_out(logp, "logp", true));
  LOSS_CHECK(check_out(token_loss, "token_loss", true));
  Layout L;
  LOSS_CHECK(layout(x->batch * x->seq, 0, &L));
  LOSS_CHECK(check_workspace(workspace, workspace_bytes, L));
  LossArgs a = base_args(*x, y, grad);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.loss = loss;
  a.logp = logp;
  a.token_loss = token_loss;
  a.count = reinterpret_cast<int*>(ws);
  a.ticket = reinterpret_cast<unsigned*>(ws + 8);
  a.part = reinterpret_cast<Sum*>(ws + L.off_part);
  a.adv = rows_of(args->advantages);
  a.old = rows_of(args->old_logp);
  a.ref = rows_of(args->ref_logp);
  a.weights = rows_of(args->weights);
  a.lo = static_cast<float>(1.0 - args->clip_low);
  a.hi = static_cast<float>(1.0 + args->clip_high);
  a.kl = static_cast<float>(args->kl_coef);
  return launch_mean(a, kPolicy, x->dtype, static_cast<cudaStream_t>(stream));
}

adaf_status loss_preference(const loss_logits* x, const loss_targets* y, const loss_preference_args* args,
                            const loss_grad* grad, float* loss, float* pair_loss, float* rewards, float* logp,
                            void* workspace, size_t workspace_bytes, void* stream) {
  LOSS_CHECK(check_logits(x));
  LOSS_CHECK(check_targets(*x, y));
  if (args == nullptr) return invalid("args is NULL");
  if (args->pairs < 1) return invalid("pairs must be >= 1");
  if (args->kind != LOSS_PREFERENCE_SIGMOID && args->kind != LOSS_PREFERENCE_HINGE &&
      args->kind != LOSS_PREFERENCE_SQUARED)
    return invalid("unknown kind");
  if (!std::isfinite(args->beta) || args->beta <= 0.0) return invalid("invalid beta (needs beta > 0)");
  if (!std::isfinite(args->label_smoothing) || args->label_smoothing < 0.0 || args->label_smoothing >= 0.5)
    return invalid("invalid label_smoothing (needs 0 <= label_smoothing < 0.5)");
  if (args->label_smoothing != 0.0 && args->kind != LOSS_PREFERENCE_SIGMOID)
    return invalid("label_smoothing is for the sigmoid kind only");
  if (!std::isfinite(args->margin)) return invalid("invalid margin");
  if (args->seq_offsets != nullptr) {
    if (args->offsets_dtype != LOSS_INT32 && args->offsets_dtype != LOSS_INT64)
      return invalid("seq_offsets: unknown dtype");
    if (!aligned(args->seq_offsets, index_size(args->offsets_dtype))) return invalid("seq_offsets is not element-aligned");
    if (x->batch != 1) return invalid("seq_offsets needs batch = 1");
  } else if (x->batch != 2 * args->pairs) {
    return invalid("batch must be 2 * pairs (chosen sequences, then rejected ones)");
  }
  if (x->batch * x->seq > 0) LOSS_CHECK(check_rows(*x, args->ref_logp, "ref_logp", 4, true));
  LOSS_CHECK(check_grad(*x, grad, true));
  LOSS_CHECK(check_out(loss, "loss", false));
  LOSS_CHECK(check_out(pair_loss, "pair_loss", true));
  LOSS_CHECK(check_out(rewards, "rewards", true));
  LOSS_CHECK(check_out(logp, "logp", true));
  Layout L;
  LOSS_CHECK(layout(x->batch * x->seq, args->pairs, &L));
  LOSS_CHECK(check_workspace(workspace, workspace_bytes, L));
  LossArgs a = base_args(*x, y, grad);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.loss = loss;
  a.pair_loss = pair_loss;
  a.rewards = rewards;
  a.logp = logp != nullptr ? logp : reinterpret_cast<float*>(ws + L.off_logp);
  a.stats = reinterpret_cast<float2*>(ws + L.off_stats);
  a.coef_out = reinterpret_cast<float*>(ws + L.off_coef);
  a.pair_part = reinterpret_cast<float*>(ws + L.off_pair);
  a.pairs = args->pairs;
  a.ref = rows_of(args->ref_logp);
  a.offsets = args->seq_offsets;
  a.odt = args->offsets_dtype;
  a.kind = args->kind;
  a.average = args->average;
  a.beta = static_cast<float>(args->beta);
  a.smooth = static_cast<float>(args->label_smoothing);
  a.margin = static_cast<float>(args->margin);
  a.ticket = reinterpret_cast<unsigned*>(ws + 8);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.tokens > 0) {
    LOSS_CHECK(launch_forward(a, x->dtype, s));
  } else {
    const cudaError_t e = cudaMemsetAsync(a.ticket, 0, sizeof(unsigned), s);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  }
  LOSS_CHECK(launch(kSlotPair, k_loss_pair, a.pairs, kPairThreads, 0, 1, a.tokens > 0, s, a));
  if (a.g == nullptr || a.tokens == 0) return ADAF_OK;
  a.coef = a.coef_out;
  return launch_grad(a, x->dtype, s);
}

adaf_status loss_distill(const loss_logits* x, const loss_distill_args* args, const loss_grad* grad, float* loss,
                         float* token_loss, void* workspace, size_t workspace_bytes, void* stream) {
  LOSS_CHECK(check_logits(x));
  if (args == nullptr) return invalid("args is NULL");
  if (args->top_k < 1 || args->top_k > LOSS_MAX_TOP_K) return invalid("top_k must be 1 .. 1024");
  if (args->ids_dtype != LOSS_INT32 && args->ids_dtype != LOSS_INT64) return invalid("ids: unknown dtype");
  if (args->values_dtype != ADAF_FLOAT32 && args->values_dtype != ADAF_BFLOAT16) return invalid("values: unknown dtype");
  if (x->batch * x->seq > 0) {
    const loss_rows ids{args->ids, args->ids_stride_b, args->ids_stride_s};
    const loss_rows values{args->values, args->values_stride_b, args->values_stride_s};
    LOSS_CHECK(check_rows(*x, ids, "ids", index_size(args->ids_dtype), false));
    LOSS_CHECK(check_rows(*x, values, "values", dtype_size(args->values_dtype), false));
    LOSS_CHECK(check_rows(*x, args->lse, "lse", 4, true));
    LOSS_CHECK(check_rows(*x, args->mask, "mask", 1, true));
    LOSS_CHECK(check_rows(*x, args->weights, "weights", 4, true));
  }
  LOSS_CHECK(check_grad(*x, grad, true));
  LOSS_CHECK(check_out(loss, "loss", false));
  LOSS_CHECK(check_out(token_loss, "token_loss", true));
  Layout L;
  LOSS_CHECK(layout(x->batch * x->seq, 0, &L));
  LOSS_CHECK(check_workspace(workspace, workspace_bytes, L));
  LossArgs a = base_args(*x, nullptr, grad);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.loss = loss;
  a.token_loss = token_loss;
  a.count = reinterpret_cast<int*>(ws);
  a.ticket = reinterpret_cast<unsigned*>(ws + 8);
  a.part = reinterpret_cast<Sum*>(ws + L.off_part);
  a.ids = args->ids;
  a.idt = args->ids_dtype;
  a.isb = args->ids_stride_b;
  a.iss = args->ids_stride_s;
  a.tv = args->values;
  a.tdt = args->values_dtype;
  a.tsb = args->values_stride_b;
  a.tss = args->values_stride_s;
  a.top_k = args->top_k;
  a.lse = rows_of(args->lse);
  a.mask = rows_of(args->mask);
  a.weights = rows_of(args->weights);
  return launch_mean(a, kDistill, x->dtype, static_cast<cudaStream_t>(stream));
}

void loss_debug_stall_copies(int32_t on) { t_stall = on != 0; }

adaf_status loss_profile_enable(int32_t on) {
  std::lock_guard<std::mutex> lock(g_mu);
  g_profile = on != 0;
  return ADAF_OK;
}

adaf_status loss_profile_read(double* ms, int64_t* launches, int32_t n) {
  std::lock_guard<std::mutex> lock(g_mu);
  adaf_status st = ADAF_OK;
  for (ProfRecord& r : g_prof) {
    float el = 0.f;
    cudaError_t e = cudaEventSynchronize(r.stop);
    if (e == cudaSuccess) e = cudaEventElapsedTime(&el, r.start, r.stop);
    if (e != cudaSuccess && st == ADAF_OK) st = cuda_fail(e, "profile event");
    if (r.slot < n) {
      if (ms) ms[r.slot] += el;
      if (launches) launches[r.slot] += 1;
    }
    cudaEventDestroy(r.start);
    cudaEventDestroy(r.stop);
  }
  g_prof.clear();
  return st;
}

int32_t loss_num_kernels(void) { return kNumKernels; }

const char* loss_kernel_name(int32_t k) { return (k >= 0 && k < kNumKernels) ? kKernelNames[k] : ""; }

}  // extern "C"
