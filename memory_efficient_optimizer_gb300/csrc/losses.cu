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
//   k_loss_grad     gradient rows from kept m, s and the tokens' coefficients
//   k_loss_pair     a pair's sums over tokens, its loss and its coefficients
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "adafactor_internal.h"
#include "losses.h"

namespace {

constexpr int kMaxThreads = 512;   // of a CTA of k_loss_row
constexpr int kGradThreads = 256;
constexpr int kPairThreads = 256;
constexpr int kCountThreads = 1024;
constexpr int kGroup = 256;        // tokens of a partial sum of the loss
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxVocab = (int64_t{1} << 30) - 1;
constexpr int64_t kMaxTokens = (int64_t{1} << 31) - 1;

enum Op : int { kLogprobs = 0, kPolicy = 1, kDistill = 2 };

struct Rows {
  const void* p;
  int64_t sb, ss;
};

// Arguments of every kernel of this file.
struct LossArgs {
  const void* x;
  void* g;                        // NULL: no gradient
  int64_t xsb, xss, gsb, gss;
  int32_t seq, tokens, vocab;
  float c, inv_t, gscale;         // log2(e) / T, 1 / T, scale of the gradient
  Rows y;
  int32_t ydt;
  int64_t ignore;
  float* loss;
  float* logp;
  float* token_loss;
  float2* stats;                  // [tokens]: m, s
  int64_t* count;                 // counted tokens
  float* part;                    // [tokens]: w l, or l
  double* group_part;             // [ceil(tokens / kGroup)]
  unsigned* tickets;              // [1 + ceil(tokens / kGroup)]; k_loss_pair: [1]
  int32_t vecs_per_cta;           // k_loss_row: vectors of a row for a CTA
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
  double beta, smooth, margin;
  float* pair_loss;
  float* rewards;
  double* pair_part;              // [pairs]
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
// exp((x - m) / T).  The difference is taken before the scaling: it is exact
// or rounded once however large x and m are, and two values at the type's
// lowest give 0, not inf - inf.  m is finite or NaN here.
__device__ __forceinline__ float term(float x, float m, float c) { return ex2((x - m) * c); }
// The shift of a part whose largest value is -inf is 0: its terms are 0.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ bool counted(const LossArgs& a, int op, int b, int s) {
  if (op == kDistill)
    return a.mask.p == nullptr || static_cast<const uint8_t*>(a.mask.p)[b * a.mask.sb + s * a.mask.ss] != 0;
  return load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss) != a.ignore;
}

// ---- sums over a block, in a fixed order ---------------------------------------
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += red[w];
  return t;
}

// ---- vectors of a row ----------------------------------------------------------
// A row is read as aligned 16-byte vectors.  Vector i of a row that starts
// `lead` values after a 16-byte boundary holds its values i kN - lead ..; the
// first and the last may reach past the row and are then loaded value by
// value, with -inf outside.
template <typename T> constexpr int kN = 16 / static_cast<int>(sizeof(T));
constexpr int kV = 8;               // vectors a thread keeps: 128 bytes of the row
constexpr uint32_t kNegInf2 = 0xff80ff80u;
template <typename T> constexpr uint32_t kNegInf = sizeof(T) == 2 ? kNegInf2 : 0xff800000u;

template <typename T>
struct Row {
  const T* x;
  int lead, n, vecs;  // values before the row in its first vector, values, vectors
  __device__ __forceinline__ Row(const T* p, int vocab) : x(p), n(vocab) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    vecs = (lead + n + kN<T> - 1) / kN<T>;
  }
  __device__ __forceinline__ bool whole(int i) const {
    const int e = i * kN<T> - lead;
    return e >= 0 && e + kN<T> <= n;
  }
  __device__ __forceinline__ bool ragged() const { return lead != 0 || vecs * kN<T> != lead + n; }
  __device__ __forceinline__ const uint4* at(int i) const {
    return reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x) & ~uintptr_t{15}) + i;
  }
};

__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

// Value j of a vector, replaced.
template <typename T>
__device__ __forceinline__ void put(uint4& w, int j, uint32_t bits) {
  uint32_t* q = &w.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (sizeof(T) == 4) {
      if (j == k) q[k] = bits;
    } else {
      if (j == 2 * k) q[k] = (q[k] & 0xffff0000u) | bits;
      if (j == 2 * k + 1) q[k] = (q[k] & 0xffffu) | (bits << 16);
    }
  }
}

// Vectors i = first + k step < last of a row.
template <typename T>
__device__ __forceinline__ void load_tile(uint4 (&w)[kV], const Row<T>& r, int first, int step, int last) {
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int i = first + k * step;
    w[k] = make_uint4(kNegInf<T>, kNegInf<T>, kNegInf<T>, kNegInf<T>);
    if (i < last && r.whole(i)) w[k] = __ldcs(r.at(i));
  }
  if (r.ragged()) {
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const int i = first + k * step;
      if (i < last && !r.whole(i)) {
#pragma unroll
        for (int j = 0; j < kN<T>; ++j) {
          const int e = i * kN<T> - r.lead + j;
          if (e >= 0 && e < r.n) put<T>(w[k], j, bits_of(r.x[e]));
        }
      }
    }
  }
}

__device__ __forceinline__ float2 pair_of(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// Values of a vector, two at a time.
template <typename T>
__device__ __forceinline__ float2 pair_at(const uint4& w, int j) {
  const uint32_t* q = &w.x;
  if (sizeof(T) == 4) return make_float2(__uint_as_float(q[2 * j]), __uint_as_float(q[2 * j + 1]));
  return pair_of(q[j]);
}
__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }
// term() of two values.
__device__ __forceinline__ float2 terms(float2 x, float m, float c) {
  const float2 z = __fmul2_rn(__fadd2_rn(x, twice(-m)), twice(c));
  return make_float2(ex2(z.x), ex2(z.y));
}

// Largest value of a tile over the warp (NaN is left out: it shows in the sum).
template <typename T>
__device__ __forceinline__ float tile_max(const uint4 (&w)[kV]) {
  float m;
  if (sizeof(T) == 2) {
    __nv_bfloat162 a;
    memcpy(&a, &w[0].x, 4);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const uint32_t q[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        __nv_bfloat162 b;
        memcpy(&b, &q[t], 4);
        a = __hmax2(a, b);
      }
    }
    m = fmaxf(__low2float(a), __high2float(a));
  } else {
    m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kV; ++k)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(w[k].x), __uint_as_float(w[k].y)),
                         fmaxf(__uint_as_float(w[k].z), __uint_as_float(w[k].w))));
  }
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
  return r;
}

// Adds the terms of a tile; with `listed` (a byte a vector, a bit a value) the
// listed words' terms go to `top`.
template <typename T, bool LISTED>
__device__ __forceinline__ void tile_sum(const uint4 (&w)[kV], float m, float c, const uint8_t* listed, int step,
                                         float& sum, float& top) {
  float2 acc = make_float2(0.f, 0.f), acc2 = acc;
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    if (LISTED) {
      const uint32_t on = listed[k * step];
      if (on != 0) {
#pragma unroll
        for (int j = 0; j < kN<T> / 2; ++j) {
          const float2 e = terms(pair_at<T>(w[k], j), m, c);
          sum += (on >> (2 * j) & 1 ? 0.f : e.x) + (on >> (2 * j + 1) & 1 ? 0.f : e.y);
          top += (on >> (2 * j) & 1 ? e.x : 0.f) + (on >> (2 * j + 1) & 1 ? e.y : 0.f);
        }
        continue;
      }
    }
#pragma unroll
    for (int j = 0; j < kN<T> / 2; j += 2) {
      acc = __fadd2_rn(acc, terms(pair_at<T>(w[k], j), m, c));
      acc2 = __fadd2_rn(acc2, terms(pair_at<T>(w[k], j + 1), m, c));
    }
  }
  sum += (acc.x + acc.y) + (acc2.x + acc2.y);
}

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
  __device__ __forceinline__ void zero(int rank, int ranks) const {
    const int vecs = (lead + n + kN<T> - 1) / kN<T>, per = (vecs + ranks - 1) / ranks;
    const int last = min(vecs, (rank + 1) * per);
    for (int i = rank * per + threadIdx.x; i < last; i += blockDim.x) {
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
// scale exp((x - m) / T) of a vector, rounded to its type.
template <typename T>
__device__ __forceinline__ uint4 scaled_terms(const uint4& w, float m, float c, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < kN<T> / 2; ++j) {
    const float2 v = __fmul2_rn(terms(pair_at<T>(w, j), m, c), twice(scale));
    if (sizeof(T) == 4) {
      o[2 * j] = __float_as_uint(v.x);
      o[2 * j + 1] = __float_as_uint(v.y);
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
// The gradient's vectors of a tile: scale exp((x - m) / T), and `at` in place
// of the value y.
template <typename T>
__device__ __forceinline__ void store_tile(const uint4 (&w)[kV], const Row<T>& r, const GradRow<T>& g, int first, int step,
                                           int last, float m, float c, float scale, int y, float at) {
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int i = first + k * step;
    if (__any_sync(0xffffffffu, i < last)) {
      const int e0 = i * kN<T> - r.lead;
      uint4 o = scaled_terms<T>(w[k], m, c, scale);
      const unsigned j = static_cast<unsigned>(y - e0);
      if (y >= 0 && j < static_cast<unsigned>(kN<T>)) put<T>(o, static_cast<int>(j), rounded_bits<T>(at));
      g.store(o, e0, i < last);
    }
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
__device__ __forceinline__ double warp_sum(double v) {
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
// Also clears the tickets of the sum over tokens.
__global__ void __launch_bounds__(kCountThreads) k_loss_count(const __grid_constant__ LossArgs a, int op) {
  __shared__ double red[32];
  let_next_start();
  const int groups = (a.tokens + kGroup - 1) / kGroup;
  for (int i = threadIdx.x; i <= groups; i += kCountThreads) a.tickets[i] = 0;
  int n = 0;
#pragma unroll 8
  for (uint32_t t = threadIdx.x; t < static_cast<uint32_t>(a.tokens); t += kCountThreads)
    n += counted(a, op, static_cast<int>(t / static_cast<uint32_t>(a.seq)), static_cast<int>(t % static_cast<uint32_t>(a.seq)));
  const double total = block_sum(n, red);  // exact: below 2^53
  if (threadIdx.x == 0) {
    *a.count = static_cast<int64_t>(total);
    if (a.tokens == 0) *a.loss = 0.f;
  }
}

// A token's share of the loss is in a.part: the warp that brings the last of a
// group of kGroup tokens sums the group, the one that brings the last group
// sums the groups, each in a fixed order.
__device__ __forceinline__ void add_to_loss(const LossArgs& a, int row, float share) {
  const int lane = threadIdx.x & 31;
  const int group = row / kGroup, groups = (a.tokens + kGroup - 1) / kGroup;
  const int members = min(kGroup, a.tokens - group * kGroup);
  int last = 0;
  if (lane == 0) {
    a.part[row] = share;
    __threadfence();
    last = atomicAdd(&a.tickets[1 + group], 1u) == static_cast<unsigned>(members - 1);
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  double v = 0.0;
#pragma unroll
  for (int k = 0; k < kGroup / 32; ++k)
    if (k * 32 + lane < members) v += __ldcg(a.part + group * kGroup + k * 32 + lane);
  v = warp_sum(v);
  last = 0;
  if (lane == 0) {
    a.group_part[group] = v;
    __threadfence();
    last = atomicAdd(&a.tickets[0], 1u) == static_cast<unsigned>(groups - 1);
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  v = 0.0;
  for (int k = lane; k < groups; k += 32) v += __ldcg(a.group_part + k);
  v = warp_sum(v);
  if (lane == 0) {
    const double n = a.weights.p == nullptr ? static_cast<double>(*a.count) : 1.0;
    *a.loss = n > 0.0 ? static_cast<float>(v / n) : 0.f;
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
  const float r = expf(logp - (a.old.p == nullptr ? logp : in.old));
  const float raw = r * in.adv;
  const float cut = fminf(fmaxf(r, a.lo), a.hi) * in.adv;
  Token t;
  const bool free = raw <= cut || isnan(raw);
  t.loss = free ? -raw : -cut;
  t.d = free ? -raw : 0.f;
  if (a.kl != 0.f) {
    const float far = in.ref - logp;
    const float e = expm1f(far);
    t.loss += a.kl * (e - far);
    t.d -= a.kl * e;
  }
  return t;
}

// Shared memory of a CTA of k_loss_row: the parts of all warps of the cluster
// and, for distill, the list's bits (a byte a vector of the tile), ids,
// probabilities and logits.
__host__ __device__ constexpr int row_shared(bool distill, int warps, int cluster, int top_k) {
  const int parts = warps * cluster * static_cast<int>(sizeof(float4));
  return distill ? parts + warps * 32 * kV + 12 * ((top_k + 3) / 4 * 4) : parts;
}

// ---- one row -----------------------------------------------------------------
// A cluster has a row, a CTA a run of a.vecs_per_cta of its vectors.  LONG:
// more than the threads keep, so the row is read again for the gradient.
template <typename T, int OP, bool LONG>
__global__ void __launch_bounds__(kMaxThreads, 1024 / kMaxThreads) k_loss_row(const __grid_constant__ LossArgs a) {
  extern __shared__ __align__(16) unsigned char shared[];
  __shared__ float4 red[kMaxThreads / 32];
  __shared__ int bad;
  constexpr bool kLists = OP == kDistill;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int step = blockDim.x, warps = step >> 5;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int row = blockIdx.x / ranks, b = row / a.seq, s = row % a.seq;
  float4* parts = reinterpret_cast<float4*>(shared);
  uint8_t* listed = shared + warps * ranks * sizeof(float4);
  int32_t* id = reinterpret_cast<int32_t*>(listed + step * kV);
  const int kpad = (a.top_k + 3) / 4 * 4;
  float* pk = reinterpret_cast<float*>(id + kpad);
  float* xk = pk + kpad;

  const Row<T> r(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss, a.vocab);
  const GradRow<T> g(a.g == nullptr ? nullptr : static_cast<T*>(a.g) + b * a.gsb + s * a.gss, a.vocab, r.lead);

  if (OP == kLogprobs) {
    // k_loss_pair may begin as these CTAs end; its ticket is cleared here
    let_next_start();
    if (a.tickets != nullptr && blockIdx.x == 0 && tid == 0) a.tickets[0] = 0;
  }
  int64_t y64 = 0;
  bool in_loss;
  if (kLists) {
    in_loss = counted(a, OP, b, s);
  } else {
    y64 = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
    in_loss = y64 != a.ignore;
  }
  if (!in_loss) {
    if (a.g != nullptr) g.zero(rank, ranks);
    if (rank == 0 && tid == 0) {
      if (a.logp != nullptr) a.logp[row] = 0.f;
      if (a.token_loss != nullptr) a.token_loss[row] = 0.f;
      if (a.stats != nullptr) a.stats[row] = make_float2(0.f, 0.f);
      if (a.coef_out != nullptr) a.coef_out[row] = 0.f;
    }
    if (OP != kLogprobs && rank == 0 && warp == 0) {
      wait_for_previous();
      add_to_loss(a, row, 0.f);
    }
    return;
  }
  if (ranks > 1) cluster_arrive();  // shared memory of the others may be written once they have all begun

  const int v0 = rank * a.vecs_per_cta, v1 = min(r.vecs, v0 + a.vecs_per_cta);
  uint4 w[kV];
  if (!LONG) load_tile<T>(w, r, v0 + tid, step, v1);

  // Per-token values, while the row is on its way.
  int y = -1;
  float x_at = 0.f, weight = 0.f;
  PolicyIn in{0.f, 0.f, 0.f};
  if (!kLists && y64 >= 0 && y64 < a.vocab) {
    y = static_cast<int>(y64);
    x_at = widen(r.x[y]);
  }
  if (OP == kPolicy) {
    in.adv = row_value(a.adv, b, s);
    if (a.old.p != nullptr) in.old = row_value(a.old, b, s);
    if (a.kl != 0.f) in.ref = row_value(a.ref, b, s);
  }
  if (OP != kLogprobs && a.weights.p != nullptr) weight = row_value(a.weights, b, s);

  // The teacher: p[k] = pk[k] pscale, their sum and the rest.
  float pscale = 1.f, sum_p = 0.f, rest = 0.f;
  if (kLists) {
    if (tid == 0) bad = 0;
    if (!LONG)
      for (int i = tid; i < step * kV / 4; i += step) reinterpret_cast<uint32_t*>(listed)[i] = 0;
    float top = -INFINITY;
    int entries = 0, wrong = 0;
    for (int k = tid; k < a.top_k; k += step) {
      int64_t i = load_index(a.ids, a.idt, b * a.isb + s * a.iss + k);
      const int64_t f = b * a.tsb + s * a.tss + k;
      float v = a.tdt == ADAF_BFLOAT16 ? widen(static_cast<const __nv_bfloat16*>(a.tv)[f])
                                       : static_cast<const float*>(a.tv)[f];
      if (i < 0 || i >= a.vocab) {
        wrong |= i != -1;
        i = -1;
        v = -INFINITY;
      } else {
        ++entries;
      }
      id[k] = static_cast<int>(i);
      pk[k] = v;
      top = fmaxf(top, v);
    }
    top = warp_max(top);
    wrong = __any_sync(0xffffffffu, wrong);
    entries = __reduce_add_sync(0xffffffffu, entries);
    if (lane == 0) red[warp] = make_float4(top, __int_as_float(entries), __int_as_float(wrong), 0.f);
    __syncthreads();
    entries = wrong = 0;
    for (int q = 0; q < warps; ++q) {
      top = fmaxf(top, red[q].x);
      entries += __float_as_int(red[q].y);
      wrong |= __float_as_int(red[q].z);
    }
    if (wrong && tid == 0) bad = 1;
    const float sh = shift_of(top), lse = a.lse.p == nullptr ? 0.f : row_value(a.lse, b, s);
    float sum = 0.f;
    for (int k = tid; k < a.top_k; k += step) {
      const int i = id[k];
      float p = 0.f, x = 0.f;
      if (i >= 0) {
        // renormalised: exp((t - max) / T) / sum; with lse: exp(t / T - lse)
        p = a.lse.p == nullptr ? term(pk[k], sh, a.c) : expf(pk[k] * a.inv_t - lse);
        const int at = (i + r.lead) / kN<T> - v0;
        const bool mine = at >= 0 && at < v1 - v0;
        if (mine || rank == 0) x = widen(r.x[i]);
        if (!LONG && mine) {
          const uint32_t bit = 1u << ((at & 3) * 8 + (i + r.lead) % kN<T>);
          if (atomicOr(reinterpret_cast<uint32_t*>(listed) + (at >> 2), bit) & bit) bad = 1;
        }
      }
      pk[k] = p;
      xk[k] = x;
      sum += p;
    }
    sum = warp_sum(sum);
    __syncthreads();  // red is read, the bits are set
    if (lane == 0) red[warp].w = sum;
    __syncthreads();
    sum = 0.f;
    for (int q = 0; q < warps; ++q) sum += red[q].w;
    if (a.lse.p == nullptr) {
      pscale = sum == 0.f ? 0.f : 1.f / sum;
      sum_p = sum == 0.f ? 0.f : sum == sum ? 1.f : sum;
    } else {
      sum_p = sum;
      if (sum != sum) rest = sum;
      else if (entries < a.vocab) rest = fmaxf(0.f, 1.f - sum);
    }
  }

  // m and the sum of the terms; the listed words' apart, so that a small rest
  // is a sum of its own and keeps its precision.
  float m = -INFINITY, sum = 0.f, top = 0.f;
  if (!LONG) {
    m = tile_max<T>(w);
    tile_sum<T, kLists>(w, shift_of(m), a.c, listed + tid, step, sum, top);
  } else {
    for (int i0 = v0; i0 < v1; i0 += step * kV) {
      if (kLists) {
        __syncthreads();
        for (int i = tid; i < step * kV / 4; i += step) reinterpret_cast<uint32_t*>(listed)[i] = 0;
        __syncthreads();
        for (int k = tid; k < a.top_k; k += step) {
          const int at = (id[k] + r.lead) / kN<T> - i0;
          if (id[k] >= 0 && at >= 0 && at < min(v1 - i0, step * kV)) {
            const uint32_t bit = 1u << ((at & 3) * 8 + (id[k] + r.lead) % kN<T>);
            if (atomicOr(reinterpret_cast<uint32_t*>(listed) + (at >> 2), bit) & bit) bad = 1;
          }
        }
        __syncthreads();
      }
      load_tile<T>(w, r, i0 + tid, step, v1);
      const float m2 = fmaxf(m, tile_max<T>(w));
      const float sh = shift_of(m2), f = term(m, sh, a.c);
      sum *= f;
      top *= f;
      tile_sum<T, kLists>(w, sh, a.c, listed + tid, step, sum, top);
      m = m2;
    }
  }
  sum = warp_sum(sum);
  if (kLists) top = warp_sum(top);

  // Every warp's part to every CTA of the cluster; each warp joins them all.
  float wrong = 0.f;
  if (kLists) {
    __syncthreads();
    wrong = bad ? NAN : 0.f;
  }
  const float4 part = make_float4(m, sum, top, wrong);
  if (ranks > 1) {
    cluster_wait();
    if (lane < ranks) store_remote(parts + rank * warps + warp, lane, part);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  } else {
    if (lane == 0) parts[warp] = part;
    __syncthreads();
  }
  const int all = warps * ranks;
  m = -INFINITY;
  for (int q = lane; q < all; q += 32) m = fmaxf(m, parts[q].x);
  m = warp_max(m);
  sum = top = wrong = 0.f;
  for (int q = lane; q < all; q += 32) {
    const float4 p = parts[q];
    const float f = term(p.x, shift_of(m), a.c);
    sum += p.y * f;
    top += p.z * f;
    wrong += p.w;
  }
  sum = warp_sum(sum);
  float off = sum;  // the terms of the words that are not listed
  if (kLists) {
    sum += warp_sum(top);
    wrong = warp_sum(wrong);
  }
  if (m == -INFINITY || m == INFINITY) wrong = NAN;  // a row without a distribution

  float scale, at = 0.f;  // gradient: scale exp((x - m) / T), at the target `at`
  float lead = 0.f, on = 0.f;
  const bool first = rank == 0 && warp == 0;
  if (!kLists) {
    const float logp = y < 0 ? NAN : (x_at - m) * a.inv_t - logf(sum) + wrong;
    if (first && lane == 0) {
      if (a.logp != nullptr) a.logp[row] = logp;
      if (a.stats != nullptr) a.stats[row] = make_float2(m + wrong, sum + wrong);
      if (a.coef_out != nullptr) a.coef_out[row] = 0.f;
    }
    if (OP == kLogprobs) return;
    const Token t = policy_token(a, logp, in);
    wait_for_previous();
    if (a.weights.p == nullptr) weight = 1.f / static_cast<float>(*a.count);
    if (first) {
      if (lane == 0 && a.token_loss != nullptr) a.token_loss[row] = t.loss;
      add_to_loss(a, row, a.weights.p != nullptr ? weight * t.loss : t.loss);
    }
    const float k_at = weight * a.gscale * a.inv_t * t.d;
    scale = -k_at / sum;
    at = scale * (y < 0 ? NAN : term(x_at, m, a.c)) + k_at;
  } else {
    wait_for_previous();
    if (a.weights.p == nullptr) weight = 1.f / static_cast<float>(*a.count);
    if (first) {
      const float log_s = logf(sum);
      float l = 0.f;
      for (int k = lane; k < a.top_k; k += 32) {
        const float p = pk[k] * pscale;
        if (p != 0.f) l += p * (logf(p) - ((xk[k] - m) * a.inv_t - log_s));
      }
      l = warp_sum(l);
      if (rest > 0.f) l += rest * (logf(rest) - (logf(off) - log_s));
      const float loss = l / (a.inv_t * a.inv_t) + wrong;
      if (lane == 0 && a.token_loss != nullptr) a.token_loss[row] = loss;
      add_to_loss(a, row, a.weights.p != nullptr ? weight * loss : loss);
    }
    // off the list q (P + u) - u q / (rest of q); on it q (P + u) - p
    lead = weight * a.gscale / a.inv_t + wrong;
    on = (sum_p + rest) / sum;
    scale = lead * (on - (rest > 0.f ? rest / off : 0.f));
  }
  if (a.g == nullptr) return;
  if (!LONG) {
    store_tile<T>(w, r, g, v0 + tid, step, v1, m, a.c, scale, y, at);
  } else {
    for (int i0 = v0; i0 < v1; i0 += step * kV) {
      load_tile<T>(w, r, i0 + tid, step, v1);
      store_tile<T>(w, r, g, i0 + tid, step, v1, m, a.c, scale, y, at);
    }
  }
  if (kLists) {
    __syncthreads();  // the listed words' values replace those written above
    for (int k = tid; k < a.top_k; k += step) {
      const int i = id[k], v = (i + r.lead) / kN<T>;
      if (i >= 0 && v >= v0 && v < v1) narrow(g.g[i], lead * (on * term(xk[k], m, a.c) - pk[k] * pscale));
    }
  }
}

// ---- gradient rows from kept statistics ------------------------------------------
// A CTA has a tile of a row; the last rows come first: of what the forward
// pass read they are the ones most likely still in L2.
template <typename T>
__global__ void __launch_bounds__(kGradThreads, 1024 / kGradThreads) k_loss_grad(const __grid_constant__ LossArgs a) {
  const int row = a.tokens - 1 - static_cast<int>(blockIdx.x / a.tiles), tile = blockIdx.x % a.tiles;
  const int b = row / a.seq, s = row % a.seq;
  const Row<T> r(static_cast<const T*>(a.x) + b * a.xsb + s * a.xss, a.vocab);
  const GradRow<T> g(static_cast<T*>(a.g) + b * a.gsb + s * a.gss, a.vocab, r.lead);
  const int64_t y0 = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
  if (a.coef != nullptr) wait_for_previous();
  if (y0 == a.ignore) {
    g.zero(tile, a.tiles);
    return;
  }
  const int first = tile * kGradThreads * kV + threadIdx.x;
  const int last = min(r.vecs, (tile + 1) * kGradThreads * kV);
  uint4 w[kV];
  load_tile<T>(w, r, first, kGradThreads, last);
  const float2 st = a.stats[row];
  const float d = (a.coef != nullptr ? a.coef[row] : row_value(a.dlogp, b, s)) * a.gscale * a.inv_t;
  const bool inside = y0 >= 0 && y0 < a.vocab;
  const float scale = inside ? -d / st.y : NAN;
  const int y = inside ? static_cast<int>(y0) : -1;
  float at = 0.f;
  // `at` matters to the thread that holds the target, which alone writes it:
  // the gradient may lie over the logits.
  const int v = (y + r.lead) / kN<T>;
  const bool mine = inside && v >= tile * kGradThreads * kV && v < last;
  if (mine) at = scale * term(widen(r.x[y]), st.x, a.c) + d;
  store_tile<T>(w, r, g, first, kGradThreads, last, st.x, a.c, scale, mine ? y : -1, at);
}

// ---- a pair's loss ---------------------------------------------------------------
__global__ void __launch_bounds__(kPairThreads) k_loss_pair(const __grid_constant__ LossArgs a) {
  __shared__ double red[32];
  __shared__ int last;
  let_next_start();
  wait_for_previous();
  const int64_t pair = blockIdx.x;
  double D[2];
  int64_t from[2], to[2];
  double n[2];
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
    double sum = 0.0, cnt = 0.0;
    for (int64_t t = from[h] + threadIdx.x; t < to[h]; t += kPairThreads) {
      const int b = static_cast<int>(t / a.seq), s = static_cast<int>(t % a.seq);
      if (!counted(a, kLogprobs, b, s)) continue;
      sum += a.logp[t];
      if (a.ref.p != nullptr) sum -= row_value(a.ref, b, s);
      cnt += 1.0;
    }
    D[h] = block_sum(sum, red);
    n[h] = block_sum(cnt, red);
    if (a.average) D[h] = n[h] > 0.0 ? D[h] / n[h] : 0.0;
  }
  const double h = D[0] - D[1];
  double loss, dh;  // and its derivative with respect to h
  if (a.kind == LOSS_PREFERENCE_SIGMOID) {
    const double z = a.beta * h - a.margin, e = exp(-fabs(z)), l = log1p(e);
    const double neg = l + fmax(-z, 0.0), pos = l + fmax(z, 0.0);  // -ln s(z), -ln s(-z)
    const double sig = z >= 0.0 ? 1.0 / (1.0 + e) : e / (1.0 + e);
    const double sig_neg = z >= 0.0 ? e / (1.0 + e) : 1.0 / (1.0 + e);
    loss = (1.0 - a.smooth) * neg + a.smooth * pos;
    dh = a.beta * (a.smooth * sig - (1.0 - a.smooth) * sig_neg);
  } else if (a.kind == LOSS_PREFERENCE_HINGE) {
    const double z = 1.0 + a.margin - a.beta * h;
    loss = z > 0.0 || isnan(z) ? z : 0.0;
    dh = z > 0.0 || isnan(z) ? -a.beta + 0.0 * z : 0.0;
  } else {
    const double z = h - 1.0 / (2.0 * a.beta) - a.margin;
    loss = z * z;
    dh = 2.0 * z;
  }
  if (!ok) loss = dh = NAN;
  if (threadIdx.x == 0) {
    if (a.pair_loss != nullptr) a.pair_loss[pair] = static_cast<float>(loss);
    a.pair_part[pair] = loss;
    __threadfence();
    last = atomicAdd(a.tickets, 1u) == static_cast<unsigned>(a.pairs - 1);
    if (a.rewards != nullptr) {
      a.rewards[pair] = static_cast<float>(a.beta * D[0]);
      a.rewards[pair + a.pairs] = static_cast<float>(a.beta * D[1]);
    }
  }
  for (int q = 0; q < 2; ++q) {
    double c = (q == 0 ? dh : -dh) / static_cast<double>(a.pairs);
    if (a.average) c = n[q] > 0.0 ? c / n[q] : 0.0;
    for (int64_t t = from[q] + threadIdx.x; t < to[q]; t += kPairThreads) a.coef_out[t] = static_cast<float>(c);
  }
  __syncthreads();
  if (!last) return;
  // the last pair to come sums them all, in order
  __threadfence();
  double v = 0.0;
  for (int64_t k = threadIdx.x; k < a.pairs; k += kPairThreads) v += __ldcg(a.pair_part + k);
  v = block_sum(v, red);
  if (threadIdx.x == 0) *a.loss = static_cast<float>(v / static_cast<double>(a.pairs));
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
  if (x->vocab > kMaxVocab) return fail(ADAF_ERR_UNSUPPORTED, "logits: vocab must be below 2^30");
  if (x->batch > kMaxTokens || x->seq > kMaxTokens || x->batch * x->seq > kMaxTokens)
    return fail(ADAF_ERR_UNSUPPORTED, "logits: batch * seq must be below 2^31");
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
  size_t off_count = 0, off_tickets = 0, off_groups = 0, off_part = 0, off_stats = 0, off_logp = 0, off_coef = 0, off_pair = 0, bytes = 0;
};
adaf_status layout(int64_t tokens, int64_t pairs, Layout* L) {
  if (tokens < 0 || pairs < 0) return invalid("tokens or pairs < 0");
  if (tokens > kMaxTokens || pairs > kMaxTokens / 2)
    return fail(ADAF_ERR_UNSUPPORTED, "tokens must be below 2^31, pairs below 2^30");
  size_t o = 0;
  const size_t n = static_cast<size_t>(tokens);
  const size_t groups = (n + kGroup - 1) / kGroup;
  L->off_count = o;   o += 64;
  L->off_tickets = o; o = round_up(o + sizeof(unsigned) * (1 + groups), 256);
  if (pairs == 0) {
    L->off_groups = o; o = round_up(o + sizeof(double) * groups, 256);
    L->off_part = o;   o = round_up(o + sizeof(float) * n, 256);
  } else {
    L->off_stats = o; o = round_up(o + sizeof(float2) * n, 256);
    L->off_logp = o;  o = round_up(o + sizeof(float) * n, 256);
    L->off_coef = o;  o = round_up(o + sizeof(float) * n, 256);
    L->off_pair = o;  o = round_up(o + sizeof(double) * static_cast<size_t>(pairs), 256);
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
  a.seq = static_cast<int32_t>(x.seq);
  a.tokens = static_cast<int32_t>(x.batch * x.seq);
  a.vocab = static_cast<int32_t>(x.vocab);
  a.c = static_cast<float>(1.4426950408889634 / x.temperature);
  a.inv_t = static_cast<float>(1.0 / x.temperature);
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

const char* const kKernelNames[] = {"k_loss_count", "k_loss_row", "k_loss_grad", "k_loss_pair"};
enum Slot { kSlotCount = 0, kSlotRow, kSlotGrad, kSlotPair, kNumKernels };
struct ProfRecord {
  int slot;
  cudaEvent_t start, stop;
};
std::mutex g_mu;
bool g_profile = false;
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

static int envi(const char* n, int d) { const char* v = getenv(n); return v ? atoi(v) : d; }
static int kRowThreads() { return envi("MEO_T", 512); }
static int kFewCtas() { return envi("MEO_F", 304); }
// How a row is cut: CTAs, threads of each, vectors of each; `again`: the
// threads cannot keep the row and read it twice.
struct Cut {
  int cluster, threads, vecs;
  bool again;
};
Cut cut_row(int64_t tokens, int64_t vocab, size_t es) {
  const int64_t per = 16 / static_cast<int64_t>(es), vecs = (vocab + 2 * per - 2) / per;  // the most, at any alignment
  auto threads_of = [&](int64_t c) { return ((vecs + c - 1) / c + kV * 32 - 1) / (kV * 32) * 32; };
  int64_t c = 1;
  const int64_t most = kRowThreads();
  while (c < kMaxCluster && threads_of(c) > most) c *= 2;
  while (c < kMaxCluster && tokens * c < kFewCtas() && threads_of(c) > 64) c *= 2;
  if (tokens * c > kMaxTokens) c = 1;
  Cut cut;
  cut.cluster = static_cast<int>(c);
  cut.threads = static_cast<int>(std::min<int64_t>(threads_of(c), kMaxThreads));
  cut.vecs = static_cast<int>((vecs + c - 1) / c);
  cut.again = cut.vecs > cut.threads * kV;
  return cut;
}

template <int OP>
adaf_status launch_rows(LossArgs a, int32_t dtype, cudaStream_t s) {
  const Cut cut = cut_row(a.tokens, a.vocab, dtype_size(dtype));
  a.vecs_per_cta = cut.vecs;
  const int shared = row_shared(OP == kDistill, cut.threads / 32, cut.cluster, a.top_k);
  const bool bf16 = dtype == ADAF_BFLOAT16;
  void (*const kernel)(LossArgs) =
      cut.again ? (bf16 ? k_loss_row<__nv_bfloat16, OP, true> : k_loss_row<float, OP, true>)
                : (bf16 ? k_loss_row<__nv_bfloat16, OP, false> : k_loss_row<float, OP, false>);
  return launch(kSlotRow, kernel, static_cast<int64_t>(a.tokens) * cut.cluster, cut.threads, shared, cut.cluster,
                OP != kLogprobs, s, a);
}
adaf_status launch_grad(LossArgs a, int32_t dtype, cudaStream_t s) {
  const int64_t per = 16 / static_cast<int64_t>(dtype_size(dtype)), vecs = (a.vocab + 2 * per - 2) / per;
  a.tiles = static_cast<int32_t>((vecs + kGradThreads * kV - 1) / (kGradThreads * kV));
  const int64_t grid = static_cast<int64_t>(a.tokens) * a.tiles;
  if (grid > kMaxTokens) return fail(ADAF_ERR_UNSUPPORTED, "gradient of more than 2^31 tiles");
  return launch(kSlotGrad, dtype == ADAF_BFLOAT16 ? k_loss_grad<__nv_bfloat16> : k_loss_grad<float>, grid, kGradThreads,
                0, 1, a.coef != nullptr, s, a);
}
adaf_status launch_mean(const LossArgs& a, int op, int32_t dtype, cudaStream_t s) {
  const adaf_status st = launch(kSlotCount, k_loss_count, 1, kCountThreads, 0, 1, false, s, a, op);
  if (st != ADAF_OK || a.tokens == 0) return st;
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
  return launch_rows<kLogprobs>(a, x->dtype, static_cast<cudaStream_t>(stream));
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
  a.count = reinterpret_cast<int64_t*>(ws + L.off_count);
  a.part = reinterpret_cast<float*>(ws + L.off_part);
  a.group_part = reinterpret_cast<double*>(ws + L.off_groups);
  a.tickets = reinterpret_cast<unsigned*>(ws + L.off_tickets);
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
  a.pair_part = reinterpret_cast<double*>(ws + L.off_pair);
  a.pairs = args->pairs;
  a.ref = rows_of(args->ref_logp);
  a.offsets = args->seq_offsets;
  a.odt = args->offsets_dtype;
  a.kind = args->kind;
  a.average = args->average;
  a.beta = args->beta;
  a.smooth = args->label_smoothing;
  a.margin = args->margin;
  a.tickets = reinterpret_cast<unsigned*>(ws + L.off_tickets);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.tokens > 0) {
    LOSS_CHECK(launch_rows<kLogprobs>(a, x->dtype, s));
  } else {
    const cudaError_t e = cudaMemsetAsync(a.tickets, 0, sizeof(unsigned), s);
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
  a.count = reinterpret_cast<int64_t*>(ws + L.off_count);
  a.part = reinterpret_cast<float*>(ws + L.off_part);
  a.group_part = reinterpret_cast<double*>(ws + L.off_groups);
  a.tickets = reinterpret_cast<unsigned*>(ws + L.off_tickets);
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
