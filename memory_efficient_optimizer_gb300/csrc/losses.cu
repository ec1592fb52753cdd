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
//   k_loss_finish   sum of the tokens' (or pairs') losses in a fixed order
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

constexpr int kRowThreads = 256;
constexpr int kTile = 8192;        // values of a row between two looks at the teacher's entries
constexpr int kFinishThreads = 1024;
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
  float* part;                    // [tokens]: w l
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

struct Soft {
  float m, s, top;  // largest value, sum of terms (of the words not listed, for distill), sum over the listed words
};
__device__ __forceinline__ Soft join(const Soft& p, const Soft& q, float c) {
  Soft r;
  r.m = fmaxf(p.m, q.m);
  const float sh = shift_of(r.m);
  const float fp = term(p.m, sh, c), fq = term(q.m, sh, c);
  r.s = p.s * fp + q.s * fq;
  r.top = p.top * fp + q.top * fq;
  return r;
}
__device__ __forceinline__ Soft block_join(Soft v, float c, Soft* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Soft w;
    w.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    w.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    w.top = __shfl_xor_sync(0xffffffffu, v.top, o);
    v = join(v, w, c);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  Soft t = red[0];
  for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) t = join(t, red[w], c);
  return t;
}

// ---- counted tokens ------------------------------------------------------------
__global__ void __launch_bounds__(kFinishThreads) k_loss_count(const __grid_constant__ LossArgs a, int op) {
  __shared__ double red[32];
  int n = 0;
  for (int64_t t = threadIdx.x; t < a.tokens; t += kFinishThreads) {
    const int b = static_cast<int>(t / a.seq), s = static_cast<int>(t % a.seq);
    n += counted(a, op, b, s);
  }
  const double total = block_sum(n, red);  // exact: below 2^53
  if (threadIdx.x == 0) *a.count = static_cast<int64_t>(total);
}

// ---- the operators' scalars -----------------------------------------------------
// Loss of a token and its derivative with respect to logp.
struct Token {
  float loss, d;
};
__device__ __forceinline__ Token policy_token(const LossArgs& a, float logp, int b, int s) {
  const float adv = row_value(a.adv, b, s);
  const float r = expf(logp - (a.old.p == nullptr ? logp : row_value(a.old, b, s)));
  const float raw = r * adv;
  const float cut = fminf(fmaxf(r, a.lo), a.hi) * adv;
  Token t;
  const bool free = raw <= cut || isnan(raw);
  t.loss = free ? -raw : -cut;
  t.d = free ? -raw : 0.f;
  if (a.kl != 0.f) {
    const float far = row_value(a.ref, b, s) - logp;
    const float e = expm1f(far);
    t.loss += a.kl * (e - far);
    t.d -= a.kl * e;
  }
  return t;
}

template <typename T>
__device__ __forceinline__ void zero_row(T* g, int n) {
  for (int j = threadIdx.x; j < n; j += blockDim.x) narrow(g[j], 0.f);
}

// ---- one row -----------------------------------------------------------------
template <typename T, int OP>
__global__ void __launch_bounds__(kRowThreads) k_loss_row(const __grid_constant__ LossArgs a) {
  __shared__ Soft red[kRowThreads / 32];
  __shared__ double dred[32];
  __shared__ uint32_t listed[OP == kDistill ? kTile / 32 : 1];
  __shared__ int32_t id[OP == kDistill ? LOSS_MAX_TOP_K : 1];
  __shared__ float pk[OP == kDistill ? LOSS_MAX_TOP_K : 1];
  __shared__ float xk[OP == kDistill ? LOSS_MAX_TOP_K : 1];
  __shared__ int bad, entries;
  const int row = blockIdx.x, b = row / a.seq, s = row % a.seq;
  const T* x = static_cast<const T*>(a.x) + b * a.xsb + s * a.xss;
  T* g = a.g == nullptr ? nullptr : static_cast<T*>(a.g) + b * a.gsb + s * a.gss;
  const int V = a.vocab, tid = threadIdx.x;

  if (!counted(a, OP, b, s)) {
    if (g != nullptr) zero_row(g, V);
    if (tid == 0) {
      if (a.logp != nullptr) a.logp[row] = 0.f;
      if (a.token_loss != nullptr) a.token_loss[row] = 0.f;
      if (a.stats != nullptr) a.stats[row] = make_float2(0.f, 0.f);
      if (a.part != nullptr) a.part[row] = 0.f;
    }
    return;
  }

  float sum_p = 0.f, rest = 0.f;  // distill: sum of p, the teacher's mass on other words
  if (OP == kDistill) {
    // The teacher's probabilities.  p and rest are the same in every thread.
    if (tid == 0) bad = entries = 0;
    __syncthreads();
    Soft t{-INFINITY, 0.f, 0.f};
    for (int k = tid; k < a.top_k; k += kRowThreads) {
      const int64_t e = b * a.isb + s * a.iss + k, f = b * a.tsb + s * a.tss + k;
      int64_t i = load_index(a.ids, a.idt, e);
      if (i != -1 && (i < 0 || i >= V)) {
        bad = 1;
        i = -1;
      }
      float v = a.tdt == ADAF_BFLOAT16 ? widen(static_cast<const __nv_bfloat16*>(a.tv)[f])
                                       : static_cast<const float*>(a.tv)[f];
      if (i == -1) v = -INFINITY;
      if (i >= 0) atomicAdd(&entries, 1);
      id[k] = static_cast<int>(i);
      pk[k] = v;
      xk[k] = i == -1 ? 0.f : widen(x[i]);
      t = join(t, Soft{v, i == -1 || v == -INFINITY ? 0.f : 1.f, 0.f}, a.c);
    }
    t = block_join(t, a.c, red);
    const float lse = a.lse.p == nullptr ? 0.f : row_value(a.lse, b, s);
    double sp = 0.0;
    for (int k = tid; k < a.top_k; k += kRowThreads) {
      // renormalised: exp((t - max) / T) / sum; with lse: exp(t / T - lse)
      const float p = id[k] < 0 ? 0.f
                      : a.lse.p == nullptr ? (t.s == 0.f ? 0.f : term(pk[k], shift_of(t.m), a.c) / t.s)
                                           : expf(pk[k] * a.inv_t - lse);
      pk[k] = p;
      sp += p;
    }
    sum_p = static_cast<float>(block_sum(sp, dred));
    if (a.lse.p != nullptr && entries < V) rest = fmaxf(0.f, 1.f - sum_p);
    if (isnan(sum_p)) rest = sum_p;
  }

  // m and s, with the listed words apart: their sum is not taken out of the
  // whole one again, so a small rest keeps its precision.
  Soft v{-INFINITY, 0.f, 0.f};
  for (int j0 = 0; j0 < V; j0 += kTile) {
    if (OP == kDistill) {
      for (int w = tid; w < kTile / 32; w += kRowThreads) listed[w] = 0;
      __syncthreads();
      for (int k = tid; k < a.top_k; k += kRowThreads) {
        const unsigned at = static_cast<unsigned>(id[k] - j0);
        if (id[k] >= 0 && at < kTile) {
          const uint32_t bit = 1u << (at & 31);
          if (atomicOr(&listed[at >> 5], bit) & bit) bad = 1;
        }
      }
      __syncthreads();
    }
    const int j1 = min(V, j0 + kTile);
    for (int j = j0 + tid; j < j1; j += kRowThreads) {
      const float xj = widen(x[j]);
      const float m = fmaxf(v.m, xj), sh = shift_of(m);
      const float f = term(v.m, sh, a.c), e = term(xj, sh, a.c);
      const bool on = OP == kDistill && (listed[(j - j0) >> 5] >> ((j - j0) & 31) & 1);
      v.s = v.s * f + (on ? 0.f : e);
      v.top = v.top * f + (on ? e : 0.f);
      v.m = m;
    }
    if (OP == kDistill) __syncthreads();
  }
  v = block_join(v, a.c, red);
  const float m = v.m, sum = v.s + v.top;
  float nan = m == -INFINITY || m == INFINITY ? NAN : 0.f;  // a row without a distribution

  float k_all, k_at;  // gradient: k_all exp((x - m) / T), and k_at more at the target
  int64_t y = -1;
  if (OP != kDistill) {
    y = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
    if (y < 0 || y >= V) {
      nan = NAN;
      y = -1;
    }
    const float logp = y < 0 ? NAN : (widen(x[y]) - m) * a.inv_t - logf(sum) + nan;
    if (tid == 0) {
      if (a.logp != nullptr) a.logp[row] = logp;
      if (a.stats != nullptr) a.stats[row] = make_float2(m + nan, sum + nan);
    }
    if (OP == kLogprobs) return;
    const Token t = policy_token(a, logp, b, s);
    const float w = a.weights.p != nullptr ? row_value(a.weights, b, s)
                                           : 1.f / static_cast<float>(*a.count);
    if (tid == 0) {
      if (a.token_loss != nullptr) a.token_loss[row] = t.loss;
      a.part[row] = a.weights.p != nullptr ? w * t.loss : t.loss;
    }
    k_at = w * a.gscale * a.inv_t * t.d;
    k_all = -k_at / sum;
  } else {
    const float log_s = logf(sum);
    if (bad) nan = NAN;
    double l = 0.0;
    for (int k = tid; k < a.top_k; k += kRowThreads)
      if (pk[k] != 0.f) l += pk[k] * (logf(pk[k]) - ((xk[k] - m) * a.inv_t - log_s));
    l = block_sum(l, dred);
    if (rest > 0.f) l += rest * (logf(rest) - (logf(v.s) - log_s));
    const float t2 = 1.f / (a.inv_t * a.inv_t);
    const float loss = static_cast<float>(l) * t2 + nan;
    const float w = a.weights.p != nullptr ? row_value(a.weights, b, s)
                                           : 1.f / static_cast<float>(*a.count);
    if (tid == 0) {
      if (a.token_loss != nullptr) a.token_loss[row] = loss;
      a.part[row] = a.weights.p != nullptr ? w * loss : loss;
    }
    // off the list q (P + u) - u q / (rest of q); on it q (P + u) - p
    k_at = w * a.gscale / a.inv_t + nan;
    k_all = k_at * ((sum_p + rest) / sum - (rest > 0.f ? rest / v.s : 0.f));
  }
  if (g == nullptr) return;
  const float at_value = OP == kDistill ? 0.f : k_all * (y < 0 ? NAN : term(widen(x[y]), m, a.c)) + k_at;
  __syncthreads();  // the target's logit is read before it may be written over
  for (int j = tid; j < V; j += kRowThreads) narrow(g[j], j == y ? at_value : k_all * term(widen(x[j]), m, a.c));
  if (OP == kDistill) {
    __syncthreads();  // the listed words' values replace those written above
    const float on = (sum_p + rest) / sum;
    for (int k = tid; k < a.top_k; k += kRowThreads)
      if (id[k] >= 0) narrow(g[id[k]], k_at * (on * term(xk[k], m, a.c) - pk[k]));
  }
}

// ---- gradient rows from kept statistics ------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_loss_grad(const __grid_constant__ LossArgs a) {
  const int row = blockIdx.x, b = row / a.seq, s = row % a.seq;
  const T* x = static_cast<const T*>(a.x) + b * a.xsb + s * a.xss;
  T* g = static_cast<T*>(a.g) + b * a.gsb + s * a.gss;
  const int64_t y0 = load_index(a.y.p, a.ydt, b * a.y.sb + s * a.y.ss);
  if (y0 == a.ignore) {
    zero_row(g, a.vocab);
    return;
  }
  const float2 st = a.stats[row];
  const float d = (a.coef != nullptr ? a.coef[row] : row_value(a.dlogp, b, s)) * a.gscale * a.inv_t;
  const bool inside = y0 >= 0 && y0 < a.vocab;
  const float k_all = inside ? -d / st.y : NAN;
  for (int j = threadIdx.x; j < a.vocab; j += kRowThreads) {
    const float e = k_all * term(widen(x[j]), st.x, a.c);
    narrow(g[j], j == y0 ? e + d : e);
  }
}

// ---- a pair's loss ---------------------------------------------------------------
__global__ void __launch_bounds__(kRowThreads) k_loss_pair(const __grid_constant__ LossArgs a) {
  __shared__ double red[32];
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
    for (int64_t t = from[h] + threadIdx.x; t < to[h]; t += kRowThreads) {
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
    if (a.rewards != nullptr) {
      a.rewards[pair] = static_cast<float>(a.beta * D[0]);
      a.rewards[pair + a.pairs] = static_cast<float>(a.beta * D[1]);
    }
  }
  for (int q = 0; q < 2; ++q) {
    double c = (q == 0 ? dh : -dh) / static_cast<double>(a.pairs);
    if (a.average) c = n[q] > 0.0 ? c / n[q] : 0.0;
    for (int64_t t = from[q] + threadIdx.x; t < to[q]; t += kRowThreads) a.coef_out[t] = static_cast<float>(c);
  }
}

// ---- the loss ------------------------------------------------------------------
__global__ void __launch_bounds__(kFinishThreads) k_loss_finish(const __grid_constant__ LossArgs a) {
  __shared__ double red[32];
  double v = 0.0;
  if (a.pairs > 0) {
    for (int64_t i = threadIdx.x; i < a.pairs; i += kFinishThreads) v += a.pair_part[i];
  } else {
    for (int64_t i = threadIdx.x; i < a.tokens; i += kFinishThreads) v += a.part[i];
  }
  v = block_sum(v, red);
  if (threadIdx.x == 0) {
    double n = 1.0;
    if (a.pairs > 0) n = static_cast<double>(a.pairs);
    else if (a.weights.p == nullptr) n = static_cast<double>(*a.count);
    *a.loss = n > 0.0 ? static_cast<float>(v / n) : 0.f;
  }
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
  size_t off_count = 0, off_part = 0, off_stats = 0, off_logp = 0, off_coef = 0, off_pair = 0, bytes = 0;
};
adaf_status layout(int64_t tokens, int64_t pairs, Layout* L) {
  if (tokens < 0 || pairs < 0) return invalid("tokens or pairs < 0");
  if (tokens > kMaxTokens || pairs > kMaxTokens / 2)
    return fail(ADAF_ERR_UNSUPPORTED, "tokens must be below 2^31, pairs below 2^30");
  size_t o = 0;
  const size_t n = static_cast<size_t>(tokens);
  L->off_count = o; o = round_up(o + 64, 256);
  L->off_part = o;  o = round_up(o + sizeof(float) * n, 256);
  if (pairs > 0) {
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

const char* const kKernelNames[] = {"k_loss_count", "k_loss_row", "k_loss_grad", "k_loss_pair", "k_loss_finish"};
enum Slot { kSlotCount = 0, kSlotRow, kSlotGrad, kSlotPair, kSlotFinish, kNumKernels };
struct ProfRecord {
  int slot;
  cudaEvent_t start, stop;
};
std::mutex g_mu;
bool g_profile = false;
std::vector<ProfRecord> g_prof;

// Launches through f(); under profiling between two events.
template <typename F>
adaf_status launch(int slot, cudaStream_t s, F f) {
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
  f();
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, kKernelNames[slot]);
  if (prof) {
    if ((e = cudaEventRecord(rec.stop, s)) != cudaSuccess) return cuda_fail(e, "profile event");
    std::lock_guard<std::mutex> lock(g_mu);
    g_prof.push_back(rec);
  }
  return ADAF_OK;
}

template <int OP>
adaf_status launch_rows(const LossArgs& a, int32_t dtype, cudaStream_t s) {
  return launch(kSlotRow, s, [&] {
    if (dtype == ADAF_BFLOAT16) k_loss_row<__nv_bfloat16, OP><<<a.tokens, kRowThreads, 0, s>>>(a);
    else k_loss_row<float, OP><<<a.tokens, kRowThreads, 0, s>>>(a);
  });
}
adaf_status launch_grad(const LossArgs& a, int32_t dtype, cudaStream_t s) {
  return launch(kSlotGrad, s, [&] {
    if (dtype == ADAF_BFLOAT16) k_loss_grad<__nv_bfloat16><<<a.tokens, kRowThreads, 0, s>>>(a);
    else k_loss_grad<float><<<a.tokens, kRowThreads, 0, s>>>(a);
  });
}
adaf_status launch_finish(const LossArgs& a, cudaStream_t s) {
  return launch(kSlotFinish, s, [&] { k_loss_finish<<<1, kFinishThreads, 0, s>>>(a); });
}
// The loss of no tokens: 0, by the finish kernel with nothing to sum.
adaf_status launch_mean(const LossArgs& a, int op, int32_t dtype, cudaStream_t s) {
  adaf_status st = ADAF_OK;
  st = launch(kSlotCount, s, [&] { k_loss_count<<<1, kFinishThreads, 0, s>>>(a, op); });
  if (st != ADAF_OK) return st;
  if (a.tokens > 0) st = op == kPolicy ? launch_rows<kPolicy>(a, dtype, s) : launch_rows<kDistill>(a, dtype, s);
  return st == ADAF_OK ? launch_finish(a, s) : st;
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
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.tokens > 0) {
    // A token outside every sequence (bad offsets) has coefficient 0.
    const cudaError_t e = cudaMemsetAsync(a.coef_out, 0, sizeof(float) * static_cast<size_t>(a.tokens), s);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    LOSS_CHECK(launch_rows<kLogprobs>(a, x->dtype, s));
  }
  LOSS_CHECK(launch(kSlotPair, s, [&] {
    k_loss_pair<<<static_cast<unsigned>(a.pairs), kRowThreads, 0, s>>>(a);
  }));
  LOSS_CHECK(launch_finish(a, s));
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
