// Multi-tensor Muon step and its orthogonalisation for sm_103a: the C ABI of
// include/muon.h.
//
// Matrices of one shape (with the smaller side as m, the larger as n; a taller
// matrix is worked on transposed) go through a sequence of launches together:
//
//   k_muon_moment   m = mu m + g; sum u^2 of every matrix, in parts
//   k_muon_pack     x = u / max(||u||, eps), in the layout of the products
//   then per step of the iteration three products (tc_gemm.cuh), which do
//   everything else in their endings:
//   k_muon_gram     A = x x^T          (only tiles on or above the diagonal)
//   k_muon_poly     B = b A + c A A    (the same)
//   k_muon_apply    x = a x + B x; the last one updates p, or writes the result
//
// Numbers.  The factors of the products are fp16, scaled by powers of two: an
// element of x is at most its largest singular value, 1.21, so x 2^15 fits, and
// so do A 2^15 and B 2^14, and at any size the usual elements are far above the
// subnormal range (1 / sqrt(mn) 2^15 is 8 at 4096 x 4096).  What rounding does
// depends on where it enters:
//   - rounding of the factors of x x^T, A A and B x acts like a multiplication
//     of x by I + d with small d from the left or the right: directions turn by
//     2^-12 or so, and a small singular value stays as accurate as a large one;
//   - rounding of x where it is carried to the next step adds noise at the level
//     of the large singular values, which the small ones drown in (they grow by
//     3.44 a step, and the noise with them).  So x is carried as hi + lo 2^-11,
//     two fp16 numbers with 22 bits, of which hi is the factor of the products;
//   - as x comes near orthogonal, A comes near a multiple of I, and a rounding of
//     the diagonal would weigh most.  With A = D + F, B = G + E (D, G diagonal,
//     in fp32), A A = F F + D F + F D + D D and a x + B x = (a + G) x + E x: only
//     F and E are rounded and multiplied.
// Against the formula in 64 bits this is 2e-4 to 8e-4 off (2-norms) for flat and
// for decaying spectra alike, where fp16 iterates are 1.3e-3 to 1.2e-2 off and
// bf16 ones 1e-2 to 9e-2.
//
// What bounds it: the tensor cores, for matrices from about 2000 on; (3 m^2 n +
// m^3) 2 / 2 flops a step, half of what plain products of the symmetric A and B
// would take.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "adafactor_internal.h"
#include "muon.h"
#include "tc_host.cuh"

namespace {

using meo::tc::Part;
using meo::tc::Shape;

constexpr int kMaxGroup = 64;                      // matrices of a launch
constexpr int64_t kGroupValues = int64_t{1} << 28;  // and their values, unless one alone has more
constexpr int kMaxParts = 256;                     // of a matrix's sum of squares
constexpr int kPartValues = 8192;                  // values of a part, at least
constexpr int64_t kMaxSide = int64_t{1} << 20;
constexpr float kLoScale = 2048.f, kLoUnscale = 1.f / 2048.f;

enum Flag : unsigned char { kTurned = 1, kBf16 = 2 };   // x is u^T; u is bf16

// A launch's matrices.  u: the gradient, or the matrix to orthogonalise; p: the
// parameter, or the result.
struct Group {
  float* p[kMaxGroup];
  const void* u[kMaxGroup];
  float* mom[kMaxGroup];
  float rate[kMaxGroup];           // p = keep p - rate o
  unsigned char flags[kMaxGroup];
};

struct MuonArgs {
  int32_t m, n, ldx, lda;          // of x, and row lengths of x and of A and B in memory
  int32_t parts;
  int64_t stride_r;                // of u
  float mu, nesterov_mu, eps;      // u = g + nesterov_mu m, or m itself (nesterov_mu < 0)
  float* part;                     // [matrices][kMaxParts]
  __half* hi;
  __half* lo;
  int32_t* status;
  int32_t clear;                   // this launch clears the status word
};

// ---- norm and layout ------------------------------------------------------------------
__device__ __forceinline__ float block_sum(float v, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) v += scratch[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ float value_at(const void* u, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(u)[i]) : static_cast<const float*>(u)[i];
}
__device__ __forceinline__ float4 four_at(const void* u, bool bf16, int64_t i) {
  if (!bf16) return __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(u) + i));
  const uint2 r = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(u) + i));
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float update_of(float g, float m, const MuonArgs& a) {
  return a.nesterov_mu < 0.f ? m : fmaf(a.nesterov_mu, m, g);
}

// One part of a matrix a CTA.  STEP: the momentum is brought up to date too.
// Read 2 or 4 + 4 bytes a value, write 4: bound by memory.
template <bool STEP>
__global__ void __launch_bounds__(256) k_muon_moment(const __grid_constant__ Group grp, const MuonArgs a, int32_t rows, int32_t cols) {
  __shared__ float scratch[8];
  const int b = blockIdx.y;
  if (a.clear != 0 && blockIdx.x == 0 && b == 0 && threadIdx.x == 0) *a.status = 0;
  const bool bf16 = grp.flags[b] & kBf16;
  const void* u = grp.u[b];
  float* mom = grp.mom[b];
  const bool flat = STEP || a.stride_r == cols;
  const int64_t numel = static_cast<int64_t>(rows) * cols;
  const int64_t per = ((numel + a.parts - 1) / a.parts + 3) & ~int64_t{3};
  const int64_t e0 = per * blockIdx.x, e1 = min(numel, e0 + per);
  float sum = 0.f;
  if (flat) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(u) % (bf16 ? 8 : 16) | (STEP ? reinterpret_cast<uintptr_t>(mom) % 16 : 0);
    int64_t tail = e0;
    if (at == 0 && e0 < e1) {
      const int64_t quads = (e1 - e0) >> 2;
      tail = e0 + 4 * quads;
      for (int64_t q = threadIdx.x; q < quads; q += 256) {
        const int64_t i = e0 + 4 * q;
        float4 v = four_at(u, bf16, i);
        if (STEP) {
          float4 m = *reinterpret_cast<const float4*>(mom + i);
          m.x = fmaf(a.mu, m.x, v.x);
          m.y = fmaf(a.mu, m.y, v.y);
          m.z = fmaf(a.mu, m.z, v.z);
          m.w = fmaf(a.mu, m.w, v.w);
          *reinterpret_cast<float4*>(mom + i) = m;
          v = make_float4(update_of(v.x, m.x, a), update_of(v.y, m.y, a), update_of(v.z, m.z, a), update_of(v.w, m.w, a));
        }
        sum += (v.x * v.x + v.y * v.y) + (v.z * v.z + v.w * v.w);
      }
    }
    for (int64_t i = tail + threadIdx.x; i < e1; i += 256) {
      float v = value_at(u, bf16, i);
      if (STEP) {
        const float m = fmaf(a.mu, mom[i], v);
        mom[i] = m;
        v = update_of(v, m, a);
      }
      sum += v * v;
    }
  } else {
    for (int64_t i = e0 + threadIdx.x; i < e1; i += 256) {
      const int r = static_cast<int>(i / cols), c = static_cast<int>(i - static_cast<int64_t>(r) * cols);
      const float v = value_at(u, bf16, r * a.stride_r + c);
      sum += v * v;
    }
  }
  sum = block_sum(sum, scratch);
  if (threadIdx.x == 0) a.part[b * kMaxParts + blockIdx.x] = sum;
}

__device__ __forceinline__ void split(float x, __half* hi, __half* lo) {
  *hi = __float2half_rn(x);
  *lo = __float2half_rn((x - __half2float(*hi)) * kLoScale);
}

// x of a matrix, 64 x 64 values a CTA, through shared memory so that both u and
// x are walked along their rows where x is u^T.
template <bool STEP>
__global__ void __launch_bounds__(256) k_muon_pack(const __grid_constant__ Group grp, const MuonArgs a, int32_t rows, int32_t cols) {
  __shared__ float tile[64][65];
  __shared__ float scratch[8];
  const int b = blockIdx.z;
  const float sum = block_sum(static_cast<int>(threadIdx.x) < a.parts ? a.part[b * kMaxParts + threadIdx.x] : 0.f, scratch);
  const float norm = sqrtf(sum);
  // (a norm that is not finite makes x NaN)
  const float scale = norm <= FLT_MAX ? 32768.f / fmaxf(norm, a.eps) : __int_as_float(0x7fc00000);
  const bool bf16 = grp.flags[b] & kBf16, turned = grp.flags[b] & kTurned;
  const void* u = grp.u[b];
  const float* mom = grp.mom[b];
  // rows and cols are those of x; u has them the other way round if turned
  const int ur = turned ? cols : rows, uc = turned ? rows : cols;
  const int r0 = (turned ? blockIdx.x : blockIdx.y) * 64, c0 = (turned ? blockIdx.y : blockIdx.x) * 64;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int r = r0 + (i >> 6), c = c0 + (i & 63);
    float v = 0.f;
    if (r < ur && c < uc) {
      const int64_t at = static_cast<int64_t>(r) * (STEP ? uc : a.stride_r) + c;
      v = value_at(u, bf16, at);
      if (STEP) v = update_of(v, mom[at], a);
      v *= scale;
    }
    tile[i >> 6][i & 63] = v;
  }
  __syncthreads();
  const int x0 = blockIdx.y * 64, y0 = blockIdx.x * 64;   // of x
  __half* const hi = a.hi + static_cast<int64_t>(b) * rows * a.ldx;
  __half* const lo = a.lo + static_cast<int64_t>(b) * rows * a.ldx;
  for (int i = threadIdx.x; i < 64 * 32; i += 256) {
    const int r = i >> 5, c = (i & 31) * 2;
    if (x0 + r >= rows || y0 + c >= a.ldx) continue;
    const float v0 = turned ? tile[c][r] : tile[r][c], v1 = turned ? tile[c + 1][r] : tile[r][c + 1];
    __half2 h, l;
    split(v0, &h.x, &l.x);
    split(v1, &h.y, &l.y);
    const int64_t at = static_cast<int64_t>(x0 + r) * a.ldx + y0 + c;
    *reinterpret_cast<__half2*>(hi + at) = h;
    *reinterpret_cast<__half2*>(lo + at) = l;
  }
}

// ---- endings of the products ------------------------------------------------------------
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t r) { return __half22float2(*reinterpret_cast<const __half2*>(&r)); }

// 32 values of a row of a symmetric matrix s [m][ld] (values beyond column m are 0 and
// go up to ld), and their mirror image in column `row`.
__device__ __forceinline__ void store_symmetric(__half* s, int ld, int m, int row, int col, bool mirror, const float (&v)[32]) {
  uint32_t h[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = pack(v[2 * i], v[2 * i + 1]);
  if (row < m) {
    uint4* const to = reinterpret_cast<uint4*>(s + static_cast<int64_t>(row) * ld + col);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + 8 * i < ld) to[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
  }
  if (mirror) {
    // Two lanes swap halves, so that each stores two values side by side.
    const bool odd = row & 1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // column col + 2i has (mine.low, theirs.low), column col + 2i + 1 the high ones
      const uint32_t other = __shfl_xor_sync(0xffffffffu, h[i], 1);
      const uint32_t pair = odd ? __byte_perm(other, h[i], 0x7632) : __byte_perm(h[i], other, 0x5410);
      const int r = col + 2 * i + (odd ? 1 : 0), c = row & ~1;
      if (r < m && c < ld) *reinterpret_cast<uint32_t*>(s + static_cast<int64_t>(r) * ld + c) = pair;
    }
  }
}

// A = x x^T: F = A without its diagonal (scaled by 2^15), D the diagonal.
struct GramEnd {
  static constexpr bool kSym = true;
  struct Args {
    __half* f;
    float* d;
    int32_t ld;
  };
  static __device__ __forceinline__ void part(const Args& a, const Part& p) {
    __half* const f = a.f + static_cast<int64_t>(p.tile.batch) * p.m * a.ld;
    float* const d = a.d + static_cast<int64_t>(p.tile.batch) * a.ld;
    for (int c = 0; c < p.cols && p.col + c < p.m; c += 32) {
      float v[32];
      p.load(c, v);
      const int diag = p.row - (p.col + c);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[i] *= 0x1p-15f;
        if (i == diag) {
          if (p.row < p.m) d[p.row] = v[i] * 0x1p-15f;
          v[i] = 0.f;
        }
      }
      store_symmetric(f, a.ld, p.m, p.row, p.col + c, p.tile.mirror, v);
    }
  }
};

// B = b A + c A A: E without the diagonal (scaled by 2^14), G the diagonal.
struct PolyEnd {
  static constexpr bool kSym = true;
  struct Args {
    const __half* f;
    const float* d;
    __half* e;
    float* g;
    int32_t ld;
    float b, c;
  };
  static __device__ __forceinline__ void part(const Args& a, const Part& p) {
    const int64_t at = static_cast<int64_t>(p.tile.batch) * p.m * a.ld;
    const float* const d = a.d + static_cast<int64_t>(p.tile.batch) * a.ld;
    const float di = p.row < p.m ? d[p.row] : 0.f;
    for (int c = 0; c < p.cols && p.col + c < p.m; c += 32) {
      const int j0 = p.col + c;
      float v[32];
      p.load(c, v);
      const int diag = p.row - j0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (j0 + 8 * i >= a.ld) {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[8 * i + q] = 0.f;
          continue;
        }
        uint4 r = make_uint4(0, 0, 0, 0);
        if (p.row < p.m) r = *reinterpret_cast<const uint4*>(a.f + at + static_cast<int64_t>(p.row) * a.ld + j0 + 8 * i);
        const float4 d0 = *reinterpret_cast<const float4*>(d + j0 + 8 * i), d1 = *reinterpret_cast<const float4*>(d + j0 + 8 * i + 4);
        const float dj[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 two = unpack(w[q >> 1]);
          const float f = (q & 1) ? two.y : two.x;   // F 2^15
          float& x = v[8 * i + q];                   // (F F) 2^30
          if (8 * i + q == diag) {
            if (p.row < p.m) a.g[static_cast<int64_t>(p.tile.batch) * a.ld + p.row] = fmaf(a.c, fmaf(di, di, x * 0x1p-30f), a.b * di);
            x = 0.f;
          } else {
            x = fmaf(f * 0.5f, fmaf(a.c, di + dj[q], a.b), a.c * (x * 0x1p-16f));
          }
        }
      }
      if (p.row >= p.m) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (j0 + i >= p.m) v[i] = 0.f;
      store_symmetric(a.e + at, a.ld, p.m, p.row, j0, p.tile.mirror, v);
    }
  }
};

// x = (a + G) x + E x.  LAST: the update of p, or the result.
enum Last : int { kNext, kUpdate, kResult };
template <int LAST>
struct ApplyEnd {
  static constexpr bool kSym = false;
  struct Args {
    const __half* hi;
    __half* lo;            // read and written in place: nobody else needs these values
    __half* hi_next;
    const float* g;
    int32_t ldx, lda;
    float a, keep;
    int32_t out_bf16;
    const int32_t* status;
  };
};

__device__ __forceinline__ void applied(const Part& p, int c, const __half* hi, const __half* lo, int64_t at, int ldx, float factor,
                                        float (&v)[32]) {
  p.load(c, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.row < p.m && p.col + c + 8 * i < ldx) {
      const uint4 h = *reinterpret_cast<const uint4*>(hi + at + c + 8 * i), l = *reinterpret_cast<const uint4*>(lo + at + c + 8 * i);
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 x = unpack(hw[q]), y = unpack(lw[q]);
        v[8 * i + 2 * q] = fmaf(factor, fmaf(y.x, kLoUnscale, x.x), v[8 * i + 2 * q] * 0x1p-14f);
        v[8 * i + 2 * q + 1] = fmaf(factor, fmaf(y.y, kLoUnscale, x.y), v[8 * i + 2 * q + 1] * 0x1p-14f);
      }
    }
  }
}

struct NextEnd : ApplyEnd<kNext> {
  static __device__ __forceinline__ void part(const Args& a, const Part& p) {
    const int64_t at = (static_cast<int64_t>(p.tile.batch) * p.m + p.row) * a.ldx + p.col;
    const float factor = a.a + (p.row < p.m ? a.g[static_cast<int64_t>(p.tile.batch) * a.lda + p.row] : 0.f);
    for (int c = 0; c < p.cols && p.col + c < p.n; c += 32) {
      float v[32];
      applied(p, c, a.hi, a.lo, at, a.ldx, factor, v);
      if (p.row >= p.m) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p.col + c + 8 * i >= a.ldx) continue;
        uint32_t h[4], l[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float x = v[8 * i + 2 * q], y = v[8 * i + 2 * q + 1];
          h[q] = pack(x, y);
          const float2 r = unpack(h[q]);
          l[q] = pack((x - r.x) * kLoScale, (y - r.y) * kLoScale);
        }
        *reinterpret_cast<uint4*>(a.hi_next + at + c + 8 * i) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(a.lo + at + c + 8 * i) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  }
};

template <int LAST>
struct LastEnd : ApplyEnd<LAST> {
  struct Args : ApplyEnd<LAST>::Args {
    Group grp;
  };
  static __device__ __forceinline__ void part(const Args& a, const Part& p) {
    if (LAST == kUpdate && (p.bad || *reinterpret_cast<const volatile int32_t*>(a.status) != 0)) return;   // p stays as it is
    const int b = p.tile.batch;
    const int64_t at = (static_cast<int64_t>(b) * p.m + p.row) * a.ldx + p.col;
    const float factor = a.a + (p.row < p.m ? a.g[static_cast<int64_t>(b) * a.lda + p.row] : 0.f);
    const bool turned = a.grp.flags[b] & kTurned;
    const bool wide = !turned && p.n % 8 == 0 && reinterpret_cast<uintptr_t>(a.grp.p[b]) % 16 == 0;
    for (int c = 0; c < p.cols && p.col + c < p.n; c += 32) {
      float v[32];
      applied(p, c, a.hi, a.lo, at, a.ldx, factor, v);
      if (p.row >= p.m) continue;
      const int j0 = p.col + c;
      // value i of p's or the result's memory: along its row, or down its column
      const int64_t to = turned ? static_cast<int64_t>(j0) * p.m + p.row : static_cast<int64_t>(p.row) * p.n + j0;
      const int64_t step = turned ? p.m : 1;
      if (LAST == kUpdate) {
        float* const q = a.grp.p[b] + to;
        const float rate = a.grp.rate[b] * 0x1p-15f;
        if (wide) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (j0 + 4 * i >= p.n) break;
            float4 x = *reinterpret_cast<const float4*>(q + 4 * i);
            x.x = fmaf(-rate, v[4 * i], a.keep * x.x);
            x.y = fmaf(-rate, v[4 * i + 1], a.keep * x.y);
            x.z = fmaf(-rate, v[4 * i + 2], a.keep * x.z);
            x.w = fmaf(-rate, v[4 * i + 3], a.keep * x.w);
            *reinterpret_cast<float4*>(q + 4 * i) = x;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (j0 + i < p.n) q[i * step] = fmaf(-rate, v[i], a.keep * q[i * step]);
        }
      } else if (a.out_bf16) {
        __nv_bfloat16* const q = reinterpret_cast<__nv_bfloat16*>(a.grp.p[b]) + to;
        if (wide) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (j0 + 8 * i >= p.n) break;
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 two = __floats2bfloat162_rn(v[8 * i + 2 * k] * 0x1p-15f, v[8 * i + 2 * k + 1] * 0x1p-15f);
              w[k] = *reinterpret_cast<const uint32_t*>(&two);
            }
            *reinterpret_cast<uint4*>(q + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (j0 + i < p.n) q[i * step] = __float2bfloat16_rn(v[i] * 0x1p-15f);
        }
      } else {
        float* const q = a.grp.p[b] + to;
        if (wide) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (j0 + 4 * i >= p.n) break;
            *reinterpret_cast<float4*>(q + 4 * i) = make_float4(v[4 * i] * 0x1p-15f, v[4 * i + 1] * 0x1p-15f,
                                                                v[4 * i + 2] * 0x1p-15f, v[4 * i + 3] * 0x1p-15f);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (j0 + i < p.n) q[i * step] = v[i] * 0x1p-15f;
        }
      }
    }
  }
};

// ---- host side ------------------------------------------------------------------------
adaf_status fail(adaf_status st, const std::string& msg) { return meo::set_last_error(st, ("muon: " + msg).c_str()); }
adaf_status invalid(const std::string& msg) { return fail(ADAF_ERR_INVALID_ARGUMENT, msg); }
adaf_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(ADAF_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

const char* const kKernelNames[] = {"k_muon_moment", "k_muon_pack", "k_muon_gram", "k_muon_poly", "k_muon_apply"};
constexpr int kNumKernels = 5;
enum Slot { kSlotMoment, kSlotPack, kSlotGram, kSlotPoly, kSlotApply };
meo::tc::Profile g_profile;
thread_local bool t_stall = false;

adaf_status check_iteration(const muon_iteration* it) {
  if (it == nullptr) return invalid("iteration is NULL");
  if (it->steps < 1 || it->steps > MUON_MAX_STEPS) return invalid("steps must be 1 to 16");
  if (!std::isfinite(it->eps) || !(static_cast<float>(it->eps) >= FLT_MIN)) return invalid("eps must be a positive (normal) fp32 number");
  // How far singular values can get, on a grid over what the step before reaches
  // (the products' factors hold a little more than the limits below).
  constexpr int kGrid = 4096;
  double top = 1.0;
  for (int k = 0; k < it->steps; ++k) {
    const double a = it->coef[k][0], b = it->coef[k][1], c = it->coef[k][2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return invalid("coefficients must be finite");
    // over the whole interval that the step before can have reached
    double reach = 0.0, poly = 0.0;
    for (int i = 0; i <= kGrid; ++i) {
      const double x = top * i / kGrid, q = b * x * x + c * x * x * x * x;
      reach = std::max(reach, std::fabs((a + q) * x));
      poly = std::max(poly, std::fabs(q));
    }
    if (poly > 3.9 || reach > 1.9 || std::fabs(a) > 1000.0)
      return invalid("coefficients of step " + std::to_string(k) + " take singular values beyond 1.9, or b s^2 + c s^4 beyond 3.9");
    if (reach < 1e-4) return invalid("coefficients of step " + std::to_string(k) + " take every singular value to 0");
    top = reach;
  }
  return ADAF_OK;
}

adaf_status check_hp(const muon_hparams* hp) {
  if (hp == nullptr) return invalid("hparams is NULL");
  if (!std::isfinite(hp->lr) || hp->lr < 0.0) return invalid("invalid learning rate");
  if (!std::isfinite(hp->momentum) || hp->momentum < 0.0 || hp->momentum >= 1.0) return invalid("invalid momentum (needs 0 <= momentum < 1)");
  if (!std::isfinite(hp->weight_decay) || hp->weight_decay < 0.0) return invalid("invalid weight_decay");
  if (hp->adjust_lr != MUON_ADJUST_ORIGINAL && hp->adjust_lr != MUON_ADJUST_MATCH_RMS) return invalid("unknown adjust_lr");
  return check_iteration(&hp->iteration);
}

// One matrix of the list.
struct Matrix {
  int64_t m, n;
  int64_t rows, cols;
  float* p;
  const void* u;
  float* mom;
  unsigned char flags;
};

adaf_status check_size(int64_t batch, int64_t rows, int64_t cols, const std::string& who) {
  if (batch < 0 || rows < 0 || cols < 0) return invalid(who + "negative size");
  if (batch == 0 || rows == 0 || cols == 0) return ADAF_OK;
  if (rows > kMaxSide || cols > kMaxSide || rows * cols > INT32_MAX)
    return fail(ADAF_ERR_UNSUPPORTED, who + "a side above 2^20 or more than 2^31 - 1 values a matrix");
  if (batch > (1 << 24)) return fail(ADAF_ERR_UNSUPPORTED, who + "more than 2^24 matrices");
  return ADAF_OK;
}

int group_size(int64_t m, int64_t n, int64_t count) {
  return static_cast<int>(std::min<int64_t>({count, kMaxGroup, std::max<int64_t>(1, kGroupValues / (m * n))}));
}

struct Layout {
  size_t part, hi0, hi1, lo, f, e, d, g, bytes;
};
Layout layout(int64_t m, int64_t n, int64_t count) {
  const int64_t ldx = round_up(n, 8), lda = round_up(m, 8);
  Layout L{};
  size_t o = 256;   // the status word
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = static_cast<size_t>(round_up(static_cast<int64_t>(o + bytes), 256));
    return at;
  };
  const size_t x = static_cast<size_t>(count) * m * ldx * 2, s = static_cast<size_t>(count) * m * lda * 2;
  L.part = take(static_cast<size_t>(count) * kMaxParts * 4);
  L.hi0 = take(x);
  L.hi1 = take(x);
  L.lo = take(x);
  L.f = take(s);
  L.e = take(s);
  L.d = take(static_cast<size_t>(count) * lda * 4);
  L.g = take(static_cast<size_t>(count) * lda * 4);
  L.bytes = o;
  return L;
}

// Bytes for all groups of a sorted list of (m, n), one after another in the same memory.
size_t bytes_of(std::vector<std::pair<std::pair<int64_t, int64_t>, int64_t>>& sizes) {
  std::sort(sizes.begin(), sizes.end());
  size_t most = 256;
  for (size_t i = 0; i < sizes.size();) {
    int64_t count = 0;
    size_t j = i;
    for (; j < sizes.size() && sizes[j].first == sizes[i].first; ++j) count += sizes[j].second;
    const int64_t m = sizes[i].first.first, n = sizes[i].first.second;
    most = std::max(most, layout(m, n, group_size(m, n, count)).bytes);
    i = j;
  }
  return most;
}

adaf_status check_tensors(const muon_tensor* tensors, int32_t n, size_t* bytes) {
  if (n < 0) return invalid("n < 0");
  if (n > 0 && tensors == nullptr) return invalid("tensors is NULL");
  std::vector<std::pair<std::pair<int64_t, int64_t>, int64_t>> sizes;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const muon_tensor& t = tensors[i];
    const std::string who = "tensor " + std::to_string(i) + ": ";
    const adaf_status st = check_size(t.batch, t.rows, t.cols, who);
    if (st != ADAF_OK) return st;
    if (t.grad_dtype != ADAF_FLOAT32 && t.grad_dtype != ADAF_BFLOAT16) return invalid(who + "unknown grad_dtype");
    if (t.batch == 0 || t.rows == 0 || t.cols == 0) continue;
    if ((total += t.batch) > (1 << 24)) return fail(ADAF_ERR_UNSUPPORTED, "more than 2^24 matrices");
    sizes.push_back({{std::min(t.rows, t.cols), std::max(t.rows, t.cols)}, t.batch});
  }
  *bytes = sizes.empty() ? 0 : bytes_of(sizes);
  return ADAF_OK;
}

adaf_status check_workspace(const void* ws, size_t have, size_t need) {
  if (ws == nullptr || !aligned(ws, 256)) return invalid("workspace is NULL or not 256-byte aligned");
  if (have < need) return fail(ADAF_ERR_WORKSPACE_TOO_SMALL, "workspace needs " + std::to_string(need) + " bytes");
  return ADAF_OK;
}

// How the launches of a call differ.
struct Call {
  const muon_iteration* it;
  const muon_hparams* hp;      // NULL: orthogonalise
  int64_t stride_r;
  int32_t out_bf16;
  unsigned char* ws;
  cudaStream_t s;
};

template <int CG, int BN, int STAGES, bool B_MN, class End>
cudaError_t product(int slot, const CUtensorMap& a, const CUtensorMap& b, const Shape& s, const typename End::Args& end,
                    cudaStream_t stream) {
  return g_profile.run(slot, stream, [&] { return meo::tc::launch_product<CG, BN, STAGES, false, B_MN, false, End>(a, b, s, end, stream); });
}

#define MUON_TRY(expr, what)                          \
  do {                                                \
    const cudaError_t e_ = (expr);                    \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)

// The iteration on one group; x is packed in hi0, lo.
template <int CG, int BN, int STAGES>
adaf_status iterate(const Call& c, const Layout& L, const Group& grp, int64_t m, int64_t n, int count, float keep) {
  unsigned char* const ws = c.ws;
  const int64_t ldx = round_up(n, 8), lda = round_up(m, 8);
  __half* hi[2] = {reinterpret_cast<__half*>(ws + L.hi0), reinterpret_cast<__half*>(ws + L.hi1)};
  __half* const lo = reinterpret_cast<__half*>(ws + L.lo);
  __half* const f = reinterpret_cast<__half*>(ws + L.f);
  __half* const e = reinterpret_cast<__half*>(ws + L.e);
  float* const d = reinterpret_cast<float*>(ws + L.d);
  float* const g = reinterpret_cast<float*>(ws + L.g);
  CUtensorMap xk[2], xn[2], fk, ek;
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    ok = ok && meo::tc::make_map(&xk[i], hi[i], false, m, n, ldx, count, m * ldx, meo::tc::kBoxK);
    ok = ok && meo::tc::make_map(&xn[i], hi[i], false, m, n, ldx, count, m * ldx, meo::tc::kBoxMN);
  }
  ok = ok && meo::tc::make_map(&fk, f, false, m, m, lda, count, m * lda, meo::tc::kBoxK);
  ok = ok && meo::tc::make_map(&ek, e, false, m, m, lda, count, m * lda, meo::tc::kBoxK);
  if (!ok) return fail(ADAF_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  Shape sq{};
  sq.m = sq.n = static_cast<int32_t>(m);
  sq.batch = count;
  sq.splits = 1;
  sq.group = 8;
  sq.status = reinterpret_cast<int32_t*>(ws);
  sq.stall = t_stall ? 1 : 0;
  for (int k = 0; k < c.it->steps; ++k) {
    const float ca = static_cast<float>(c.it->coef[k][0]), cb = static_cast<float>(c.it->coef[k][1]),
                cc = static_cast<float>(c.it->coef[k][2]);
    Shape s = sq;
    s.k = static_cast<int32_t>(n);
    MUON_TRY((product<CG, BN, STAGES, false, GramEnd>(kSlotGram, xk[k & 1], xk[k & 1], s, {f, d, static_cast<int32_t>(lda)}, c.s)), "k_muon_gram");
    s.k = static_cast<int32_t>(m);
    MUON_TRY((product<CG, BN, STAGES, false, PolyEnd>(kSlotPoly, fk, fk, s, {f, d, e, g, static_cast<int32_t>(lda), cb, cc}, c.s)), "k_muon_poly");
    s.n = static_cast<int32_t>(n);
    ApplyEnd<kNext>::Args next{hi[k & 1], lo, hi[(k + 1) & 1], g, static_cast<int32_t>(ldx), static_cast<int32_t>(lda), ca, keep, c.out_bf16, sq.status};
    if (k + 1 < c.it->steps) {
      MUON_TRY((product<CG, BN, STAGES, true, NextEnd>(kSlotApply, ek, xn[k & 1], s, next, c.s)), "k_muon_apply");
    } else if (c.hp != nullptr) {
      LastEnd<kUpdate>::Args last;
      std::memcpy(static_cast<ApplyEnd<kUpdate>::Args*>(&last), &next, sizeof next);
      last.grp = grp;
      MUON_TRY((product<CG, BN, STAGES, true, LastEnd<kUpdate>>(kSlotApply, ek, xn[k & 1], s, last, c.s)), "k_muon_apply");
    } else {
      LastEnd<kResult>::Args last;
      std::memcpy(static_cast<ApplyEnd<kResult>::Args*>(&last), &next, sizeof next);
      last.grp = grp;
      MUON_TRY((product<CG, BN, STAGES, true, LastEnd<kResult>>(kSlotApply, ek, xn[k & 1], s, last, c.s)), "k_muon_apply");
    }
  }
  return ADAF_OK;
}

template <bool STEP>
adaf_status run_group(const Call& c, const Matrix* mats, int count, bool first) {
  const int64_t m = mats[0].m, n = mats[0].n;
  const Layout L = layout(m, n, count);
  Group grp;
  std::memset(&grp, 0, sizeof grp);
  for (int i = 0; i < count; ++i) {
    grp.p[i] = mats[i].p;
    grp.u[i] = mats[i].u;
    grp.mom[i] = mats[i].mom;
    grp.flags[i] = mats[i].flags;
    if (STEP) {
      const double h = static_cast<double>(mats[i].rows), w = static_cast<double>(mats[i].cols);
      const bool original = c.hp->adjust_lr == MUON_ADJUST_ORIGINAL;
      grp.rate[i] = static_cast<float>(c.hp->lr * (original ? std::sqrt(std::max(1.0, h / w)) : 0.2 * std::sqrt(std::max(h, w))));
    }
  }
  MuonArgs a{};
  a.m = static_cast<int32_t>(m);
  a.n = static_cast<int32_t>(n);
  a.ldx = static_cast<int32_t>(round_up(n, 8));
  a.lda = static_cast<int32_t>(round_up(m, 8));
  a.parts = static_cast<int32_t>(std::min<int64_t>(kMaxParts, (m * n + kPartValues - 1) / kPartValues));
  a.stride_r = c.stride_r;
  a.eps = static_cast<float>(c.it->eps);
  if (STEP) {
    a.mu = static_cast<float>(c.hp->momentum);
    a.nesterov_mu = c.hp->nesterov != 0 ? a.mu : -1.f;
  }
  a.part = reinterpret_cast<float*>(c.ws + L.part);
  a.hi = reinterpret_cast<__half*>(c.ws + L.hi0);
  a.lo = reinterpret_cast<__half*>(c.ws + L.lo);
  a.status = reinterpret_cast<int32_t*>(c.ws);
  a.clear = first ? 1 : 0;
  // (rows and columns as u has them only matter where its rows have gaps: then there is one shape)
  MUON_TRY(g_profile.run(kSlotMoment, c.s, [&] {
    k_muon_moment<STEP><<<dim3(a.parts, count), 256, 0, c.s>>>(grp, a, static_cast<int32_t>(mats[0].rows), static_cast<int32_t>(mats[0].cols));
    return cudaGetLastError();
  }), "k_muon_moment");
  MUON_TRY(g_profile.run(kSlotPack, c.s, [&] {
    k_muon_pack<STEP><<<dim3(static_cast<unsigned>((n + 63) / 64), static_cast<unsigned>((m + 63) / 64), count), 256, 0, c.s>>>(
        grp, a, static_cast<int32_t>(m), static_cast<int32_t>(n));
    return cudaGetLastError();
  }), "k_muon_pack");
  const float keep = STEP ? static_cast<float>(1.0 - c.hp->lr * c.hp->weight_decay) : 1.f;
  const int64_t big = ((m + 255) / 256) * ((m + 255) / 256 + 1) / 2 * count;
  if (big >= 64) return iterate<2, 256, 6>(c, L, grp, m, n, count, keep);
  return iterate<1, 128, 6>(c, L, grp, m, n, count, keep);
}

template <bool STEP>
adaf_status run(const Call& c, std::vector<Matrix>& mats) {
  // matrices of the same sides, tall and wide ones, are worked on together
  std::stable_sort(mats.begin(), mats.end(),
                   [](const Matrix& x, const Matrix& y) { return std::make_pair(x.m, x.n) < std::make_pair(y.m, y.n); });
  bool first = true;
  for (size_t i = 0; i < mats.size();) {
    size_t j = i;
    while (j < mats.size() && mats[j].m == mats[i].m && mats[j].n == mats[i].n) ++j;
    const int most = group_size(mats[i].m, mats[i].n, static_cast<int64_t>(j - i));
    for (; i < j; i += static_cast<size_t>(most)) {
      const adaf_status st = run_group<STEP>(c, &mats[i], static_cast<int>(std::min<size_t>(static_cast<size_t>(most), j - i)), first);
      if (st != ADAF_OK) return st;
      first = false;
    }
    i = j;
  }
  return ADAF_OK;
}

}  // namespace

extern "C" {

void muon_default_iteration(muon_iteration* it) {
  if (it == nullptr) return;
  std::memset(it, 0, sizeof *it);
  it->steps = 5;
  for (int k = 0; k < 5; ++k) {
    it->coef[k][0] = 3.4445;
    it->coef[k][1] = -4.7750;
    it->coef[k][2] = 2.0315;
  }
  it->eps = 1e-7;
}

adaf_status muon_validate(const muon_hparams* hp) { return check_hp(hp); }
adaf_status muon_validate_iteration(const muon_iteration* it) { return check_iteration(it); }

adaf_status muon_workspace_size(const muon_tensor* tensors, int32_t n, size_t* bytes) {
  if (bytes == nullptr) return invalid("bytes is NULL");
  return check_tensors(tensors, n, bytes);
}

adaf_status muon_orthogonalize_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
  if (bytes == nullptr) return invalid("bytes is NULL");
  const adaf_status st = check_size(batch, rows, cols, "");
  if (st != ADAF_OK) return st;
  std::vector<std::pair<std::pair<int64_t, int64_t>, int64_t>> sizes;
  if (batch > 0 && rows > 0 && cols > 0) sizes.push_back({{std::min(rows, cols), std::max(rows, cols)}, batch});
  *bytes = sizes.empty() ? 0 : bytes_of(sizes);
  return ADAF_OK;
}

adaf_status muon_step(const muon_tensor* tensors, int32_t n, const muon_hparams* hp, void* workspace, size_t workspace_bytes,
                      void* stream) {
  adaf_status st = check_hp(hp);
  if (st != ADAF_OK) return st;
  size_t need = 0;
  if ((st = check_tensors(tensors, n, &need)) != ADAF_OK) return st;
  std::vector<Matrix> mats;
  for (int32_t i = 0; i < n; ++i) {
    const muon_tensor& t = tensors[i];
    if (t.batch == 0 || t.rows == 0 || t.cols == 0) continue;
    const std::string who = "tensor " + std::to_string(i);
    if (t.p == nullptr || t.g == nullptr || t.momentum == nullptr) return invalid(who + " has a NULL pointer");
    const size_t es = t.grad_dtype == ADAF_BFLOAT16 ? 2 : 4;
    if (!aligned(t.p, 4) || !aligned(t.momentum, 4) || !aligned(t.g, es)) return invalid(who + " is not element-aligned");
    const int64_t numel = t.rows * t.cols;
    for (int64_t b = 0; b < t.batch; ++b)
      mats.push_back({std::min(t.rows, t.cols), std::max(t.rows, t.cols), t.rows, t.cols, t.p + b * numel,
                      static_cast<const char*>(t.g) + static_cast<size_t>(b * numel) * es, t.momentum + b * numel,
                      static_cast<unsigned char>((t.rows > t.cols ? kTurned : 0) | (es == 2 ? kBf16 : 0))});
  }
  if (mats.empty()) return ADAF_OK;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != ADAF_OK) return st;
  const Call c{&hp->iteration, hp, 0, 0, static_cast<unsigned char*>(workspace), static_cast<cudaStream_t>(stream)};
  return run<true>(c, mats);
}

adaf_status muon_orthogonalize(const muon_matrices* x, const muon_iteration* it, void* out, int32_t out_dtype, void* workspace,
                               size_t workspace_bytes, void* stream) {
  adaf_status st = check_iteration(it);
  if (st != ADAF_OK) return st;
  if (x == nullptr) return invalid("x is NULL");
  size_t need = 0;
  if ((st = muon_orthogonalize_workspace_size(x->batch, x->rows, x->cols, &need)) != ADAF_OK) return st;
  if (x->dtype != ADAF_FLOAT32 && x->dtype != ADAF_BFLOAT16) return invalid("unknown dtype");
  if (out_dtype != ADAF_FLOAT32 && out_dtype != ADAF_BFLOAT16) return invalid("unknown out_dtype");
  if (need == 0) return ADAF_OK;
  const size_t es = x->dtype == ADAF_BFLOAT16 ? 2 : 4, os = out_dtype == ADAF_BFLOAT16 ? 2 : 4;
  if (x->x == nullptr || out == nullptr) return invalid("x or out is NULL");
  if (!aligned(x->x, es) || !aligned(out, os)) return invalid("x or out is not element-aligned");
  if (x->stride_b < 0 || x->stride_r < 0 || x->stride_b > (int64_t{1} << 40) || x->stride_r > (int64_t{1} << 40))
    return invalid("strides must be 0 to 2^40");
  const int64_t numel = x->rows * x->cols;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x->x), o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t x1 = x0 + static_cast<size_t>((x->batch - 1) * x->stride_b + (x->rows - 1) * x->stride_r + x->cols) * es;
  const uintptr_t o1 = o0 + static_cast<size_t>(x->batch * numel) * os;
  const bool same = x0 == o0 && es == os && (x->rows == 1 || x->stride_r == x->cols) && (x->batch == 1 || x->stride_b == numel);
  if (!same && x0 < o1 && o0 < x1) return invalid("out overlaps x, and is not x itself");
  if ((st = check_workspace(workspace, workspace_bytes, need)) != ADAF_OK) return st;
  std::vector<Matrix> mats;
  for (int64_t b = 0; b < x->batch; ++b)
    mats.push_back({std::min(x->rows, x->cols), std::max(x->rows, x->cols), x->rows, x->cols,
                    reinterpret_cast<float*>(static_cast<char*>(out) + static_cast<size_t>(b * numel) * os),
                    static_cast<const char*>(x->x) + static_cast<size_t>(b * x->stride_b) * es, nullptr,
                    static_cast<unsigned char>((x->rows > x->cols ? kTurned : 0) | (es == 2 ? kBf16 : 0))});
  const Call c{it, nullptr, x->rows == 1 ? x->cols : x->stride_r, os == 2 ? 1 : 0, static_cast<unsigned char*>(workspace),
               static_cast<cudaStream_t>(stream)};
  return run<false>(c, mats);
}

adaf_status muon_device_status(const void* workspace, void* stream, int32_t* status) {
  if (workspace == nullptr || status == nullptr) return invalid("workspace or status is NULL");
  cudaError_t e = cudaMemcpyAsync(status, workspace, sizeof *status, cudaMemcpyDeviceToHost, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAF_OK : cuda_fail(e, "device status");
}

void muon_debug_stall_copies(int32_t on) { t_stall = on != 0; }

adaf_status muon_profile_enable(int32_t on) {
  g_profile.on = on != 0;
  return ADAF_OK;
}
adaf_status muon_profile_read(double* ms, int64_t* launches, int32_t nk) {
  const cudaError_t e = g_profile.read(ms, launches, nk);
  return e == cudaSuccess ? ADAF_OK : cuda_fail(e, "profile event");
}
int32_t muon_num_kernels(void) { return kNumKernels; }
const char* muon_kernel_name(int32_t k) { return k >= 0 && k < kNumKernels ? kKernelNames[k] : ""; }

}  // extern "C"
