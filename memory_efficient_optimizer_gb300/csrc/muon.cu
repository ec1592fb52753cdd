// Multi-tensor Muon step and its orthogonalisation for sm_103a: the C ABI of
// include/muon.h.
//
// The matrices of a list (with the smaller side as m, the larger as n; a taller
// matrix is worked on transposed) go through three launches together:
//
//   k_muon_moment   m = mu m + g; sum u^2 of every matrix, in parts
//   k_muon_pack     x = u / max(||u||, eps), in the layout of the products
//   k_muon_iterate  the steps of the iteration; each is three phases of products,
//                   which do everything else in their endings:
//                     A = x x^T          (only tiles on or above the diagonal)
//                     B = b A + c A A    (the same)
//                     x = a x + B x; the last one updates p, or writes the result
//
// Numbers.  The factors of the products are fp16, scaled by powers of two: an
// element of x is at most its largest singular value, 1.21 (1.9 with other
// coefficients), so x 2^15 fits, and so do A 2^14 and B 2^14, and at any size the
// usual elements are far above the subnormal range (1 / sqrt(mn) 2^15 is 8 at
// 4096 x 4096).  What rounding does depends on where it enters:
//   - rounding of the factors of x x^T, A A and B x acts like a multiplication
//     of x by I + d with small d from the left or the right: directions turn by
//     2^-12 or so, and a small singular value stays as accurate as a large one;
//   - rounding of x where it is carried to the next step adds noise at the level
//     of the large singular values, which the small ones drown in (they grow by
//     3.44 a step, and the noise with them).  So x is carried in fp32, beside the
//     fp16 copy that is the factor of the products;
//   - as x comes near orthogonal, A comes near a multiple of I, and a rounding of
//     the diagonal would weigh most.  With A = D + F, B = G + E (D, G diagonal,
//     in fp32), A A = F F + D F + F D + D D and a x + B x = (a + G) x + E x: only
//     F and E are rounded and multiplied.
// Against the formula in 64 bits this is 2e-4 to 1.1e-3 off (2-norms) for flat
// and for decaying spectra alike, from 128 rows on, where fp16 iterates are
// 1.3e-3 to 1.2e-2 off and bf16 ones 1e-2 to 9e-2 (the header has the bounds).
//
// What bounds it: the tensor cores under the power cap, for matrices from about
// 2000 on (a decoder layer of 218 M values: 10.9 ms, 1340 TFLOP/s of the 3 m^2 n +
// m^3 flops a step that are left when the symmetric A and B are computed by one
// half); L2 where m is about 1000; the way from one phase to the next, 5 to 6 us,
// for small ones.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <exception>
#include <string>
#include <vector>

#include "adafactor_internal.h"
#include "muon.h"
#include "tc_host.cuh"

namespace {

constexpr int kMaxGroup = 48;                      // matrices of a launch
constexpr int kFew = 8;                            // a launch of few matrices has smaller arguments
constexpr int64_t kGroupValues = int64_t{1} << 28;  // their values, unless one alone has more
constexpr int kMaxParts = 256;                     // of a matrix's sum of squares
constexpr int kPartValues = 8192;                  // values of a part, at least
constexpr int64_t kMaxSide = int64_t{1} << 20;
// x x^T of few wide matrices is summed in parts, so many tiles of them at most: one round of the SMs.
// A part has ten stages or more (3 us); to write and join the parts takes 2 to 4 us.  64 x 20000 took
// 570 us in one sum, 163 in 16 parts; 1024 x 4096 304, 256 in 4; 16 x 2688 127, 91 in 4.  In parts of 8
// stages 2 x 1024 x 1024 took 193 us instead of 184.
constexpr int kPartTiles = 144, kMostParts = 16, kPartStages = 10;
constexpr int kMaxJoined = kPartTiles / 2 * meo::tc::kEndWarps;   // counters of the tiles' warps
constexpr int64_t kMaxMatrices = int64_t{1} << 20;

enum Flag : int32_t { kTurned = 1, kBf16 = 2 };   // x is u^T; u is bf16

// A matrix as the passes before the products see it.
struct Item {
  const void* u;                   // the gradient, or the matrix to orthogonalise
  float* mom;
  __half* hi;
  float* x;
  int32_t rows, cols;              // of u
  int32_t m, n, ldx;               // of x: m <= n
  int32_t flags;
  int32_t parts, part0, tile0;     // parts of its sum of squares; its first part and tile of the launches
};

struct MuonArgs {
  int32_t count;
  int64_t stride_r;                // of u
  float mu, nesterov_mu, eps;      // u = g + nesterov_mu m, or m itself (nesterov_mu < 0)
  float2* part;                    // [parts of all matrices]: the sums of u^2 and of (2^80 u)^2
  int32_t* status;
  unsigned* done;
  unsigned* joined;
  int32_t clear;                   // this launch clears the status word
  Item item[kMaxGroup];
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
// The squares of values below 1e-19 or so are no longer normal fp32 numbers, or 0.  So the squares of 2^80 u
// are summed beside those of u, and count where the latter's sum is below kSmallSum (what is lost of that
// sum's terms is then below 2^-78 of it).
constexpr float kUp = 0x1p80f, kSmallSum = 0x1p-40f, kSmallEps = 0x1p-20f;
__device__ __forceinline__ float2 squares(float v) {
  const float w = v * kUp;
  return make_float2(v * v, w * w);
}
__device__ __forceinline__ void add_four(float2& sum, const float4& v) {
  const float2 x = squares(v.x), y = squares(v.y), z = squares(v.z), w = squares(v.w);
  sum.x += (x.x + y.x) + (z.x + w.x);
  sum.y += (x.y + y.y) + (z.y + w.y);
}
__device__ __forceinline__ void add_one(float2& sum, float v) {
  const float2 x = squares(v);
  sum.x += x.x;
  sum.y += x.y;
}
__device__ __forceinline__ float update_of(float g, float m, const MuonArgs& a) {
  return a.nesterov_mu < 0.f ? m : fmaf(a.nesterov_mu, m, g);
}

// Matrix of a launch that has block `at` of those that `first` counts.
template <class First>
__device__ __forceinline__ int owner(int count, int at, First&& first) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first(mid) <= at)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// One part of a matrix a CTA.  STEP: the momentum is brought up to date too.
// Read 2 or 4 + 4 bytes a value, write 4: bound by memory.
template <bool STEP>
__global__ void __launch_bounds__(256) k_muon_moment(const __grid_constant__ MuonArgs a) {
  __shared__ float scratch[8];
  meo::tc::next_may_begin();
  if (blockIdx.x == 0) {
    if (a.clear != 0 && threadIdx.x == 0) *a.status = 0;
    if (threadIdx.x < kMaxGroup + 1) a.done[threadIdx.x] = 0;   // (and the ticket behind them)
    for (int i = threadIdx.x; i < kMaxJoined; i += 256) a.joined[i] = 0;
  }
  const Item& t = a.item[owner(a.count, blockIdx.x, [&](int i) { return a.item[i].part0; })];
  const bool bf16 = t.flags & kBf16;
  const void* const u = t.u;
  float* const mom = t.mom;
  const int cols = t.cols;
  const bool flat = STEP || a.stride_r == cols;
  const int64_t numel = static_cast<int64_t>(t.rows) * cols;
  const int64_t per = ((numel + t.parts - 1) / t.parts + 3) & ~int64_t{3};
  const int64_t e0 = per * (blockIdx.x - t.part0), e1 = min(numel, e0 + per);
  float2 sum = make_float2(0.f, 0.f);
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
        add_four(sum, v);
      }
    }
    for (int64_t i = tail + threadIdx.x; i < e1; i += 256) {
      float v = value_at(u, bf16, i);
      if (STEP) {
        const float m = fmaf(a.mu, mom[i], v);
        mom[i] = m;
        v = update_of(v, m, a);
      }
      add_one(sum, v);
    }
  } else {
    for (int64_t i = e0 + threadIdx.x; i < e1; i += 256) {
      const int r = static_cast<int>(i / cols), c = static_cast<int>(i - static_cast<int64_t>(r) * cols);
      add_one(sum, value_at(u, bf16, r * a.stride_r + c));
    }
  }
  sum.x = block_sum(sum.x, scratch);
  sum.y = block_sum(sum.y, scratch);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
}

// Values that only endings read and write again are kept in the order in which a warp holds them:
// blocks of 32 x 32, lane l has row l, and word i (16 bytes) of all lanes lies side by side.
// Then a warp's accesses are whole lines, with nothing to exchange between lanes.
__device__ __forceinline__ int64_t block_at(int row, int col, int n) {
  return (static_cast<int64_t>(row >> 5) * ((n + 31) >> 5) + (col >> 5)) << 10;   // values
}

// x of a matrix, 64 x 64 values a CTA, through shared memory so that both u and
// x are walked along their rows where x is u^T.
template <bool STEP>
__global__ void __launch_bounds__(256) k_muon_pack(const __grid_constant__ MuonArgs a) {
  __shared__ float tile[64][65];
  __shared__ float scratch[8];
  meo::tc::next_may_begin();
  meo::tc::previous_done();
  const Item& t = a.item[owner(a.count, blockIdx.x, [&](int i) { return a.item[i].tile0; })];
  const int rows = t.m, cols = t.n, ldx = t.ldx;
  const int across = (cols + 63) >> 6, at_tile = blockIdx.x - t.tile0;
  const int by = at_tile / across, bx = at_tile - by * across;
  const float2 part = static_cast<int>(threadIdx.x) < t.parts ? a.part[t.part0 + threadIdx.x] : make_float2(0.f, 0.f);
  const float sum = block_sum(part.x, scratch), sum_up = block_sum(part.y, scratch);
  // (both sides times 2^80; an eps above the norm needs none of it)
  const bool small = sum < kSmallSum && a.eps < kSmallEps;
  const float up = small ? kUp : 1.f, norm = sqrtf(small ? sum_up : sum);
  // (a norm that is not finite makes x NaN)
  const float scale = norm <= FLT_MAX ? 32768.f / fmaxf(norm, a.eps * up) : __int_as_float(0x7fc00000);
  const bool bf16 = t.flags & kBf16, turned = t.flags & kTurned;
  const void* const u = t.u;
  const float* const mom = t.mom;
  const int r0 = (turned ? bx : by) * 64, c0 = (turned ? by : bx) * 64;   // of u
  const int64_t pitch = STEP ? t.cols : a.stride_r;
  const bool quads = (pitch | t.cols) % 4 == 0 && reinterpret_cast<uintptr_t>(u) % (bf16 ? 8 : 16) == 0 &&
                     (!STEP || reinterpret_cast<uintptr_t>(mom) % 16 == 0);
  if (quads) {
    // 4 values side by side, all of a thread's under way before the first is used
    float4 v[4], m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + (threadIdx.x >> 4) + 16 * i, c = c0 + (threadIdx.x & 15) * 4;
      v[i] = m[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < t.rows && c < t.cols) {
        v[i] = four_at(u, bf16, r * pitch + c);
        if (STEP) m[i] = __ldcs(reinterpret_cast<const float4*>(mom + r * pitch + c));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* const to = &tile[(threadIdx.x >> 4) + 16 * i][(threadIdx.x & 15) * 4];
      if (STEP) v[i] = make_float4(update_of(v[i].x, m[i].x, a), update_of(v[i].y, m[i].y, a), update_of(v[i].z, m[i].z, a), update_of(v[i].w, m[i].w, a));
      to[0] = v[i].x * up * scale, to[1] = v[i].y * up * scale, to[2] = v[i].z * up * scale, to[3] = v[i].w * up * scale;
    }
  } else {
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
      const int r = r0 + (i >> 6), c = c0 + (i & 63);
      float v = 0.f;
      if (r < t.rows && c < t.cols) {
        const int64_t at = r * pitch + c;
        v = value_at(u, bf16, at);
        if (STEP) v = update_of(v, mom[at], a);
        v = v * up * scale;
      }
      tile[i >> 6][i & 63] = v;
    }
  }
  __syncthreads();
  const int x0 = by * 64, y0 = bx * 64;   // of x
  for (int i = threadIdx.x; i < 64 * 32; i += 256) {
    const int r = i >> 5, c = (i & 31) * 2;
    if (x0 + r >= rows || y0 + c >= ldx) continue;
    const float v0 = turned ? tile[c][r] : tile[r][c], v1 = turned ? tile[c + 1][r] : tile[r][c + 1];
    *reinterpret_cast<__half2*>(t.hi + static_cast<int64_t>(x0 + r) * ldx + y0 + c) = __floats2half2_rn(v0, v1);
  }
  // four blocks of 32 x 32, two warps each
  const int blk = threadIdx.x >> 6, r0x = (blk >> 1) * 32, c0x = (blk & 1) * 32, lane = threadIdx.x & 31;
  if (x0 + r0x < rows && y0 + c0x < cols) {
    float4* const to = reinterpret_cast<float4*>(t.x + block_at(x0 + r0x, y0 + c0x, cols)) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = i * 2 + ((threadIdx.x >> 5) & 1), r = r0x + lane, c = c0x + 4 * w;
      to[32 * w] = turned ? make_float4(tile[c][r], tile[c + 1][r], tile[c + 2][r], tile[c + 3][r])
                          : make_float4(tile[r][c], tile[r][c + 1], tile[r][c + 2], tile[r][c + 3]);
    }
  }
}

// ---- endings of the products ------------------------------------------------------------
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t r) { return __half22float2(*reinterpret_cast<const __half2*>(&r)); }

// 32 fp16 values a row of a matrix with rows of ld values, from column col on (values beyond the
// last column are 0 and go up to ld).
__device__ __forceinline__ void store_rows(__half* to, int ld, const meo::tc::Part& p, int col, uint4 (&w)[4]) {
  p.ex.to_memory(w);
  p.ex.put(to + static_cast<int64_t>(p.row0()) * ld + col, static_cast<int64_t>(ld) * 2, p.m - p.row0(), (ld - col) * 2, w);
}
__device__ __forceinline__ void pack32(const float (&v)[32], uint4 (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = make_uint4(pack(v[8 * i], v[8 * i + 1]), pack(v[8 * i + 2], v[8 * i + 3]), pack(v[8 * i + 4], v[8 * i + 5]),
                      pack(v[8 * i + 6], v[8 * i + 7]));
}

// A matrix as the products see it.
struct Matrix {
  __half* hi;            // [2][m][ldx]: of this step and of the next
  float* xb;             // x in blocks (block_at), updated in place
  __half* fe;            // [slabs][m][lda]: symmetric matrices without their diagonals, the tiles on and above it
  __half* fb;            // the same in blocks
  float* dg;             // [slabs][lda]: the diagonals
  float* p;              // the parameter, or the result
  int32_t m, n, ldx, lda;
  int32_t flags;
  float rate;            // p = keep p - rate o
  int32_t sym0, app0;    // its first tile of the symmetric products and of the others
  int32_t splits, gram0; // parts of the sums of x x^T; its first tile of those
  float* parts;          // [tiles][splits][warps][32 rows x BN / 2 columns in the lanes' order]
  unsigned* joined;      // [tiles][warps]: parts that are there
};

enum Out : int32_t { kUpdate, kFp32, kBf16Out };

constexpr int kSlabs = 2, kPairSlabs = 4;   // symmetric matrices that are kept: A and its polynomial; for two steps at once
// Scales of the symmetric matrices' elements beside the diagonals: at most 3.9, so 2^14; a product
// of two polynomials at most 15.5, so 2^12.
constexpr int kSymScale = 14, kPairScale = 12;

enum Kind : int32_t { kGram, kPoly, kMul, kApply };
struct Phase {
  int32_t kind;
  int32_t a, b, out;     // slabs of the symmetric factors and the result; of x: 0 or 1
  float c0, c1, c2;      // kPoly: a, b, c; kMul: factors of the product and of the diagonals' parts; kApply: of the product
  int32_t start;         // first tile
  int32_t syms, apps;    // phases before it, by the kind of their results
  int32_t last;          // kApply: of the last step
};
constexpr int kMaxPhases = 3 * MUON_MAX_STEPS + 1;

template <int COUNT>
struct IterateArgs {
  struct {
    CUtensorMap x, s;    // hi and fe
  } map[COUNT];
  Matrix mat[COUNT];     // (copied to shared memory first: at every phase's first tile the constants
                         // would be asked for anew, a microsecond or two each)
  Phase phase[kMaxPhases];
  int32_t count, phases, tiles;
  int32_t out;
  float keep;
  int32_t stall;
  int32_t* status;
  unsigned* done;        // of each matrix, tiles that are done
  unsigned* ticket;      // tiles that are taken
};

using meo::tc::Part;

// 32 columns of a symmetric result without its diagonal, into slab `out`.
__device__ __forceinline__ void store_symmetric(const Matrix& t, const Part& p, int j0, int out, uint4 (&w)[4]) {
  if (p.row0() < p.m) {
    uint4* const to = reinterpret_cast<uint4*>(t.fb + (block_at((p.m + 31) & ~31, 0, p.m) * out + block_at(p.row0(), j0, p.m))) + p.ex.lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) to[32 * i] = w[i];
  }
  store_rows(t.fe + static_cast<int64_t>(out) * p.m * t.lda, t.lda, p, j0, w);
}
// The element of a lane's row that lies on the diagonal, in a block on it; and what is stored there.
__device__ __forceinline__ float on_diagonal(const Part& p, const float (&v)[32]) {
  float d = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) d = i == p.ex.lane ? v[i] : d;
  return d;
}
__device__ __forceinline__ void clear_diagonal(const Part& p, uint4 (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t& x = i % 4 == 0 ? w[i / 4].x : i % 4 == 1 ? w[i / 4].y : i % 4 == 2 ? w[i / 4].z : w[i / 4].w;
    if (p.ex.lane == 2 * i) x &= 0xffff0000u;
    if (p.ex.lane == 2 * i + 1) x &= 0xffffu;
  }
}

// A = x x^T = D + F.  load(c, v): 32 columns of the sums.
template <class Load>
__device__ __forceinline__ void end_gram(const Matrix& t, const Part& p, Load&& load) {
#pragma unroll 1
  for (int c = 0; c < p.cols && p.col + c < p.m; c += 32) {
    const int j0 = p.col + c;
    float v[32];
    load(c, v);   // A 2^30
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= 0x1p-16f;
    uint4 w[4];
    pack32(v, w);
    if (p.row0() == j0) {
      const float d = on_diagonal(p, v);
      if (p.row < p.m) t.dg[p.row] = d * 0x1p-14f;
      clear_diagonal(p, w);
    }
    store_symmetric(t, p, j0, 0, w);
  }
}

// The same where the sums are in parts: the warp's part is written out, and the warp that brings the
// last one adds them up in their order.  Whether that is this one; `warp`: of the tile's.
template <int COLS>
__device__ __forceinline__ bool end_gram_part(const Matrix& t, const Part& p, int warp) {
  constexpr int kWords = COLS / 4 * 32;   // of 16 bytes, a warp's part
  const int at = p.tile.number * meo::tc::kEndWarps + warp;
  const bool rows = p.row0() < p.m;
  float4* const first = reinterpret_cast<float4*>(t.parts) + (static_cast<int64_t>(p.tile.number) * t.splits * meo::tc::kEndWarps + warp) * kWords + p.ex.lane;
  constexpr int64_t kNext = meo::tc::kEndWarps * kWords;
#pragma unroll
  for (int c = 0; c < COLS; c += 32) {
    float v[32];
    p.load(c, v);
    if (rows && p.col + c < p.m) {
#pragma unroll
      for (int i = 0; i < 8; ++i) first[p.tile.split * kNext + c * 8 + 32 * i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
  __syncwarp();
  unsigned before = 0;
  if (p.ex.lane == 0) {
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(t.joined + at) : "memory");
    if (before + 1 == static_cast<unsigned>(t.splits)) t.joined[at] = 0;   // (for the next step, which waits for this one)
  }
  __syncwarp();   // (what lane 0 has acquired, all have: the other warps' parts)
  before = __shfl_sync(0xffffffffu, before, 0);
  if (before + 1 != static_cast<unsigned>(t.splits)) return false;
  end_gram(t, p, [&](int c, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
    if (!rows) return;
#pragma unroll 2
    for (int s = 0; s < t.splits; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = __ldcg(first + s * kNext + c * 8 + 32 * i);
        v[4 * i] += x.x, v[4 * i + 1] += x.y, v[4 * i + 2] += x.z, v[4 * i + 3] += x.w;
      }
  });
  return true;
}

// What an ending reads beside the sums.  It is asked for before the sums are there: behind the
// ring's copies, which keep the SM's port to L2 full, an answer takes two microseconds, and a
// tile's four in a row took longer than its products.
template <int WORDS, int CHUNKS>
struct Ahead {
  uint4 w[CHUNKS][WORDS];
  // `from`: the block of the warp's first row and first column; `left`: columns that are there
  __device__ __forceinline__ void fetch(const Part& p, const void* from, bool rows, int left) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const uint4* const at = static_cast<const uint4*>(from) + c * 32 * WORDS + p.ex.lane;
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[c][i] = rows && 32 * c < left ? at[32 * i] : make_uint4(0, 0, 0, 0);
    }
  }
};

// P = a + b A + c A A, A = D + F.  di, dj: D of the row, and of the columns (in the warp's shared
// memory).
template <int CHUNKS>
__device__ __forceinline__ void end_poly(const Matrix& t, const Part& p, const Ahead<4, CHUNKS>& f, float di, const float* dj,
                                         const Phase& ph) {
  const float cb = ph.c1, cc = ph.c2;
  float* const diagonal = t.dg + static_cast<int64_t>(ph.out) * t.lda;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int j0 = p.col + 32 * c;
    if (j0 >= p.m) break;
    float v[32];
    p.load(32 * c, v);
    // (b + c (d_i + d_j)) F + c F F, two columns at a time; F is scaled by 2^14, F F by 2^28
    const float2 own = make_float2(cb + cc * di, cb + cc * di), c2 = make_float2(cc, cc), small_c = make_float2(cc * 0x1p-14f, cc * 0x1p-14f);
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r[4] = {f.w[c][i].x, f.w[c][i].y, f.w[c][i].z, f.w[c][i].w};
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 d = *reinterpret_cast<const float2*>(dj + 32 * c + 8 * i + 2 * q);
        const float2 x = __fmul2_rn(small_c, make_float2(v[8 * i + 2 * q], v[8 * i + 2 * q + 1]));
        const float2 e = __ffma2_rn(unpack(r[q]), __ffma2_rn(c2, d, own), x);
        o[q] = pack(e.x, e.y);
      }
      w[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (p.row0() == j0) {
      const float x = on_diagonal(p, v) * 0x1p-28f;
      if (p.row < p.m) diagonal[p.row] = ph.c0 + fmaf(cc, fmaf(di, di, x), cb * di);
      clear_diagonal(p, w);
    }
    store_symmetric(t, p, j0, ph.out, w);
  }
}

// The product of two symmetric matrices that commute, U = D + E and V = D' + E': E E' + D E' + E D' + D D'.
// di: D of the row, own: D' of the row, dj: D' of the columns.
template <int CHUNKS>
__device__ __forceinline__ void end_mul(const Matrix& t, const Part& p, const Ahead<4, CHUNKS>& u, const Ahead<4, CHUNKS>& f, float di,
                                        float own, const float* dj, const Phase& ph) {
  float* const diagonal = t.dg + static_cast<int64_t>(ph.out) * t.lda;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int j0 = p.col + 32 * c;
    if (j0 >= p.m) break;
    float v[32];
    p.load(32 * c, v);
    const float2 c0 = make_float2(ph.c0, ph.c0), c1 = make_float2(ph.c1, ph.c1), d2 = make_float2(di * ph.c1, di * ph.c1);
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r[4] = {f.w[c][i].x, f.w[c][i].y, f.w[c][i].z, f.w[c][i].w}, s[4] = {u.w[c][i].x, u.w[c][i].y, u.w[c][i].z, u.w[c][i].w};
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 d = __fmul2_rn(c1, *reinterpret_cast<const float2*>(dj + 32 * c + 8 * i + 2 * q));
        const float2 x = __fmul2_rn(c0, make_float2(v[8 * i + 2 * q], v[8 * i + 2 * q + 1]));
        const float2 e = __ffma2_rn(unpack(r[q]), d2, __ffma2_rn(unpack(s[q]), d, x));
        o[q] = pack(e.x, e.y);
      }
      w[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (p.row0() == j0) {
      const float x = on_diagonal(p, v) * 0x1p-28f;
      if (p.row < p.m) diagonal[p.row] = fmaf(di, own, x);
      clear_diagonal(p, w);
    }
    store_symmetric(t, p, j0, ph.out, w);
  }
}

// 32 columns of D x + E x, scaled by 2^15; the product comes with the scale of E too.
__device__ __forceinline__ void applied(const Part& p, int c, const uint4 (&x)[8], float factor, float scale, float (&v)[32]) {
  p.load(c, v);
  const float2 f = make_float2(factor, factor), s = make_float2(scale, scale);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 a = __ffma2_rn(f, make_float2(__uint_as_float(x[i].x), __uint_as_float(x[i].y)), __fmul2_rn(s, make_float2(v[4 * i], v[4 * i + 1])));
    const float2 b = __ffma2_rn(f, make_float2(__uint_as_float(x[i].z), __uint_as_float(x[i].w)), __fmul2_rn(s, make_float2(v[4 * i + 2], v[4 * i + 3])));
    v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = b.x, v[4 * i + 3] = b.y;
  }
}

// x of the next step.
template <int CHUNKS>
__device__ __forceinline__ void end_next(const Matrix& t, const Part& p, const Ahead<8, CHUNKS>& x, int slab, float factor, float scale) {
  __half* const next = t.hi + (slab ^ 1) * (static_cast<int64_t>(p.m) * t.ldx) + static_cast<int64_t>(p.row0()) * t.ldx + p.col;
  uint4* const xb = reinterpret_cast<uint4*>(t.xb + block_at(p.row0(), p.col, p.n)) + p.ex.lane;
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
    if (p.col + 32 * k >= p.n) break;
    float v[32];
    applied(p, 32 * k, x.w[k], factor, scale, v);
    if (p.row0() < p.m) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        xb[k * 256 + 32 * i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                          __float_as_uint(v[4 * i + 3]));
    }
    uint4 h[4];
    pack32(v, h);
    p.ex.to_memory(h);
    p.ex.put(next + 32 * k, static_cast<int64_t>(t.ldx) * 2, p.m - p.row0(), (t.ldx - p.col - 32 * k) * 2, h);
  }
}

// The last step: the update of p, or the result.
template <int CHUNKS>
__device__ __forceinline__ void end_last(const Matrix& t, const Part& p, const Ahead<8, CHUNKS>& x, float factor, float scale, int out,
                                         float keep) {
  const bool turned = t.flags & kTurned;
  const bool wide = p.n % (out == kBf16Out ? 8 : 4) == 0 && reinterpret_cast<uintptr_t>(t.p) % 16 == 0;
  const float rate = t.rate * 0x1p-15f;
  const int rows = p.m - p.row0();
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
    const int c = 32 * k, j0 = p.col + c;
    if (j0 >= p.n) break;
    float v[32];
    applied(p, c, x.w[k], factor, scale, v);
    if (turned) {
      // down a column of the parameter: the warp's lanes lie side by side there
      if (p.row >= p.m) continue;
      const int64_t to = static_cast<int64_t>(j0) * p.m + p.row;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (j0 + i >= p.n) break;
        const int64_t q = to + static_cast<int64_t>(i) * p.m;
        if (out == kUpdate)
          t.p[q] = fmaf(-rate, v[i], keep * t.p[q]);
        else if (out == kBf16Out)
          reinterpret_cast<__nv_bfloat16*>(t.p)[q] = __float2bfloat16_rn(v[i] * 0x1p-15f);
        else
          t.p[q] = v[i] * 0x1p-15f;
      }
    } else if (out == kBf16Out) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t two[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __nv_bfloat162 r = __floats2bfloat162_rn(v[8 * i + 2 * q] * 0x1p-15f, v[8 * i + 2 * q + 1] * 0x1p-15f);
          two[q] = *reinterpret_cast<const uint32_t*>(&r);
        }
        w[i] = make_uint4(two[0], two[1], two[2], two[3]);
      }
      p.ex.to_memory(w);
      __nv_bfloat16* const q = reinterpret_cast<__nv_bfloat16*>(t.p) + static_cast<int64_t>(p.row0()) * p.n + j0;
      if (wide) {
        p.ex.put(q, static_cast<int64_t>(p.n) * 2, rows, (p.n - j0) * 2, w);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (p.ex.row(i) >= rows) continue;
          const __nv_bfloat16* const one = reinterpret_cast<const __nv_bfloat16*>(&w[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int j = p.ex.place() / 2 + e;
            if (j0 + j < p.n) q[static_cast<int64_t>(p.ex.row(i)) * p.n + j] = one[e];
          }
        }
      }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {   // 16 columns, 64 bytes
        uint4 w[4], old[4];
        float* const q = t.p + static_cast<int64_t>(p.row0()) * p.n + j0 + 16 * half;
        const int left = p.n - j0 - 16 * half;
        if (out == kUpdate && wide) p.ex.fetch(q, static_cast<int64_t>(p.n) * 4, rows, left * 4, old);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = make_uint4(__float_as_uint(v[16 * half + 4 * i]), __float_as_uint(v[16 * half + 4 * i + 1]),
                            __float_as_uint(v[16 * half + 4 * i + 2]), __float_as_uint(v[16 * half + 4 * i + 3]));
        p.ex.to_memory(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float r[4] = {__uint_as_float(w[i].x), __uint_as_float(w[i].y), __uint_as_float(w[i].z), __uint_as_float(w[i].w)};
          const float o[4] = {__uint_as_float(old[i].x), __uint_as_float(old[i].y), __uint_as_float(old[i].z), __uint_as_float(old[i].w)};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (wide) {
              r[e] = out == kUpdate ? fmaf(-rate, r[e], keep * o[e]) : r[e] * 0x1p-15f;
            } else if (p.ex.row(i) < rows && p.ex.place() / 4 + e < left) {
              float* const one = q + static_cast<int64_t>(p.ex.row(i)) * p.n + p.ex.place() / 4 + e;
              *one = out == kUpdate ? fmaf(-rate, r[e], keep * *one) : r[e] * 0x1p-15f;
            }
          }
          w[i] = make_uint4(__float_as_uint(r[0]), __float_as_uint(r[1]), __float_as_uint(r[2]), __float_as_uint(r[3]));
        }
        if (wide) p.ex.put(q, static_cast<int64_t>(p.n) * 4, rows, left * 4, w);
      }
    }
  }
}

// ---- the iteration ------------------------------------------------------------------------
// All steps for all matrices of a group, in one launch: a step is three phases
// (A = x x^T, the polynomial P of it, P x), each over the tiles of all matrices.
// Two steps at once are seven: with P1 of A1, the second step's A is P1 A1 P1 and
// its P2 follows; x = P2 P1 x.  That is three more products of m x m and one each
// less of m x m x n and of two sides of n.
//
// All tiles of all phases are one list, from which a cluster takes the next (an
// atomic counter) when it begins to have room for it; a tile waits until the phase
// before is done with its matrix, which another counter tells.  What a tile waits
// for comes before it in the list, so clusters that run have taken it, and the
// first tile of those that are not done waits for nothing: the clusters need not all
// be there together.  (With tiles in fixed turns they had to be, and a cooperative
// launch holds up the host and the launch: 256 x 512 took 100 us.)  The last tiles
// of one matrix's phase run beside the first of another's.  Fifteen launches in a
// row took 11 us each on a matrix of 256 x 512, of which the copies and products
// are one or two.  The roles of the warps and the ring are k_product's; they go on
// from tile to tile.  A tile's number goes from the first CTA's copying thread to
// the others that work on it, in both CTAs, through a queue in shared memory.
struct Place {
  int phase, at;         // at: the matrix
  int need;              // tiles of the matrix that have to be done
};

// Tile number i, going up from call to call; false beyond the last.
template <int CG, int BN>
__device__ __forceinline__ bool find_tile(const Matrix* mat, int count, const Phase* phase, int phases, int tiles, int i, Place* w,
                                          meo::tc::Tile* t) {
  if (i >= tiles) return false;
  while (w->phase + 1 < phases && i >= phase[w->phase + 1].start) {
    ++w->phase;
    w->at = 0;
  }
  const Phase& ph = phase[w->phase];
  i -= ph.start;
  const bool sym = ph.kind != kApply, gram = ph.kind == kGram;
  while (w->at + 1 < count && i >= (gram ? mat[w->at + 1].gram0 : sym ? mat[w->at + 1].sym0 : mat[w->at + 1].app0)) ++w->at;
  const Matrix& m = mat[w->at];
  meo::tc::Shape s{};
  s.splits = 1;
  s.group = 16;
  constexpr int kRows = meo::tc::kTileM * CG;
  const int mt = (m.m + kRows - 1) / kRows, nt = (m.n + BN - 1) / BN;
  const int mtn = (m.m + BN - 1) / BN;   // column tiles of the symmetric products
  const int syms = static_cast<int>(meo::tc::sym_tiles<kRows / BN>(mtn));
  w->need = ph.syms * syms + ph.apps * mt * nt;
  if (gram) {
    i -= m.gram0;
    const int tile = CG == 1 ? i / m.splits : i;
    const bool there = meo::tc::tile_of<true, kRows, BN>(tile, mt, mtn, s, t);
    t->number = tile;
    t->split = i - tile * (CG == 1 ? m.splits : 1);
    return there;
  }
  if (sym) return meo::tc::tile_of<true, kRows, BN>(i - m.sym0, mt, mtn, s, t);
  return meo::tc::tile_of<false, kRows, BN>(i - m.app0, mt, nt, s, t);
}

constexpr int kQueue = 4;

template <int CG, int BN, int STAGES, int COUNT>
__global__ void __launch_bounds__(meo::tc::kThreads, 1) k_muon_iterate(const __grid_constant__ IterateArgs<COUNT> a) {
  using namespace meo::tc;
  using S = Shared<CG, BN, STAGES>;
  constexpr uint32_t kCols = 2 * BN;
  constexpr int kBCta = BN / CG;
  constexpr int kRows = kTileM * CG;
  static_assert(kRows == BN || kRows == 2 * BN, "tiles of the symmetric products");
  extern __shared__ unsigned char raw[];
  unsigned char* ring = raw + ((1024 - (shared_at(raw) & 1023)) & 1023);
  unsigned char* const exchange = ring + STAGES * S::kStage;
  float* const columns = reinterpret_cast<float*>(exchange + kEndWarps * kExchange);   // of each warp: BN / 2 values
  Matrix* const mat = reinterpret_cast<Matrix*>(columns + kEndWarps * (BN / 2));
  Phase* const phase = reinterpret_cast<Phase*>(mat + COUNT);
  uint64_t* full = reinterpret_cast<uint64_t*>((reinterpret_cast<uintptr_t>(phase + kMaxPhases) + 7) & ~uintptr_t{7});
  uint64_t* empty = full + STAGES;
  uint64_t* sum_full = empty + STAGES;
  uint64_t* sum_empty = sum_full + 2;
  uint64_t* q_full = sum_empty + 2;
  uint64_t* q_empty = q_full + kQueue;    // the first CTA's counts both CTAs' readers
  int* q_tile = reinterpret_cast<int*>(q_empty + kQueue);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(q_tile + kQueue);
  volatile int* off = reinterpret_cast<volatile int*>(tmem_at + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int count = a.count, phases = a.phases, tiles = a.tiles, out = a.out;
  const float keep = a.keep;
  for (int i = threadIdx.x; i < count * static_cast<int>(sizeof(Matrix) / 4); i += kThreads)
    reinterpret_cast<uint32_t*>(mat)[i] = reinterpret_cast<const uint32_t*>(a.mat)[i];
  for (int i = threadIdx.x; i < phases * static_cast<int>(sizeof(Phase) / 4); i += kThreads)
    reinterpret_cast<uint32_t*>(phase)[i] = reinterpret_cast<const uint32_t*>(a.phase)[i];
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      bar_init(full + i, 1);
      bar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(sum_full + i, 1);
      bar_init(sum_empty + i, CG * kEndWarps);
    }
    for (int i = 0; i < kQueue; ++i) {
      bar_init(q_full + i, 1);
      bar_init(q_empty + i, CG * (kEndWarps + 1));
    }
    *off = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc<CG>(tmem_at, kCols);
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = *tmem_at;
  previous_done();

  // (the status first: who learns of a tile that this CTA could not finish learns of it too)
  auto gave_up = [&] {
    atomicOr(a.status, 1);
    __threadfence();
    *off = 1;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (bar_try(bar, parity)) return true;
    const long long from = clock64();
    while (!bar_try(bar, parity)) {
      if (*off != 0) return false;
      if (clock64() - from > kWaitCycles) {
        gave_up();
        return false;
      }
    }
    return true;
  };
  auto wait_cluster = [&](uint64_t* bar, uint32_t parity) -> bool {
    const long long from = clock64();
    while (!bar_try_cluster(bar, parity)) {
      if (*off != 0) return false;
      if (clock64() - from > 4 * kWaitCycles) {   // (as long as what the other CTA may be waiting for)
        gave_up();
        return false;
      }
    }
    return true;
  };
  // The queue's readers: waits for the next number; tells that it has been read (one thread of a reader).
  auto take = [&](int q, uint32_t bit, int* i) -> bool {
    if (!wait_cluster(q_full + q, bit)) return false;
    *i = *reinterpret_cast<volatile int*>(q_tile + q);
    return true;
  };
  auto taken = [&](int q) { bar_arrive_cluster(CG == 2 ? at_rank(shared_at(q_empty + q), 0) : shared_at(q_empty + q)); };
  // Waits until `need` tiles of matrix `at` are done (each of a tile's warps counts).
  auto wait_done = [&](int at, int need) -> bool {
    const unsigned* const counter = a.done + at;
    const unsigned all = static_cast<unsigned>(need) * (CG * kEndWarps);
    const long long from = clock64();
    for (;;) {
      unsigned seen;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(counter) : "memory");
      if (seen >= all) return true;
      if (*off != 0) return false;
      if (clock64() - from > 4 * kWaitCycles) {
        gave_up();
        return false;
      }
    }
  };
  // The stages of a part of a sum (every part has some: there are kPartStages times as many or more).
  auto part_of = [&](const Matrix& m, int kind, const Tile& t, int* b0, int* b1) {
    if (CG > 1 || kind != kGram || m.splits == 1) return;
    const int blocks = *b1;
    *b0 = blocks * t.split / m.splits;
    *b1 = blocks * (t.split + 1) / m.splits;
  };
  auto next_tile = [&](int i, Place* w, Tile* t) { return find_tile<CG, BN>(mat, count, phase, phases, tiles, i, w, t); };
  if (warp < 4) {
    fewer_registers();
    int stage = 0, acc = 0;
    uint32_t phase_bit = 0, acc_bit = 0;
    bool ok = true;
    Place w{0, 0, 0};
    Tile t;
    int q = 0;
    uint32_t q_bit = 0;
    if (warp == 0 && lane == 0) {
      // ---- copies
      int known_at = -1, known = 0;
      int mine = rank == 0 ? static_cast<int>(atomicAdd(a.ticket, 1u)) : 0;
      for (;;) {
        int i = mine;
        if (rank == 0) {
          if (!(ok = wait(q_empty + q, q_bit ^ 1))) break;
          q_tile[q] = i;
          bar_arrive(q_full + q);
          if constexpr (CG == 2) {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_rank(shared_at(q_tile + q), 1)), "r"(i) : "memory");
            bar_arrive_release(at_rank(shared_at(q_full + q), 1));
          }
        } else {
          if (!(ok = take(q, q_bit, &i))) break;
        }
        const bool more = next_tile(i, &w, &t);
        if (rank != 0) taken(q);
        if (++q == kQueue) q = 0, q_bit ^= 1;
        if (!more) break;
        const Matrix& m = mat[w.at];
        const int kind = phase[w.phase].kind, za = phase[w.phase].a, zb = phase[w.phase].b;
        const bool both = kind == kPoly || kind == kMul;   // both factors are symmetric
        const CUtensorMap* const map_a = kind == kGram ? &a.map[w.at].x : &a.map[w.at].s;
        const CUtensorMap* const map_b = both ? &a.map[w.at].s : &a.map[w.at].x;
        int b0 = 0, b1 = ((kind == kGram ? m.n : m.m) + kBlockK - 1) / kBlockK;
        part_of(m, kind, t, &b0, &b1);
        const int am = t.m0 + static_cast<int>(rank) * kTileM, bn = t.n0 + static_cast<int>(rank) * kBCta;
        if (w.at != known_at || w.need > known) {
          if (!(ok = wait_done(w.at, w.need))) break;
          known_at = w.at;
          known = w.need;
          asm volatile("fence.proxy.async;" ::: "memory");
        }
        for (int kb = b0; kb < b1; ++kb) {
          if (!(ok = wait(empty + stage, phase_bit ^ 1))) break;
          const uint32_t pa = shared_at(ring + stage * S::kStage), pb = pa + S::kA;
          uint32_t bar = shared_at(full + stage);
          if (rank == 0) bar_expect(full + stage, S::kStage * CG);
          if constexpr (CG == 2) bar = at_rank(bar, 0);
          const int k = kb * kBlockK;
          // (the next number is there when this tile's copies have been asked for)
          if (rank == 0 && kb == max(b0, b1 - 8)) mine = static_cast<int>(atomicAdd(a.ticket, 1u));
          if (a.stall == 0) {
            // of a symmetric factor, what lies below its diagonal tile is read from above, transposed
            const bool ta = kind != kGram && k < t.m0, tb = kind == kApply || (both && k < t.n0 / kRows * kRows);
#pragma unroll
            for (int j = 0; j < kTileM / 64; ++j)
              tma_load<CG>(pa + j * 8192, map_a, ta ? am + j * 64 : k, ta ? k : am + j * 64, za, bar);
#pragma unroll
            for (int j = 0; j < kBCta / 64; ++j)
              tma_load<CG>(pb + j * 8192, map_b, tb ? bn + j * 64 : k, tb ? k : bn + j * 64, zb, bar);
          }
          if (++stage == STAGES) stage = 0, phase_bit ^= 1;
        }
        if (!ok) break;
      }
      for (int i = 0; ok && i < STAGES; ++i) {   // the products' last arrivals have to find the barriers there
        ok = wait(empty + stage, phase_bit ^ 1);
        if (++stage == STAGES) stage = 0, phase_bit ^= 1;
      }
    }
    if (warp == 1 && lane == 0 && rank == 0) {
      // ---- products
      constexpr uint32_t idesc = (1u << 4) | (uint32_t{BN >> 3} << 17) | (uint32_t{kTileM * CG >> 4} << 24);
      for (;;) {
        int i;
        if (!(ok = take(q, q_bit, &i))) break;
        const bool more = next_tile(i, &w, &t);
        taken(q);
        if (++q == kQueue) q = 0, q_bit ^= 1;
        if (!more) break;
        const Matrix& m = mat[w.at];
        const int kind = phase[w.phase].kind;
        const bool both = kind == kPoly || kind == kMul;
        int b0 = 0, b1 = ((kind == kGram ? m.n : m.m) + kBlockK - 1) / kBlockK;
        part_of(m, kind, t, &b0, &b1);
        if (!(ok = wait(sum_empty + acc, acc_bit ^ 1))) break;
        fence_after();
        for (int kb = b0; kb < b1; ++kb) {
          if (!(ok = wait(full + stage, phase_bit))) break;
          fence_after();
          const uint32_t pa = shared_at(ring + stage * S::kStage), pb = pa + S::kA;
          const int k = kb * kBlockK;
          const bool ta = kind != kGram && k < t.m0, tb = kind == kApply || (both && k < t.n0 / kRows * kRows);
          const uint32_t a_step = ta ? 16 * 128 : 32, b_step = tb ? 16 * 128 : 32, a_lbo = ta ? 8192 : 16, b_lbo = tb ? 8192 : 16;
          const uint32_t form = idesc | ((ta ? 1u : 0u) << 15) | ((tb ? 1u : 0u) << 16);
#pragma unroll
          for (int j = 0; j < kBlockK / 16; ++j)
            mma<CG>(tmem + acc * BN, operand(pa + j * a_step, a_lbo, 1024), operand(pb + j * b_step, b_lbo, 1024), form, kb > b0 || j > 0);
          commit<CG>(empty + stage);
          if (++stage == STAGES) stage = 0, phase_bit ^= 1;
        }
        if (!ok) break;
        commit<CG>(sum_full + acc);
        if (++acc == 2) acc = 0, acc_bit ^= 1;
      }
    }
  } else {
    // ---- endings
    more_registers();
    const int group = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) * 32;
    int acc = 0;
    uint32_t acc_bit = 0;
    Part p;
    p.zero = p.bad = false;
    p.cols = BN / 2;
    p.ex = {exchange + (warp - 4) * kExchange, lane};
    float* const dj = columns + (warp - 4) * (BN / 2);
    Place w{0, 0, 0};
    int known_at = -1, known = 0, q = 0;
    uint32_t q_bit = 0;
    for (;;) {
      int i;
      const bool got = take(q, q_bit, &i);
      if (__any_sync(0xffffffffu, !got)) break;
      const bool more = next_tile(i, &w, &p.tile);
      if (lane == 0) taken(q);
      if (++q == kQueue) q = 0, q_bit ^= 1;
      if (!more) break;
      // (all that is known before the wait is looked up before it)
      const Matrix m = mat[w.at];
      const Phase ph = phase[w.phase];
      p.m = m.m;
      p.n = m.n;
      p.row = p.tile.m0 + static_cast<int>(rank) * kTileM + static_cast<int>(lanes) + lane;
      p.col = p.tile.n0 + group * p.cols;
      p.tmem = tmem + (lanes << 16) + acc * BN + group * p.cols;
      auto arrived = [&] {
        const bool there = wait(sum_full + acc, acc_bit);
        p.bad = __any_sync(0xffffffffu, !there) || p.bad;
        fence_after();
      };
      // of slab z: its blocks from this tile's on; its diagonal at this row
      const int64_t slab = block_at((p.m + 31) & ~31, 0, p.m);
      auto blocks_of = [&](int z) { return m.fb + (slab * z + block_at(p.row0(), p.col, p.m)); };
      auto diagonal_of = [&](int z) { return p.row < p.m ? m.dg[static_cast<int64_t>(z) * m.lda + p.row] : 0.f; };
      if (w.at != known_at || w.need > known) {
        bool done = true;
        if (lane == 0) done = wait_done(w.at, w.need);
        __syncwarp();   // (what lane 0 has seen, all have)
        p.bad = __any_sync(0xffffffffu, !done) || p.bad;
        known_at = w.at;
        known = w.need;
      }
      bool done = true;
      if (ph.kind == kGram) {
        arrived();
        if (CG == 1 && m.splits > 1)
          done = end_gram_part<BN / 2>(m, p, warp - 4);
        else
          end_gram(m, p, [&](int c, float (&v)[32]) { p.load(c, v); });
      } else if (ph.kind == kApply) {
        Ahead<8, BN / 64> x;
        x.fetch(p, m.xb + block_at(p.row0(), p.col, p.n), p.row0() < p.m, p.n - p.col);
        float factor = diagonal_of(ph.a);
        const int32_t status = *reinterpret_cast<const volatile int32_t*>(a.status);
        arrived();
        // (what a tile that was not finished has gone into: NaN, also where another CTA's NaNs came first)
        if (p.bad || status != 0) factor = __int_as_float(0x7fc00000);
        if (ph.last == 0)
          end_next(m, p, x, ph.b, factor, ph.c0);
        else if (out != kUpdate || (!p.bad && status == 0))   // (otherwise p stays as it is)
          end_last(m, p, x, factor, ph.c0, out, keep);
      } else {
        Ahead<4, BN / 64> f;
        f.fetch(p, blocks_of(ph.b), p.row0() < p.m, p.m - p.col);
        const float di = diagonal_of(ph.a), own = CG == 1 ? 0.f : diagonal_of(ph.b);
        // (beyond the last column the products are 0: the diagonal only has to be finite there)
        const float* const columns_of = m.dg + static_cast<int64_t>(ph.b) * m.lda;
#pragma unroll
        for (int c = 0; c < BN / 64; ++c) dj[32 * c + lane] = p.col + 32 * c + lane < p.m ? columns_of[p.col + 32 * c + lane] : 0.f;
        __syncwarp();
        if (CG == 1 || ph.kind == kPoly) {   // (one CTA a tile: no two steps at once)
          arrived();
          end_poly(m, p, f, di, dj, ph);
        } else {
          Ahead<4, BN / 64> u;
          u.fetch(p, blocks_of(ph.a), p.row0() < p.m, p.m - p.col);
          arrived();
          end_mul(m, p, u, f, di, own, dj, ph);
        }
      }
      fence_before();
      // what was written here is read by other CTAs' bulk copies
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        bar_arrive_cluster(CG == 2 ? at_rank(shared_at(sum_empty + acc), 0) : shared_at(sum_empty + acc));
        if (done) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.done + w.at) : "memory");
      }
      if (++acc == 2) acc = 0, acc_bit ^= 1;
    }
  }
  __syncwarp();
  __syncthreads();
  if (*off != 0 && threadIdx.x == 0) {
    // Copies and products that were under way when a wait ran out: they are done in microseconds.
    const long long from = clock64();
    while (clock64() - from < 2000000) {
    }
  }
  __syncthreads();
  if (*off != 0 && out != kUpdate) {
    // Tiles may have been left: the results say so.
    for (int k = 0; k < count; ++k) {
      const int64_t n = static_cast<int64_t>(mat[k].m) * mat[k].n;
      for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        if (out == kBf16Out)
          reinterpret_cast<__nv_bfloat16*>(mat[k].p)[i] = __float2bfloat16_rn(__int_as_float(0x7fc00000));
        else
          mat[k].p[i] = __int_as_float(0x7fc00000);
      }
    }
  }
  if constexpr (CG == 2) cluster_sync();
  if (warp == 2) tmem_free<CG>(tmem, kCols);
}

// ---- host side ------------------------------------------------------------------------
adaf_status fail(adaf_status st, const std::string& msg) { return meo::set_last_error(st, ("muon: " + msg).c_str()); }
adaf_status invalid(const std::string& msg) { return fail(ADAF_ERR_INVALID_ARGUMENT, msg); }
adaf_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(ADAF_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

const char* const kKernelNames[] = {"k_muon_moment", "k_muon_pack", "k_muon_iterate"};
constexpr int kNumKernels = 3;
enum Slot { kSlotMoment, kSlotPack, kSlotIterate };
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
struct Listed {
  int64_t m, n;
  int64_t rows, cols;
  float* p;
  const void* u;
  float* mom;
  int32_t flags;
};

adaf_status check_size(int64_t batch, int64_t rows, int64_t cols, const std::string& who) {
  if (batch < 0 || rows < 0 || cols < 0) return invalid(who + "negative size");
  if (batch == 0 || rows == 0 || cols == 0) return ADAF_OK;
  if (rows > kMaxSide || cols > kMaxSide || rows * cols > INT32_MAX)
    return fail(ADAF_ERR_UNSUPPORTED, who + "a side above 2^20 or more than 2^31 - 1 values a matrix");
  if (batch > kMaxMatrices) return fail(ADAF_ERR_UNSUPPORTED, who + "more than 2^20 matrices");
  return ADAF_OK;
}

// Bytes of a matrix in the workspace, and where its parts are.
struct Layout {
  size_t hi, xb, fe, fb, dg, bytes;
};
Layout layout(int64_t m, int64_t n, int slabs) {
  const int64_t ldx = round_up(n, 8), lda = round_up(m, 8);
  Layout L{};
  auto take = [&](int64_t bytes) {
    const size_t at = L.bytes;
    L.bytes += static_cast<size_t>(round_up(bytes, 256));
    return at;
  };
  L.hi = take(2 * m * ldx * 2);
  L.xb = take(round_up(m, 32) * round_up(n, 32) * 4);
  L.fe = take(slabs * m * lda * 2);
  L.fb = take(slabs * round_up(m, 32) * round_up(m, 32) * 2);
  L.dg = take(slabs * lda * 4);
  return L;
}
int32_t parts_of(int64_t m, int64_t n) {
  return static_cast<int32_t>(std::min<int64_t>(kMaxParts, (m * n + kPartValues - 1) / kPartValues));
}
constexpr size_t kHead = 256 + kMaxGroup * kMaxParts * 8 + (kMaxJoined * 4 + 255) / 256 * 256;   // the status word, the tiles' counters; the sums' parts; x x^T's
static_assert(4 + (kMaxGroup + 1) * 4 <= 256, "status, counters and the ticket");

// Matrices are worked on in the order of their sizes, the longest sums first; a
// group ends at so many matrices or values.
using Size = std::pair<int64_t, int64_t>;   // n, m
int64_t tiles_256(const Size& z) { return meo::tc::sym_tiles<1>((z.second + 255) / 256); }
// Matrices whose first two steps are worth taking at once, at least twice as wide as high: 4096 x
// 14336 has 13 % fewer flops then, 1024 x 4096 14 %, 4096 x 4096 3 % more.  They make groups of their
// own where their products fill the SMs (a list of small matrices is better off in one launch; from
// 30 tiles on 2048 x 8192 would gain 7 %, 4 x 1024 x 2048 lose as much).
bool wide(const Size& z) { return z.first >= 2 * z.second && z.second >= 1024; }
constexpr int64_t kFullTiles = 64;
struct Order {
  bool apart = false;   // wide ones are apart, and come first
  void look(const std::vector<std::pair<Size, int64_t>>& sizes) {
    int64_t tiles = 0;
    for (const auto& z : sizes)
      if (wide(z.first)) tiles += tiles_256(z.first) * z.second;
    apart = tiles >= kFullTiles;
  }
  // Of a matrix, and of all in its group.
  int slabs(const Size& z) const { return apart && wide(z) ? kPairSlabs : kSlabs; }
  bool before(const Size& x, const Size& y) const {
    return apart && wide(x) != wide(y) ? wide(x) : x > y;
  }
};
// In how many parts x x^T of a matrix is summed, if it were alone; of `tiles` tiles of all matrices.
int64_t parts_alone(int64_t n) { return std::max<int64_t>(1, std::min<int64_t>(kMostParts, (n + 63) / 64 / kPartStages)); }
int64_t gram_parts(int64_t n, int64_t tiles) {
  return 2 * tiles > kPartTiles ? 1 : std::min(parts_alone(n), kPartTiles / tiles);
}
// Bytes of the parts of a group, at most, in tiles of 128 x 128 and of 128 x 64.
struct GramParts {
  int64_t tiles[2] = {0, 0}, parts[2] = {0, 0};
  void add(const Size& z) {
    const int64_t of[2] = {meo::tc::sym_tiles<1>((z.second + 127) / 128), meo::tc::sym_tiles<2>((z.second + 63) / 64)};
    for (int k = 0; k < 2; ++k) {
      tiles[k] += of[k];
      if (parts_alone(z.first) > 1) parts[k] += of[k] * parts_alone(z.first);
    }
  }
  size_t bytes() const {
    size_t most = 0;
    for (int k = 0; k < 2; ++k)
      if (2 * tiles[k] <= kPartTiles) most = std::max(most, static_cast<size_t>(std::min<int64_t>(parts[k], kPartTiles)) * (128 * (k == 0 ? 128 : 64) * 4));
    return most;
  }
};
struct Grouping {
  const Order* order;
  GramParts parts;
  int64_t count = 0, values = 0;
  size_t bytes = kHead, most = 0;
  bool first_wide = false;
  // Whether a group that goes on with this matrix would be too large, or of two kinds.
  bool full(const Size& z) const {
    return count == kMaxGroup || (count > 0 && (values + z.first * z.second > kGroupValues || (order->apart && wide(z) != first_wide)));
  }
  void add(const Size& z) {
    if (full(z)) count = values = 0, bytes = kHead, parts = GramParts{};
    if (count == 0) first_wide = wide(z);
    ++count;
    values += z.first * z.second;
    bytes += layout(z.second, z.first, order->slabs(z)).bytes;
    parts.add(z);
    most = std::max(most, bytes + parts.bytes());
  }
};
size_t bytes_of(std::vector<std::pair<Size, int64_t>>& sizes) {
  Order order;
  order.look(sizes);
  std::stable_sort(sizes.begin(), sizes.end(), [&](const auto& x, const auto& y) { return order.before(x.first, y.first); });
  Grouping g{&order};
  for (const auto& z : sizes)
    for (int64_t b = 0; b < z.second; ++b) g.add(z.first);
  return g.most;
}

adaf_status check_tensors(const muon_tensor* tensors, int32_t n, size_t* bytes) {
  if (n < 0) return invalid("n < 0");
  if (n > 0 && tensors == nullptr) return invalid("tensors is NULL");
  std::vector<std::pair<Size, int64_t>> sizes;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const muon_tensor& t = tensors[i];
    const std::string who = "tensor " + std::to_string(i) + ": ";
    const adaf_status st = check_size(t.batch, t.rows, t.cols, who);
    if (st != ADAF_OK) return st;
    if (t.grad_dtype != ADAF_FLOAT32 && t.grad_dtype != ADAF_BFLOAT16) return invalid(who + "unknown grad_dtype");
    if (t.batch == 0 || t.rows == 0 || t.cols == 0) continue;
    if ((total += t.batch) > kMaxMatrices) return fail(ADAF_ERR_UNSUPPORTED, "more than 2^20 matrices");
    sizes.push_back({{std::max(t.rows, t.cols), std::min(t.rows, t.cols)}, t.batch});
  }
  *bytes = bytes_of(sizes);
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
  int32_t out;
  unsigned char* ws;
  cudaStream_t s;
};

#define MUON_TRY(expr, what)                          \
  do {                                                \
    const cudaError_t e_ = (expr);                    \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)

// Whether the first two steps' polynomials stay within what a product of them may be.
bool pair_fits(const muon_iteration& it) {
  if (it.steps < 2) return false;
  double top = 1.0, most = 1.0;
  for (int k = 0; k < 2; ++k) {
    double reach = 0.0, poly = 0.0;
    for (int i = 0; i <= 4096; ++i) {
      const double x = top * i / 4096, p = it.coef[k][0] + it.coef[k][1] * x * x + it.coef[k][2] * x * x * x * x;
      reach = std::max(reach, std::fabs(p * x));
      poly = std::max(poly, std::fabs(p));
    }
    top = reach;
    most *= poly;
  }
  return most <= 15.5;
}

// The phases of a call; gram, sym, app: tiles of all matrices in x x^T (its parts), in another
// symmetric product and in one with x.
int phases_of(const muon_iteration& it, bool pair, int64_t gram, int64_t sym, int64_t app, Phase* phase, int32_t* tiles) {
  int n = 0, x = 0;
  int32_t at = 0, syms = 0, apps = 0;
  auto add = [&](int kind, int a, int b, int out, double c0, double c1, double c2, bool last) {
    phase[n++] = {kind, a, b, out, static_cast<float>(c0), static_cast<float>(c1), static_cast<float>(c2), at, syms, apps, last ? 1 : 0};
    at += static_cast<int32_t>(kind == kApply ? app : kind == kGram ? gram : sym);
    ++(kind == kApply ? apps : syms);
  };
  auto poly = [&](int k, int in, int out) { add(kPoly, in, in, out, it.coef[k][0], it.coef[k][1], it.coef[k][2], false); };
  auto mul = [&](int a, int b, int out, int scale) { add(kMul, a, b, out, std::ldexp(1.0, scale - 2 * kSymScale), std::ldexp(1.0, scale - kSymScale), 0, false); };
  for (int k = 0; k < it.steps;) {
    add(kGram, x, x, 0, 0, 0, 0, false);
    poly(k, 0, 1);
    const bool two = pair && k == 0;
    if (two) {
      mul(1, 0, 2, kSymScale);    // P1 A1
      mul(2, 1, 0, kSymScale);    // A2 = P1 A1 P1
      poly(1, 0, 3);              // P2
      mul(3, 1, 2, kPairScale);   // P2 P1
    }
    k += two ? 2 : 1;
    add(kApply, two ? 2 : 1, x, 0, std::ldexp(1.0, -(two ? kPairScale : kSymScale)), 0, 0, k == it.steps);
    x ^= 1;
  }
  *tiles = at;
  return n;
}

template <int CG, int BN, int STAGES, int COUNT>
adaf_status iterate(const Call& c, const Listed* mats, int count, int slabs, bool pair) {
  using namespace meo::tc;
  auto* const kernel = k_muon_iterate<CG, BN, STAGES, COUNT>;
  constexpr int kBytes = Shared<CG, BN, STAGES>::bytes + kEndWarps * (BN / 2) * 4 + COUNT * sizeof(Matrix) + kMaxPhases * sizeof(Phase) + 8 +
                         kQueue * 20;
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
  IterateArgs<COUNT> a;
  std::memset(&a, 0, sizeof a);
  a.count = count;
  a.out = c.out;
  a.keep = c.hp != nullptr ? static_cast<float>(1.0 - c.hp->lr * c.hp->weight_decay) : 1.f;
  a.stall = t_stall ? 1 : 0;
  a.status = reinterpret_cast<int32_t*>(c.ws);
  a.done = reinterpret_cast<unsigned*>(c.ws) + 1;
  a.ticket = a.done + kMaxGroup;
  unsigned char* at = c.ws + kHead;
  int32_t gram = 0, sym = 0, app = 0;
  int64_t grams = 0;   // tiles of x x^T
  constexpr int kRows = kTileM * CG;
  for (int i = 0; i < count; ++i) grams += sym_tiles<kRows / BN>((mats[i].m + BN - 1) / BN);
  for (int i = 0; i < count; ++i) {
    const Listed& z = mats[i];
    const Layout L = layout(z.m, z.n, slabs);
    Matrix& m = a.mat[i];
    m.hi = reinterpret_cast<__half*>(at + L.hi);
    m.xb = reinterpret_cast<float*>(at + L.xb);
    m.fe = reinterpret_cast<__half*>(at + L.fe);
    m.fb = reinterpret_cast<__half*>(at + L.fb);
    m.dg = reinterpret_cast<float*>(at + L.dg);
    at += L.bytes;
    m.p = z.p;
    m.m = static_cast<int32_t>(z.m);
    m.n = static_cast<int32_t>(z.n);
    m.ldx = static_cast<int32_t>(round_up(z.n, 8));
    m.lda = static_cast<int32_t>(round_up(z.m, 8));
    m.flags = z.flags;
    if (c.hp != nullptr) {
      const double h = static_cast<double>(z.rows), w = static_cast<double>(z.cols);
      const bool original = c.hp->adjust_lr == MUON_ADJUST_ORIGINAL;
      m.rate = static_cast<float>(c.hp->lr * (original ? std::sqrt(std::max(1.0, h / w)) : 0.2 * std::sqrt(std::max(h, w))));
    }
    if (!make_map(&a.map[i].x, m.hi, false, z.m, z.n, m.ldx, 2, z.m * m.ldx, 64) ||
        !make_map(&a.map[i].s, m.fe, false, z.m, z.m, m.lda, slabs, z.m * m.lda, 64))
      return fail(ADAF_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    const int64_t mt = (z.m + kRows - 1) / kRows, nt = (z.n + BN - 1) / BN;
    const int32_t own = static_cast<int32_t>(sym_tiles<kRows / BN>((z.m + BN - 1) / BN));
    m.sym0 = sym;
    m.app0 = app;
    m.gram0 = gram;
    m.splits = CG == 1 ? static_cast<int32_t>(gram_parts(z.n, grams)) : 1;
    sym += own;
    app += static_cast<int32_t>(mt * nt);
    gram += own * m.splits;
  }
  unsigned* joined = reinterpret_cast<unsigned*>(c.ws + kHead) - kMaxJoined;
  for (int i = 0; i < count; ++i) {
    Matrix& m = a.mat[i];
    if (m.splits == 1) continue;
    const int64_t own = sym_tiles<kRows / BN>((m.m + BN - 1) / BN);
    m.parts = reinterpret_cast<float*>(at);
    m.joined = joined;
    at += own * m.splits * (kTileM * BN * 4);
    joined += own * kEndWarps;
  }
  a.phases = phases_of(*c.it, pair, gram, sym, app, a.phase, &a.tiles);
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = c.s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {CG, 1, 1};
  cfg.numAttrs = CG > 1 ? 2 : 1;
  static std::atomic<unsigned long long> ready{0};   // devices whose limit has been raised
  int device = 0, sms = 0;
  MUON_TRY(sm_count(&device, &sms), "current device");
  const unsigned long long bit = device < 64 ? 1ull << device : 0;
  if (bit == 0 || (ready.load() & bit) == 0) {
    MUON_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes), "k_muon_iterate");
    ready.fetch_or(bit);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(sms / CG, std::max(gram, app)) * CG));
  MUON_TRY(g_profile.run(kSlotIterate, c.s, [&] { return cudaLaunchKernelEx(&cfg, kernel, a); }), "k_muon_iterate");
  return ADAF_OK;
}

// About how many microseconds a step takes with tiles of `side` x `side` on `slots` SMs or pairs of
// them: stages of a tile, each bound by its copies, and its way from and to the tiles around it.  The
// constants are measured; of tiles of 128 and 256 it chooses the faster, or one 3 % behind, for
// 1024 x 4096 (258 us, 281), 2048 x 2048 (335, 295), 2048 x 8192 (814, 710), 4 x 1024 x 1024 (208, 219),
// 3 x 1024 x 4096 (430, 379), 1536 x 1536 (227, 238), 5 x 700 x 900 (205, 212), 10 x 512 x 2048 (300, 285).
double step_time(const Listed* mats, int count, int64_t side, int slots, double stage, double ending) {
  const auto cut = [](int64_t x, int64_t by) { return (x + by - 1) / by; };
  int64_t grams = 0;
  for (int i = 0; i < count; ++i) grams += meo::tc::sym_tiles<1>(cut(mats[i].m, side));
  double sum[3] = {0, 0, 0}, most[3] = {0, 0, 0};
  for (int i = 0; i < count; ++i) {
    const int64_t m = mats[i].m, n = mats[i].n, sym = meo::tc::sym_tiles<1>(cut(m, side));
    const int64_t parts = side == 128 ? gram_parts(n, grams) : 1;
    const double tiles[3] = {static_cast<double>(sym * parts), static_cast<double>(sym), static_cast<double>(cut(m, side) * cut(n, side))};
    const double one[3] = {static_cast<double>(cut(cut(n, 64), parts)) * stage + ending + (parts > 1 ? 3.0 : 0.0),
                           static_cast<double>(cut(m, 64)) * stage + ending, static_cast<double>(cut(m, 64)) * stage + ending};
    for (int k = 0; k < 3; ++k) {
      sum[k] += tiles[k] * one[k];
      most[k] = std::max(most[k], one[k]);
    }
  }
  double time = 0;
  for (int k = 0; k < 3; ++k) time += std::max(sum[k] / slots, most[k]);
  return time;
}

template <bool STEP>
adaf_status run_group(const Call& c, const Listed* mats, int count, bool first, const Order& order) {
  MuonArgs a;
  std::memset(&a, 0, sizeof a);
  a.count = count;
  a.stride_r = c.stride_r;
  a.eps = static_cast<float>(c.it->eps);
  if (STEP) {
    a.mu = static_cast<float>(c.hp->momentum);
    a.nesterov_mu = c.hp->nesterov != 0 ? a.mu : -1.f;
  }
  a.status = reinterpret_cast<int32_t*>(c.ws);
  a.done = reinterpret_cast<unsigned*>(c.ws) + 1;
  a.part = reinterpret_cast<float2*>(c.ws + 256);
  a.joined = reinterpret_cast<unsigned*>(c.ws + kHead) - kMaxJoined;
  a.clear = first ? 1 : 0;
  const int slabs = order.slabs({mats[0].n, mats[0].m});
  unsigned char* at = c.ws + kHead;
  int32_t parts = 0, tiles = 0;
  int64_t big = 0, small = 0;   // tiles of 256 x 256 of a symmetric product, of 128 x 128 of the last one
  for (int i = 0; i < count; ++i) {
    const Listed& z = mats[i];
    const Layout L = layout(z.m, z.n, slabs);
    Item& t = a.item[i];
    t.u = z.u;
    t.mom = z.mom;
    t.hi = reinterpret_cast<__half*>(at + L.hi);
    t.x = reinterpret_cast<float*>(at + L.xb);
    at += L.bytes;
    t.rows = static_cast<int32_t>(z.rows);
    t.cols = static_cast<int32_t>(z.cols);
    t.m = static_cast<int32_t>(z.m);
    t.n = static_cast<int32_t>(z.n);
    t.ldx = static_cast<int32_t>(round_up(z.n, 8));
    t.flags = z.flags;
    t.parts = parts_of(z.m, z.n);
    t.part0 = parts;
    t.tile0 = tiles;
    parts += t.parts;
    tiles += static_cast<int32_t>(((z.m + 63) / 64) * ((z.n + 63) / 64));
    big += tiles_256({z.n, z.m});
    small += ((z.m + 127) / 128) * ((z.n + 127) / 128);
  }
  MUON_TRY(g_profile.run(kSlotMoment, c.s, [&] {
    k_muon_moment<STEP><<<static_cast<unsigned>(parts), 256, 0, c.s>>>(a);
    return cudaGetLastError();
  }), "k_muon_moment");
  MUON_TRY(g_profile.run(kSlotPack, c.s, [&] {
    return meo::tc::launch_early(k_muon_pack<STEP>, dim3(static_cast<unsigned>(tiles)), 256, c.s, a);
  }), "k_muon_pack");
  int device = 0, sms = 0;
  MUON_TRY(meo::tc::sm_count(&device, &sms), "current device");
  // (a group's matrices are all wide, or none is)
  const bool pair = slabs == kPairSlabs && big >= kFullTiles && pair_fits(*c.it);
  // Narrow tiles where each of them has an SM: half as much to load and to write out a tile, for
  // 256 x 512 102 us to 115, six matrices of 256 x 256 to 1024 126 to 140; 1403 x 777, where two
  // rounds would be needed, 198 to 175.
  if (!pair && 2 * small <= sms) return count <= kFew ? iterate<1, 64, 8, kFew>(c, mats, count, slabs, false) : iterate<1, 64, 8, kMaxGroup>(c, mats, count, slabs, false);
  if (!pair && step_time(mats, count, 128, sms, 0.29, 1.5) < step_time(mats, count, 256, sms / 2, 0.27, 3.5))
    return count <= kFew ? iterate<1, 128, 6, kFew>(c, mats, count, slabs, false) : iterate<1, 128, 6, kMaxGroup>(c, mats, count, slabs, false);
  return count <= kFew ? iterate<2, 256, 6, kFew>(c, mats, count, slabs, pair) : iterate<2, 256, 6, kMaxGroup>(c, mats, count, slabs, pair);
}

template <bool STEP>
adaf_status run(const Call& c, std::vector<Listed>& mats) {
  std::vector<std::pair<Size, int64_t>> sizes;
  for (const Listed& z : mats) sizes.push_back({{z.n, z.m}, 1});
  Order order;
  order.look(sizes);
  std::stable_sort(mats.begin(), mats.end(), [&](const Listed& x, const Listed& y) { return order.before({x.n, x.m}, {y.n, y.m}); });
  bool first = true;
  for (size_t i = 0; i < mats.size();) {
    Grouping g{&order};
    size_t j = i;
    for (; j < mats.size() && !g.full({mats[j].n, mats[j].m}); ++j) g.add({mats[j].n, mats[j].m});
    const adaf_status st = run_group<STEP>(c, &mats[i], static_cast<int>(j - i), first, order);
    if (st != ADAF_OK) return st;
    first = false;
    i = j;
  }
  return ADAF_OK;
}

// Bytes for a stack of matrices.
size_t bytes_of(int64_t batch, int64_t rows, int64_t cols) {
  std::vector<std::pair<Size, int64_t>> sizes;
  if (batch > 0 && rows > 0 && cols > 0) sizes.push_back({{std::max(rows, cols), std::min(rows, cols)}, batch});
  return bytes_of(sizes);
}

// Tensors that share memory: a step writes p and momentum of all of them at once, and reads g beside that.
struct Extent {
  uintptr_t from, to;
  int32_t tensor;
  bool written;
};
adaf_status check_apart(std::vector<Extent>& all) {
  std::sort(all.begin(), all.end(), [](const Extent& x, const Extent& y) { return x.from < y.from; });
  // the furthest end so far, of what is written and of everything
  const Extent *written = nullptr, *any = nullptr;
  for (const Extent& e : all) {
    const Extent* const other = e.written ? any : written;
    if (other != nullptr && other->to > e.from) {
      const int32_t lo = std::min(e.tensor, other->tensor), hi = std::max(e.tensor, other->tensor);
      return invalid(lo == hi ? "tensor " + std::to_string(lo) + ": p, g and momentum overlap"
                              : "tensors " + std::to_string(lo) + " and " + std::to_string(hi) + " overlap");
    }
    if (any == nullptr || e.to > any->to) any = &e;
    if (e.written && (written == nullptr || e.to > written->to)) written = &e;
  }
  return ADAF_OK;
}

adaf_status step(const muon_tensor* tensors, int32_t n, const muon_hparams* hp, void* workspace, size_t workspace_bytes, void* stream) {
  adaf_status st = check_hp(hp);
  if (st != ADAF_OK) return st;
  size_t need = 0;
  if ((st = check_tensors(tensors, n, &need)) != ADAF_OK) return st;
  std::vector<Listed> mats;
  std::vector<Extent> extents;
  extents.reserve(3 * static_cast<size_t>(n));
  for (int32_t i = 0; i < n; ++i) {
    const muon_tensor& t = tensors[i];
    if (t.batch == 0 || t.rows == 0 || t.cols == 0) continue;
    const std::string who = "tensor " + std::to_string(i);
    if (t.p == nullptr || t.g == nullptr || t.momentum == nullptr) return invalid(who + " has a NULL pointer");
    const size_t es = t.grad_dtype == ADAF_BFLOAT16 ? 2 : 4;
    if (!aligned(t.p, 4) || !aligned(t.momentum, 4) || !aligned(t.g, es)) return invalid(who + " is not element-aligned");
    const int64_t numel = t.rows * t.cols;
    const auto extent = [&](const void* p, size_t size, bool written) {
      const uintptr_t from = reinterpret_cast<uintptr_t>(p);
      extents.push_back({from, from + static_cast<size_t>(t.batch * numel) * size, i, written});
    };
    extent(t.p, 4, true);
    extent(t.g, es, false);
    extent(t.momentum, 4, true);
    for (int64_t b = 0; b < t.batch; ++b)
      mats.push_back({std::min(t.rows, t.cols), std::max(t.rows, t.cols), t.rows, t.cols, t.p + b * numel,
                      static_cast<const char*>(t.g) + static_cast<size_t>(b * numel) * es, t.momentum + b * numel,
                      (t.rows > t.cols ? kTurned : 0) | (es == 2 ? kBf16 : 0)});
  }
  if (mats.empty()) return ADAF_OK;
  if ((st = check_apart(extents)) != ADAF_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != ADAF_OK) return st;
  const Call c{&hp->iteration, hp, 0, kUpdate, static_cast<unsigned char*>(workspace), static_cast<cudaStream_t>(stream)};
  return run<true>(c, mats);
}

adaf_status orthogonalize(const muon_matrices* x, const muon_iteration* it, void* out, int32_t out_dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  adaf_status st = check_iteration(it);
  if (st != ADAF_OK) return st;
  if (x == nullptr) return invalid("x is NULL");
  size_t need = 0;
  if ((st = check_size(x->batch, x->rows, x->cols, "")) != ADAF_OK) return st;
  need = bytes_of(x->batch, x->rows, x->cols);
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
  std::vector<Listed> mats;
  for (int64_t b = 0; b < x->batch; ++b)
    mats.push_back({std::min(x->rows, x->cols), std::max(x->rows, x->cols), x->rows, x->cols,
                    reinterpret_cast<float*>(static_cast<char*>(out) + static_cast<size_t>(b * numel) * os),
                    static_cast<const char*>(x->x) + static_cast<size_t>(b * x->stride_b) * es, nullptr,
                    (x->rows > x->cols ? kTurned : 0) | (es == 2 ? kBf16 : 0)});
  const Call c{it, nullptr, x->rows == 1 ? x->cols : x->stride_r, os == 2 ? kBf16Out : kFp32,
               static_cast<unsigned char*>(workspace), static_cast<cudaStream_t>(stream)};
  return run<false>(c, mats);
}

// Nothing thrown leaves a C entry point (long lists take host memory).
template <class Body>
adaf_status guarded(Body&& body) {
  try {
    return body();
  } catch (const std::exception&) {
    return fail(ADAF_ERR_UNSUPPORTED, "out of host memory");
  }
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
  return guarded([&] { return check_tensors(tensors, n, bytes); });
}

adaf_status muon_orthogonalize_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
  if (bytes == nullptr) return invalid("bytes is NULL");
  const adaf_status st = check_size(batch, rows, cols, "");
  if (st != ADAF_OK) return st;
  return guarded([&] {
    *bytes = bytes_of(batch, rows, cols);
    return ADAF_OK;
  });
}

adaf_status muon_step(const muon_tensor* tensors, int32_t n, const muon_hparams* hp, void* workspace, size_t workspace_bytes,
                      void* stream) {
  return guarded([&] { return step(tensors, n, hp, workspace, workspace_bytes, stream); });
}

adaf_status muon_orthogonalize(const muon_matrices* x, const muon_iteration* it, void* out, int32_t out_dtype, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return guarded([&] { return orthogonalize(x, it, out, out_dtype, workspace, workspace_bytes, stream); });
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
