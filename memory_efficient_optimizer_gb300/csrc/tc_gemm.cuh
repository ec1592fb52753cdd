// Products of matrices on the tensor cores of sm_103a, with the work on each
// result tile given by the caller (the "ending").
//
//   D[i, j] = sum over k of A[i, k] B[j, k]
//
// A and B are 16-bit, both bf16 in k_product (fp16 in Muon's iteration, which has
// the parts below in a kernel of its own), each either with k innermost
// ("K-major") or with i or j innermost ("MN-major"); sums are fp32.
//
// Layout.  A tile of the result is 128 CG rows by BN columns, CG = 2: the two
// CTAs of a cluster work on one tile with tcgen05 instructions that read both
// CTAs' shared memory, so each CTA loads its own 128 rows of A and half of the
// tile's columns of B, half of what two CTAs apart would.  A persistent grid
// walks the tiles.  In a CTA
//
//   warp 0     copies the operands' tiles of 64 k values into a ring of
//              stages (TMA, 128-byte swizzle; it also zero-fills what lies
//              beyond the matrices, so no size has to be a multiple of anything)
//   warp 1     issues the products (one thread, of the cluster's first CTA)
//   warp 2     holds the tensor memory
//   warps 4..  take the finished tile out of tensor memory (the ending), while
//              the next tile is summed in the other half of it
//
// What bounds it: at 256 x 256 x 64 a CTA's stage is 32 KB for 512 cycles of
// the tensor cores, 64 bytes a cycle, which L2 just gives; smaller tiles are
// bound by those copies and are taken where there are too few large ones.
//
// Every wait is bounded.  One that runs out sets the kernel's status word and
// the CTA's flag: its tiles' values are NaN from then on, nothing more is
// waited for, and the CTA ends after its copies have had time to land.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace meo {
namespace tc {
namespace {

constexpr int kBlockK = 64;        // k values of a stage: 128 bytes, the swizzle's width
constexpr int kTileM = 128;        // rows of a CTA
constexpr int kEndWarps = 8;       // two groups of four warps, each half of the columns
constexpr int kThreads = 128 + 32 * kEndWarps;
constexpr long long kWaitCycles = 2000000000LL;   // about a second

__device__ __forceinline__ uint32_t shared_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t arrivals) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_at(bar)), "r"(arrivals) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_at(bar)), "r"(bytes) : "memory");
}
// Address of the same place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// (relaxed: what it tells of is tensor memory, which the tcgen05 fences order; a release at
// cluster scope waits for the thread's global stores, a microsecond or two at every tile)
__device__ __forceinline__ void bar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_at(bar)) : "memory");
}
// For a word written to another CTA's shared memory, and for who waits for it there.
__device__ __forceinline__ void bar_arrive_release(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool bar_try_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(shared_at(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(shared_at(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Instructions that are ".aligned" are for a whole warp together: each of the functions that hold one begins
// by bringing its lanes together, whatever branches and loops they come from.
//
// The endings' warps take registers over from the first four (at launch all have 168: 384
// threads of 65536): 128 x 56 + 256 x 224 = 64512, what the block holds.  Each is
// called by all warps of its kind at the head of their branch.
__device__ __forceinline__ void fewer_registers() {
  __syncwarp();
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}
__device__ __forceinline__ void more_registers() {
  __syncwarp();
  asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A kernel launched to begin while the one before it on the stream ends waits here until that
// one is done and what it wrote is there.
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- tcgen05 ------------------------------------------------------------------------
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols) {
  __syncwarp();
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_at(where)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_at(where)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
  __syncwarp();
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  const uint32_t p = add ? 1u : 0u;
  if constexpr (CG == 2)
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(p)
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(p)
                 : "memory");
}
// `bar` (of both CTAs of a pair) gets one arrival when the products issued before are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     shared_at(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(shared_at(bar)) : "memory");
}
// 32 columns of the warp's 32 lanes (rows).
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[32]) {
  __syncwarp();
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, "
      "%26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 64 columns, both halves under way together.
__device__ __forceinline__ void tmem_load64(uint32_t at, float (&v)[32], float (&w)[32]) {
  __syncwarp();
  uint32_t r[32], q[32];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t(&t)[32] = half == 0 ? r : q;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, "
        "%26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(t[0]), "=r"(t[1]), "=r"(t[2]), "=r"(t[3]), "=r"(t[4]), "=r"(t[5]), "=r"(t[6]), "=r"(t[7]), "=r"(t[8]), "=r"(t[9]),
          "=r"(t[10]), "=r"(t[11]), "=r"(t[12]), "=r"(t[13]), "=r"(t[14]), "=r"(t[15]), "=r"(t[16]), "=r"(t[17]), "=r"(t[18]),
          "=r"(t[19]), "=r"(t[20]), "=r"(t[21]), "=r"(t[22]), "=r"(t[23]), "=r"(t[24]), "=r"(t[25]), "=r"(t[26]), "=r"(t[27]),
          "=r"(t[28]), "=r"(t[29]), "=r"(t[30]), "=r"(t[31])
        : "r"(at + 32 * half));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]), w[i] = __uint_as_float(q[i]);
}
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&v)[16]) {
  __syncwarp();
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Descriptor of an operand in shared memory, 128-byte swizzle: rows of 128 bytes,
// groups of 8 rows 1024 bytes apart (`sbo`).  K-major: a row is 64 k values of one
// i or j.  MN-major: a row is 64 i or j of one k; blocks of 64 i or j `lbo` apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

template <int CG>
__device__ __forceinline__ void tma_load(uint32_t to, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            to),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     to),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

// ---- a tile's rows and memory --------------------------------------------------------
// In an ending a lane holds a row of the result, 64 bytes of it at a time.  Read or
// written that way, an instruction touches 32 rows, 16 bytes of each, and a tile of
// 128 x 256 took 5 us (bf16) to 15 us (two fp16 in, two out).  Through 2.5 KB of
// shared memory a warp, four lanes side by side hold a row's 64 bytes.
constexpr int kPitch = 80;                       // of a row in shared memory
constexpr int kExchange = 32 * kPitch;           // bytes of a warp

struct Exchange {
  unsigned char* at;
  int lane;
  __device__ __forceinline__ void to_rows(uint4 (&w)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(at + (8 * i + (lane >> 2)) * kPitch + (lane & 3) * 16) = w[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(at + lane * kPitch + 16 * i);
    __syncwarp();
  }
  __device__ __forceinline__ void to_memory(uint4 (&w)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(at + lane * kPitch + 16 * i) = w[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(at + (8 * i + (lane >> 2)) * kPitch + (lane & 3) * 16);
    __syncwarp();
  }
  // In memory order: lane l has 16 bytes from byte place() of rows row(0) .. row(3) of the warp's.
  __device__ __forceinline__ int row(int i) const { return 8 * i + (lane >> 2); }
  __device__ __forceinline__ int place() const { return (lane & 3) * 16; }
  // 64 bytes of each of `rows` rows from p on, `pitch` bytes apart, of which `left` (a multiple
  // of 16) are there; zeros beyond.
  __device__ __forceinline__ void fetch(const void* p, int64_t pitch, int rows, int left, uint4 (&w)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = make_uint4(0, 0, 0, 0);
      if (row(i) < rows && place() < left) w[i] = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p) + row(i) * pitch + place());
    }
  }
  __device__ __forceinline__ void put(void* p, int64_t pitch, int rows, int left, const uint4 (&w)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row(i) < rows && place() < left) *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p) + row(i) * pitch + place()) = w[i];
  }
};

// ---- the product --------------------------------------------------------------------
struct Shape {
  int32_t m, n, k;
  int32_t splits;          // parts of k, each a result of its own; 0: as choose_splits has it
  int64_t split_room;      // then: values that the parts' results may take
  int32_t group;           // tiles are walked in groups of so many rows of tiles
  const int32_t* m_live;   // not NULL: the rows that count (on the device) are *m_live - first, at most m
  const int32_t* k_live;   // the same for k
  int32_t first;
  int32_t* status;         // bit 0: a wait ran out
  int32_t stall;           // testing: make no copies
};

struct Tile {
  int32_t split, m0, n0;   // the cluster tile's first row and column
  int32_t number;          // of the tile, where Muon's iteration needs it
};

// What an ending is given: a row of the result a thread, and the columns of its group.
struct Part {
  Tile tile;
  int32_t row;            // of the result
  int32_t col, cols;      // its columns: col, ..., col + cols - 1 (a multiple of 32)
  int32_t m, n;
  uint32_t tmem;
  Exchange ex;            // of the warp
  int32_t splits;
  bool zero, bad;         // there was nothing to sum; a wait ran out
  __device__ __forceinline__ int row0() const { return row - ex.lane; }   // the warp's first row
  __device__ __forceinline__ void load64(int c, float (&v)[32], float (&w)[32]) const {
    tmem_load64(tmem + c, v, w);
    if (zero || bad) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = w[i] = bad ? __int_as_float(0x7fc00000) : 0.f;
    }
  }
  __device__ __forceinline__ void load(int c, float (&v)[32]) const {
    tmem_load(tmem + c, v);
    if (zero || bad) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = bad ? __int_as_float(0x7fc00000) : 0.f;
    }
  }
};

// In how many parts to sum, so that the tiles' parts come out near a multiple of the clusters that
// work on them.  `blocks`: stages of a whole sum; a part more costs a write and a read of the result,
// `cost` stages' time.  96 tiles on 76 clusters are two rounds; in three parts 1.3.
__host__ __device__ inline int choose_splits(uint32_t tiles, uint32_t blocks, uint32_t clusters, uint32_t most, uint32_t cost) {
  uint32_t best = 1, least = 0xffffffffu;
  for (uint32_t s = 1; s <= 16 && s <= most && (s == 1 || blocks >= 16 * s); ++s) {
    const uint32_t time = (tiles * s + clusters - 1) / clusters * ((blocks + s - 1) / s) + (s > 1 ? cost * s : 0);
    if (time < least) least = time, best = s;
  }
  return static_cast<int>(best);
}
// The same for a result of m x n values, in tiles of tm x tn, with room for so many values.  (A
// result so large that this overflows 32 bits is summed in one part.)
__host__ __device__ inline int splits_of(int m, int n, int blocks, int tm, int tn, int clusters, int64_t room) {
  const int64_t values = static_cast<int64_t>(m) * n;
  if (values == 0 || 2 * values > room) return 1;
  const uint32_t tiles = static_cast<uint32_t>((m + tm - 1) / tm) * static_cast<uint32_t>((n + tn - 1) / tn);
  return choose_splits(tiles, blocks, clusters, static_cast<uint32_t>(room / values < 16 ? room / values : 16),
                       static_cast<uint32_t>(values >> 18) + 1);
}

__device__ __forceinline__ int live(const int32_t* p, int32_t first, int32_t most) {
  if (p == nullptr) return most;
  const int n = *p - first;
  return n < 0 ? 0 : n < most ? n : most;
}

// Tiles of a symmetric result on and above its diagonal: TM rows by TN columns, TM / TN = R
// column tiles a row tile; column tile c has the row tiles 0 .. c / R.
template <int R>
__host__ __device__ constexpr int64_t sym_tiles(int64_t columns) {
  static_assert(R >= 1, "whole column tiles");
  const int64_t q = columns / R, rest = columns % R;
  return R * (q * (q + 1) / 2) + rest * (q + 1);
}

// The tile of number i of a matrix's; false beyond the last.
template <bool SYM, int TM, int TN>
__device__ __forceinline__ bool tile_of(int64_t i, int mt, int nt, const Shape& s, Tile* t) {
  constexpr int R = TM / TN;
  const int64_t per = SYM ? sym_tiles<SYM ? R : 1>(nt) : static_cast<int64_t>(mt) * nt * s.splits;
  if (i >= per) return false;
  int r = static_cast<int>(i);
  if constexpr (SYM) {
    // groups of R columns: group q has R (q + 1) tiles, R q (q + 1) / 2 before it
    int q = static_cast<int>((sqrtf(8.f / R * static_cast<float>(r) + 1.f) - 1.f) * 0.5f);
    while (R * (q * (q + 1) / 2) > r) --q;
    while (R * ((q + 1) * (q + 2) / 2) <= r) ++q;
    r -= R * (q * (q + 1) / 2);
    t->m0 = r % (q + 1) * TM;
    t->n0 = (R * q + r / (q + 1)) * TN;
    t->split = 0;
  } else {
    t->split = r / (mt * nt);
    r -= t->split * (mt * nt);
    const int g = r / (s.group * nt);            // group of rows of tiles
    const int left = mt - g * s.group, high = left < s.group ? left : s.group;
    r -= g * s.group * nt;
    t->n0 = r / high * TN;
    t->m0 = (g * s.group + r % high) * TM;
  }
  return true;
}

template <int CG, int BN, int STAGES>
struct Shared {
  static constexpr int kA = kTileM * kBlockK * 2;        // bytes of a stage of a CTA
  static constexpr int kB = BN / CG * kBlockK * 2;
  static constexpr int kStage = kA + kB;
  static constexpr int kBars = 2 * STAGES + 4;
  static constexpr int bytes = STAGES * kStage + kEndWarps * kExchange + kBars * 8 + 64 + 1024;   // and the alignment to 1024
};

// End: what is done with a result tile.
//   struct Args;
//   static constexpr int kChunk = 0;   static __device__ void part(const Args&, const Part&)
// or, with kChunk > 0, static __device__ void whole(const Args&, const Part&, float (&v)[BN / 2]):
// the sums are taken out of tensor memory every kChunk stages and added up in registers.  The
// tensor cores cut off what does not fit a sum's 24 bits, so a long sum is off toward zero by
// half of 2^-25 of itself and more for each of its steps of 16 values.
template <int CG, int BN, int STAGES, bool A_MN, bool B_MN, class End>
__global__ void __launch_bounds__(kThreads, 1)
    k_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Shape given,
              const typename End::Args end) {
  Shape s = given;
  using S = Shared<CG, BN, STAGES>;
  constexpr uint32_t kCols = 2 * BN;      // two accumulators
  constexpr int kBCta = BN / CG;          // rows of B (columns of the result) that a CTA loads
  extern __shared__ unsigned char raw[];
  unsigned char* ring = raw + ((1024 - (shared_at(raw) & 1023)) & 1023);
  unsigned char* const exchange = ring + STAGES * S::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(exchange + kEndWarps * kExchange);
  uint64_t* empty = full + STAGES;
  uint64_t* sum_full = empty + STAGES;
  uint64_t* sum_empty = sum_full + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sum_empty + 2);
  volatile int* off = reinterpret_cast<volatile int*>(tmem_at + 1);   // a wait of this CTA ran out

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int64_t first = blockIdx.x / CG, step = gridDim.x / CG;
  next_may_begin();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      bar_init(full + i, 1);
      bar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(sum_full + i, 1);
      bar_init(sum_empty + i, CG * kEndWarps);
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
  const int m = live(s.m_live, s.first, s.m), k_all = live(s.k_live, s.first, s.k);
  const int mt = (m + kTileM * CG - 1) / (kTileM * CG), nt = (s.n + BN - 1) / BN;
  const int blocks = (k_all + kBlockK - 1) / kBlockK;
  if (s.splits == 0) s.splits = splits_of(m, s.n, blocks, kTileM * CG, BN, gridDim.x / CG, s.split_room);
  const int per_split = (blocks + s.splits - 1) / s.splits;

  // False if the wait ran out, or another of the CTA's had before.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (bar_try(bar, parity)) return true;
    const long long from = clock64();
    while (!bar_try(bar, parity)) {
      if (*off != 0) return false;
      if (clock64() - from > kWaitCycles) {
        *off = 1;
        atomicOr(s.status, 1);
        return false;
      }
    }
    return true;
  };

  if (warp < 4) {
    fewer_registers();
    if (warp == 0 && lane == 0) {
      // ---- copies
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Tile t;
      for (int64_t i = first; ok && tile_of<false, kTileM * CG, BN>(i, mt, nt, s, &t); i += step) {
        const int b0 = t.split * per_split, b1 = min(blocks, b0 + per_split);
        const int am = t.m0 + static_cast<int>(rank) * kTileM, bn = t.n0 + static_cast<int>(rank) * kBCta;
        for (int kb = b0; kb < b1; ++kb) {
          if (!(ok = wait(empty + stage, phase ^ 1))) break;
          const uint32_t a = shared_at(ring + stage * S::kStage), b = a + S::kA;
          uint32_t bar = shared_at(full + stage);
          if (rank == 0) bar_expect(full + stage, S::kStage * CG);
          if constexpr (CG == 2) bar = at_rank(bar, 0);
          const int k = kb * kBlockK;
          if (s.stall == 0) {
            if constexpr (A_MN) {
#pragma unroll
              for (int j = 0; j < kTileM / 64; ++j) tma_load<CG>(a + j * 64 * kBlockK * 2, &map_a, am + j * 64, k, 0, bar);
            } else {
              tma_load<CG>(a, &map_a, k, am, 0, bar);
            }
            if constexpr (B_MN) {
#pragma unroll
              for (int j = 0; j < kBCta / 64; ++j) tma_load<CG>(b + j * 64 * kBlockK * 2, &map_b, bn + j * 64, k, 0, bar);
            } else {
#pragma unroll
              for (int j = 0; j < kBCta / 128; ++j) tma_load<CG>(b + j * 128 * kBlockK * 2, &map_b, k, bn + j * 128, 0, bar);
            }
          }
          if (++stage == STAGES) stage = 0, phase ^= 1;
        }
      }
      // The products' last arrivals have to find this CTA's barriers there.
      for (int i = 0; ok && i < STAGES; ++i) {
        ok = wait(empty + stage, phase ^ 1);
        if (++stage == STAGES) stage = 0, phase ^= 1;
      }
    }
    if (warp == 1 && lane == 0 && rank == 0) {
      // ---- products
      constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((A_MN ? 1u : 0u) << 15) |
                                 ((B_MN ? 1u : 0u) << 16) | (uint32_t{BN >> 3} << 17) | (uint32_t{kTileM * CG >> 4} << 24);
      constexpr uint32_t a_step = A_MN ? 16 * 128 : 32, b_step = B_MN ? 16 * 128 : 32;   // bytes of 16 k values
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      Tile t;
      for (int64_t i = first; ok && tile_of<false, kTileM * CG, BN>(i, mt, nt, s, &t); i += step) {
        const int b0 = t.split * per_split, b1 = min(blocks, b0 + per_split);
        if (!(ok = wait(sum_empty + acc, acc_phase ^ 1))) break;
        fence_after();
        bool fresh = true;   // nothing summed yet
        for (int kb = b0; kb < b1; ++kb) {
          if (!(ok = wait(full + stage, phase))) break;
          fence_after();
          const uint32_t a = shared_at(ring + stage * S::kStage), b = a + S::kA;
#pragma unroll
          for (int j = 0; j < kBlockK / 16; ++j)
            mma<CG>(tmem + acc * BN, operand(a + j * a_step, A_MN ? 64 * kBlockK * 2 : 16, 1024),
                    operand(b + j * b_step, B_MN ? 64 * kBlockK * 2 : 16, 1024), idesc, !fresh || j > 0);
          fresh = false;
          commit<CG>(empty + stage);
          if (++stage == STAGES) stage = 0, phase ^= 1;
          if (End::kChunk > 0 && kb + 1 < b1 && (kb + 1 - b0) % max(End::kChunk, 1) == 0) {
            commit<CG>(sum_full + acc);
            if (++acc == 2) acc = 0, acc_phase ^= 1;
            if (!(ok = wait(sum_empty + acc, acc_phase ^ 1))) break;
            fence_after();
            fresh = true;
          }
        }
        if (!ok) break;
        commit<CG>(sum_full + acc);
        if (++acc == 2) acc = 0, acc_phase ^= 1;
      }
    }
  } else {
    // ---- endings
    more_registers();
    const int group = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) * 32;
    int acc = 0;
    uint32_t acc_phase = 0;
    Part p;
    p.m = m;
    p.n = s.n;
    p.splits = s.splits;
    p.bad = false;
    p.ex = {exchange + (warp - 4) * kExchange, lane};
    for (int64_t i = first; tile_of<false, kTileM * CG, BN>(i, mt, nt, s, &p.tile); i += step) {
      const int b0 = p.tile.split * per_split, b1 = min(blocks, b0 + per_split);
      p.zero = b1 <= b0;
      p.row = p.tile.m0 + static_cast<int>(rank) * kTileM + static_cast<int>(lanes) + lane;
      p.cols = BN / 2;
      p.col = p.tile.n0 + group * p.cols;
      auto arrived = [&] {
        const bool ok = wait(sum_full + acc, acc_phase);
        p.bad = __any_sync(0xffffffffu, !ok) || p.bad;
        fence_after();
        p.tmem = tmem + (lanes << 16) + acc * BN + group * p.cols;
      };
      auto release = [&] {
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive_cluster(CG == 2 ? at_rank(shared_at(sum_empty + acc), 0) : shared_at(sum_empty + acc));
        if (++acc == 2) acc = 0, acc_phase ^= 1;
      };
      if constexpr (End::kChunk > 0) {
        float v[BN / 2];
        for (int kb = b0; kb == b0 || kb < b1; kb += End::kChunk) {
          arrived();
#pragma unroll
          for (int j = 0; j < BN / 2; j += 16) {
            float w[16];
            tmem_load16(p.tmem + j, w);
#pragma unroll
            for (int q = 0; q < 16; ++q) v[j + q] = kb == b0 ? w[q] : v[j + q] + w[q];
          }
          release();
        }
        if (p.zero || p.bad) {
#pragma unroll
          for (int j = 0; j < BN / 2; ++j) v[j] = p.bad ? __int_as_float(0x7fc00000) : 0.f;
        }
        End::whole(end, p, v);
      } else {
        arrived();
        End::part(end, p);
        release();
      }
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
  if constexpr (CG == 2) cluster_sync();
  if (warp == 2) tmem_free<CG>(tmem, kCols);
}

}  // namespace
}  // namespace tc
}  // namespace meo
