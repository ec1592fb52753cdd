// Host side shared by the files that launch tc_gemm.cuh's products: tensor
// maps, launches, per-kernel timing.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "adafactor_internal.h"
#include "tc_gemm.cuh"

namespace meo {
namespace tc {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled of libcuda (which is not linked).
inline EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return static_cast<EncodeTiled>(nullptr);
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Map of `batch` matrices of rows x cols 16-bit values, `ld` values a row, read in
// boxes of 64 columns (128 bytes, swizzled) by `box` rows.  p is 16-byte aligned
// and ld and stride_b are multiples of 8.
inline bool make_map(CUtensorMap* map, const void* p, bool bf16, int64_t rows, int64_t cols, int64_t ld, int64_t batch,
                     int64_t stride_b, int box) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(stride_b) * 2};
  const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(box), 1}, ones[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides,
            boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
constexpr int kBoxK = 128, kBoxMN = 64;   // rows of a box of a K-major and of an MN-major operand

inline cudaError_t sm_count(int* device, int* sms) {
  cudaError_t e = cudaGetDevice(device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device);
  return e;
}

// Per-kernel timing with events on the launching stream.
struct Profile {
  struct Record {
    int slot;
    cudaEvent_t start, stop;
  };
  std::mutex mu;
  std::atomic<bool> on{false};
  std::vector<Record> records;

  // launch() between two events if timing is on.
  template <class Launch>
  cudaError_t run(int slot, cudaStream_t s, Launch&& launch) {
    if (!on.load(std::memory_order_relaxed)) return launch();
    Record r{slot, nullptr, nullptr};
    cudaError_t e = cudaEventCreate(&r.start);
    if (e == cudaSuccess) e = cudaEventCreate(&r.stop);
    if (e == cudaSuccess) e = cudaEventRecord(r.start, s);
    if (e == cudaSuccess) e = launch();
    if (e == cudaSuccess) e = cudaEventRecord(r.stop, s);
    if (e != cudaSuccess) {
      if (r.start) cudaEventDestroy(r.start);
      if (r.stop) cudaEventDestroy(r.stop);
      return e;
    }
    std::lock_guard<std::mutex> lock(mu);
    records.push_back(r);
    return e;
  }
  cudaError_t read(double* ms, int64_t* launches, int32_t n) {
    std::lock_guard<std::mutex> lock(mu);
    cudaError_t first = cudaSuccess;
    for (Record& r : records) {
      float el = 0.f;
      cudaError_t e = cudaEventSynchronize(r.stop);
      if (e == cudaSuccess) e = cudaEventElapsedTime(&el, r.start, r.stop);
      if (first == cudaSuccess) first = e;
      if (r.slot < n) {
        if (ms) ms[r.slot] += el;
        if (launches) launches[r.slot] += 1;
      }
      cudaEventDestroy(r.start);
      cudaEventDestroy(r.stop);
    }
    records.clear();
    return first;
  }
};

// Launches a kernel that may begin while the one before it on the stream ends (it waits for it
// itself: previous_done).
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Launches a product over a persistent grid: as many CTAs as the device has SMs,
// or as there are tiles.
template <int CG, int BN, int STAGES, bool A_MN, bool B_MN, class End>
cudaError_t launch_product(const CUtensorMap& a, const CUtensorMap& b, const Shape& s, const typename End::Args& end,
                           cudaStream_t stream) {
  auto* const kernel = k_product<CG, BN, STAGES, A_MN, B_MN, End>;
  constexpr int kBytes = Shared<CG, BN, STAGES>::bytes;
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
  static std::atomic<unsigned long long> ready{0};   // devices whose limit has been raised
  int device = 0, sms = 0;
  cudaError_t e = sm_count(&device, &sms);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = device < 64 ? 1ull << device : 0;
  if (bit == 0 || (ready.load() & bit) == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  const int64_t mt = (s.m + kTileM * CG - 1) / (kTileM * CG), nt = (s.n + BN - 1) / BN;
  const int64_t tiles = mt * nt * std::max(1, s.splits);
  const int64_t grid = std::min<int64_t>(s.splits == 0 && tiles > 0 ? sms / CG : tiles, sms / CG) * CG;
  if (grid == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {CG, 1, 1};
  cfg.numAttrs = CG > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, b, s, end);
}

}  // namespace
}  // namespace tc
}  // namespace meo
