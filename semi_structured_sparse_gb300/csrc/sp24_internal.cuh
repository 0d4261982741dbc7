// sp24_internal.cuh -- host-side helpers shared by the library's translation
// units: per-device state (SM count, architecture check, the device error
// word), tensor-map encoding through the driver entry point, and argument
// checks.  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>
#include <cstddef>
#include "../../include/sp24.h"

namespace sp24 {

// Device error word bits, set by kernels with atomicOr.
enum : unsigned int {
  DEVERR_TIMEOUT_PRODUCER = 1u,
  DEVERR_TIMEOUT_MMA = 2u,
  DEVERR_TIMEOUT_EPILOGUE = 4u,
  DEVERR_INDEX = 8u,  // an index read from device memory was out of range
};

struct DeviceInfo {
  int ordinal = -1;
  int sm_count = 0;
  int cc_major = 0, cc_minor = 0;
  size_t smem_optin = 0;
  unsigned int* err_word = nullptr;  // device address of the error word
};

// Current device's info (created on first use).  Returns SP24_ERR_CUDA or
// SP24_ERR_ARCH on failure.
sp24_status current_device(const DeviceInfo** out);

// 2D tensor map over a row-major [rows][cols] array of `elem_bytes`-sized
// elements with row stride `row_stride_bytes`; box {box_cols, box_rows};
// out-of-range elements read as zero.
// 3D: [depth][rows][cols] with row and depth strides in bytes (a batch of 2D views).
sp24_status make_tmap_3d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, uint64_t cols, uint64_t rows,
                         uint64_t depth, uint64_t row_stride_bytes, uint64_t depth_stride_bytes, uint32_t box_cols,
                         uint32_t box_rows, CUtensorMapSwizzle swizzle);
sp24_status make_tmap_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, uint64_t cols,
                         uint64_t rows, uint64_t row_stride_bytes, uint32_t box_cols, uint32_t box_rows,
                         CUtensorMapSwizzle swizzle);

// Any rank from 2 to 5, innermost dimension first; strides of dimensions 1 and up.
sp24_status make_tmap_nd(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int rank,
                         const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                         CUtensorMapSwizzle swizzle);

// Launches `kern` with programmatic stream serialisation: it may begin while
// the previous kernel in the stream finishes, and must call pdl_wait() (see
// sp24_ptx.cuh) before its first global-memory access.  `cluster`: CTAs per
// cluster, along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_clusters(void (*kern)(KArgs...), unsigned cluster, dim3 grid, dim3 block, size_t smem,
                                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              Args&&... args) {
  return launch_pdl_clusters(kern, 1, grid, block, smem, stream, static_cast<Args&&>(args)...);
}

// The same for a kernel that needs more shared memory than a kernel has by
// default: asks for it on each device's first launch (each time would cost a
// fifth of a microsecond), and again if a launch fails for its sake, as after a reset of
// the device's context.
template <auto Kern, typename... Args>
inline cudaError_t launch_pdl_clusters_smem(const DeviceInfo& dev, unsigned cluster, dim3 grid, dim3 block, size_t smem,
                                            cudaStream_t stream, const Args&... args) {
  static std::atomic<uint64_t> asked{0};  // a bit per device
  const uint64_t bit = uint64_t(1) << (dev.ordinal & 63);
  auto ask = [&] {
    return cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  };
  const bool before = asked.load(std::memory_order_relaxed) & bit;
  if (!before) {
    const cudaError_t r = ask();
    if (r != cudaSuccess) return r;
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaError_t r = launch_pdl_clusters(Kern, cluster, grid, block, smem, stream, args...);
  if (r == cudaErrorInvalidValue && before) {
    (void)cudaGetLastError();
    r = ask();
    if (r == cudaSuccess) r = launch_pdl_clusters(Kern, cluster, grid, block, smem, stream, args...);
  }
  return r;
}
template <auto Kern, typename... Args>
inline cudaError_t launch_pdl_smem(const DeviceInfo& dev, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                   const Args&... args) {
  return launch_pdl_clusters_smem<Kern>(dev, 1, grid, block, smem, stream, args...);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace sp24
