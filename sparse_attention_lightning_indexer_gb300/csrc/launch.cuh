// Launch of a kernel as the programmatic dependent of the previous kernel on its stream, with an
// optional cluster size. The kernel calls griddep_wait before its first global-memory access.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ds4idx.h"

namespace ds4w {
extern std::atomic<uint64_t>* launch_counter();
}

namespace ds4 {

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// SMs of the current device, asked once per device (0: an error).
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Lets `kernel` use `bytes` of dynamic shared memory; one call per device and kernel (`done`: a bit for
// each device on which it was made).
template <typename Kernel>
bool allow_shared(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

template <typename... Params, typename... Args>
int launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                     unsigned cluster, void* stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) {
    cudaGetLastError();  // the error is returned, not left behind for the next call
    return DS4IDX_ERR_LAUNCH;
  }
  ds4w::launch_counter()->fetch_add(1, std::memory_order_relaxed);
  return DS4IDX_OK;
}

}  // namespace ds4
