// Host code that the cache operators' translation units share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "specverify_cache.h"

namespace sv {
namespace cache {

inline int device_index() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}
inline int sm_count() {
  static std::atomic<int> cached[64];
  const int dev = device_index();
  if (dev < 0) return 152;
  if (dev < 64 && cached[dev].load(std::memory_order_relaxed) > 0) return cached[dev].load(std::memory_order_relaxed);
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
  if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Opt in to `most` bytes of dynamic shared memory, the most that any launch of
// the kernel asks for, once per kernel (`set`: a static of the launch site) and
// device: threads that come here together set the same limit.
inline bool allow_smem(std::atomic<bool> (&set)[64], const void* kern, size_t most) {
  const int dev = device_index();
  if (dev < 0 || dev >= 64) return false;
  if (set[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  set[dev].store(true, std::memory_order_release);
  return true;
}

inline sv_status launched() { return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

template <typename K, typename P>
inline sv_status launch(K kern, dim3 grid, unsigned block, size_t smem, cudaStream_t stream, const P& p,
                 cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return launched();
}

}  // namespace cache
}  // namespace sv
