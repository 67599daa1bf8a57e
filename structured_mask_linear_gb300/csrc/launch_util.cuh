// Host helper: a kernel's dynamic shared memory limit, raised once per device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace ll {

// Each call site keeps its own flags (one per device), so that a launch costs no
// cudaFuncSetAttribute after the first.  Threads that race set the same value.
struct SmemLimit {
  std::atomic<bool> done[64];
  template <typename K>
  cudaError_t raise(K kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && keep) done[dev].store(true, std::memory_order_release);
    return e;
  }
};

}  // namespace ll
