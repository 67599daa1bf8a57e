// Host helpers: a kernel's dynamic shared memory limit, raised once per device; what a device is asked
// once; launches that may start early.
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

// What `ask(answer)` finds, asked once and then kept in `slot` (NULL: not kept; 0: not asked yet, so the answer
// + 1).  Only an answer is kept: after an error the next call asks again.
template <typename F>
cudaError_t ask_once(std::atomic<int>* slot, int& answer, F ask) {
  if (slot)
    if (const int n = slot->load(std::memory_order_acquire)) {
      answer = n - 1;
      return cudaSuccess;
    }
  const cudaError_t e = ask(answer);
  if (e == cudaSuccess && slot) slot->store(answer + 1, std::memory_order_release);
  return e;
}

// A launch that may start before the kernel ahead of it on the stream has ended; the kernel waits
// for that one itself (griddepcontrol.wait) before it reads what it wrote.
template <typename... P, typename... A>
cudaError_t launch_ahead(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace ll
