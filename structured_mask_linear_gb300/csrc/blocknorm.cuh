// Shared declarations of the block norm (blocknorm.cu and its entry points).
#pragma once

#include "ll_internal.cuh"
#include "ptx.cuh"

namespace ll {

constexpr int kBnMaxD = 16384;
constexpr int kBnMaxGroups = 4096;  // groups per row (their sums sit in shared memory)

struct BnArgs {
  long long rows;
  int D, group, act;
  float eps, inv_D, inv_group;
  const void* x;     // forward: x (or NULL); backward: x' as stored (with dh)
  const void* y;
  const void* gate;
  const float* w_post;
  const float* scale;
  const float* w_pre;
  void* x_new;
  void* h;
  // backward
  const void* dx_new;
  const void* dh;
  void* dx;
  void* dy;
  void* dgate;
  float* dw_post;
  float* dscale;
  float* dw_pre;
  float* part;  // (CTAs, 3, D) partial sums: w_pre, w_post, scale
  unsigned* status;
};

constexpr int kBnMaxParts = 304;           // CTAs of the backward: at most two per SM
constexpr int kBnBwdSmem = 220 * 1024;     // its shared memory per SM

struct BnBwdPlan {
  bool fast;
  int ctas, threads, tpr, nv, smem;
};
BnBwdPlan bn_bwd_plan(const BnArgs& p, bool bf16);
cudaError_t launch_bn_fwd(const BnArgs& p, bool bf16, cudaStream_t st);
cudaError_t launch_bn_bwd(const BnArgs& p, bool bf16, cudaStream_t st);

// Bounded wait (2 s of %globaltimer) on an mbarrier.
__device__ __forceinline__ bool bn_wait(uint64_t* bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (ptx::globaltimer_ns() - t0 > 2000000000ull) return false;
  }
}

}  // namespace ll
