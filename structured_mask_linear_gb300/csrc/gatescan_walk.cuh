// What the kernels of the gated recurrence share: a lane's arithmetic, a CTA's walk over its tokens
// and how maps go round, and how a call is laid out.  (gatescan.cu, gatescan_bwd.cu)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "gatescan.cuh"
#include "launch_util.cuh"
#include "tc_common.cuh"

namespace ll {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
using ptx::add2;
using ptx::fma2;
using ptx::mul2;

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// ---- values ------------------------------------------------------------------------------
// A lane works on two neighbouring channels, whose products and sums are packed instructions.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = uint32_t;
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t put(float2 v) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  static __device__ __forceinline__ __nv_bfloat16 one(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Pair<float> {
  using type = float2;
  static __device__ __forceinline__ float2 get(float2 w) { return w; }
  static __device__ __forceinline__ float2 put(float2 v) { return v; }
  static __device__ __forceinline__ float one(float v) { return v; }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 rcp(float2 x) {
  float2 y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return y;
}
__device__ __forceinline__ float2 square_root(float2 x) {
  float2 y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return y;
}
// 1 / sqrt(x); x itself, as good as 0, below the smallest normal number, which the instruction takes for 0
// (and whose inverse would make infinities); NaN stays NaN.
__device__ __forceinline__ float inverse_root(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return x >= 1.17549435e-38f ? y : x;
}
// e^-x.  bf16: the exponent unit's own, 2^-22 relative and 2^-24 |x|, well below the inputs' step.
template <typename T>
__device__ __forceinline__ float2 exp_minus(float2 x) {
  x = mul2(x, both(-kLog2e));
  return make_float2(ex2(x.x), ex2(x.y));
}
template <>
__device__ __forceinline__ float2 exp_minus<float>(float2 x) {
  return make_float2(expf(-x.x), expf(-x.y));
}

// sigmoid = 1 / (1 + e) of e = e^-x: exact to a few steps however small, 0 for -inf and 1 for inf.
__device__ __forceinline__ float2 sigmoid_of(float2 e) { return rcp(add2(e, both(1.f))); }
// 1 - sigmoid as exactly: e times it, and the difference where e may be infinite.
__device__ __forceinline__ float2 rest_of(float2 e, float2 s) {
  const float2 p = mul2(e, s), d = fma2(s, both(-1.f), both(1.f));
  return make_float2(e.x < 1.f ? p.x : d.x, e.y < 1.f ? p.y : d.y);
}

// m = 1 - a = 1 - e^-z for z >= 0.  Below 0.7 it is z times a polynomial in z (Chebyshev fit of
// (1 - e^-z)/z, 4e-8 relative with these coefficients), since the difference would lose the small m that long memories live
// from.  a = 1 - m is as exact as fp32 holds it.
template <typename T>
__device__ __forceinline__ float2 loss_of(float2 z) {
  float2 p = both(-0.00102957711f);
  p = fma2(p, z, both(0.00806146674f));
  p = fma2(p, z, both(-0.0415687338f));
  p = fma2(p, z, both(0.166650444f));
  p = fma2(p, z, both(-0.499998987f));
  p = fma2(p, z, both(1.f));
  p = mul2(p, z);
  const float2 d = fma2(exp_minus<T>(z), both(-1.f), both(1.f));
  return make_float2(z.x < 0.7f ? p.x : d.x, z.y < 0.7f ? p.y : d.y);
}
__device__ __forceinline__ float2 kept_of(float2 m) { return fma2(m, both(-1.f), both(1.f)); }

enum { kMixRms = GS_RMS, kMixLerp = GS_LERP, kMixNone = GS_NONE };

__device__ __forceinline__ float2 not_below_0(float2 d) { return make_float2(d.x < 0.f ? 0.f : d.x, d.y < 0.f ? 0.f : d.y); }

// 1 - a^2
__device__ __forceinline__ float2 power_of(float2 m) { return mul2(m, fma2(m, both(-1.f), both(2.f))); }
// n(a) x
template <int M>
__device__ __forceinline__ float2 mixed(float2 m, float2 x) {
  if (M == kMixNone) return x;
  return mul2(M == kMixLerp ? m : square_root(power_of(m)), x);
}

// ---- shared memory -----------------------------------------------------------------------
// Maps (A, A', H, H') of a lane's two channels.
__device__ __forceinline__ float2 applied(const float4& g, float2 h) {
  return fma2(make_float2(g.x, g.y), h, make_float2(g.z, g.w));
}

// A CTA has kGsWarps warps, a warp G groups of 32 / G lanes, one after the other in time; a group has
// 64 / G channels.  Tokens of a group in a step, for N tensors of T: as many as leave room for 16
// warps on an SM (fewer backward in fp32); odd for several groups, so that they read different banks
// of shared memory.
template <typename T, int N, int G>
constexpr int kTokens = sizeof(T) == 2 && N <= 3 ? G == 1 ? 14 : 15 : G == 1 ? 8 : 7;
template <typename T, int N, int G>
constexpr int kChunk = kTokens<T, N, G> * kGsWarps * G;  // of a CTA

// Of everything that changes from step to step there are two, in turn: tokens on their way while
// others are worked on, and maps that a warp a step ahead, here or in another CTA, already writes.
template <typename T, int N, int G>
struct Shared {
  T in[2][N][kChunk<T, N, G>][kGsWidth / G];  // a step's tokens of each tensor, as they lie in memory
  uint64_t full[2];                // the tokens are there
  uint64_t told[2];                // the cluster's maps are there
  float4 group[2][kGsWarps * 32];  // maps of the groups, 32 / G of each
  float4 cta[];                    // [2][cluster][32 / G], of the CTAs
};
template <typename T, int N, int G>
constexpr int smem_bytes(int cluster) {
  return (int)sizeof(Shared<T, N, G>) + (cluster > 1 ? 2 * cluster * (32 / G) * 16 : 0);
}

// Bounded wait (2 s) for a phase.
__device__ __forceinline__ bool waited(uint64_t* bar, unsigned parity, unsigned* status) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (ptx::globaltimer_ns() - t0 > 2000000000ull) break;
  }
  atomicExch(status, kStatusTimeout);
  return false;
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A map into the shared memory of the cluster's CTA `rank`, at the place of p here; its arrival counts
// on that CTA's `bar`.  (A barrier of the cluster would wait for every store to global memory too.)
__device__ __forceinline__ void tell(unsigned rank, float4* p, float4 v, uint64_t* bar) {
  uint32_t at, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(ptx::smem_u32(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(b)
               : "memory");
}

// ---- a CTA's walk ------------------------------------------------------------------------
// Which sequence and channels a CTA has, its place among the CTAs that share them, its steps.  kAhead: how many
// steps ahead their tokens are asked for.
template <typename T, int N, int G, int kAhead>
struct Walk {
  static constexpr int L = kTokens<T, N, G>, kGroups = kGsWarps * G, kLanes = 32 / G, kWide = kGsWidth / G, kRows = L * kGroups;
  Shared<T, N, G>& s;
  const GsArgs& p;
  unsigned rank, size;
  int b, c0, c, len, steps;
  int asked;        // no step from here on is asked for: all of them but after a wait that ran out
  int lane, group;  // place in a group, and the group's in the CTA: in time order forward
  bool lost;

  __device__ __forceinline__ Walk(Shared<T, N, G>& s, const GsArgs& p) : s(s), p(p) {
    lane = threadIdx.x & (kLanes - 1);
    group = threadIdx.x / kLanes;
    size = (unsigned)p.cluster;
    rank = size > 1 ? cluster_rank() : 0u;
    const int id = (int)(blockIdx.x / size);
    b = id / p.tiles_d;
    c0 = (id - b * p.tiles_d) * kWide;
    c = c0 + 2 * lane;
    len = p.T;
    if (p.lengths) len = max(0, min(p.T, __ldg(p.lengths + b)));
    asked = steps = p.steps;
    lost = false;
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ptx::mbar_init(&s.full[i], 1);
        ptx::mbar_init(&s.told[i], 1);
      }
      ptx::fence_mbar_init();
    }
    __syncthreads();
    if (size > 1) cluster_sync();  // the others' shared memory and barriers are there from here on
  }
  // For a phase of step's; `later`: the fetch within the step is behind it.  After a wait that ran out nothing is
  // waited for, asked for or told any more.
  __device__ __forceinline__ void wait(uint64_t* bar, int step, bool later) {
    if (ptx::mbar_try_wait(bar, (unsigned)(step >> 1) & 1u) || lost) return;
    if (waited(bar, (unsigned)(step >> 1) & 1u, p.status)) return;
    lost = true;
    asked = min(steps, step + kAhead + later);
  }
  // After the last step: nobody leaves while others may still write to it, and all have read the state that
  // they began from, whose place the last one may take.  After a wait that ran out the tokens that were asked
  // for land first, and the others' maps (within another such wait for each stage, and 0.1 ms).
  template <bool kTma>
  __device__ __forceinline__ void leave() {
    if (kTma && lost && threadIdx.x == 0)
      for (int i = max(asked - 2, 0); i < asked; ++i) waited(&s.full[i & 1], (unsigned)(i >> 1) & 1u, p.status);
    if (size > 1) {
      cluster_sync();
      if (lost)
        for (const uint64_t t0 = ptx::globaltimer_ns(); ptx::globaltimer_ns() - t0 < 100000;) {
        }
    }
  }

  // The tokens from t0 (of tensor n from t0 - shift_n) of a step.  By TMA: one thread asks for them,
  // what lies outside the tensor comes as zeros.  Otherwise all threads copy them, between barriers.
  template <bool kTma>
  __device__ __forceinline__ void fetch(const GsMaps<N>& maps, const void* const* x, int stage, int t0, int shifted) {
    if (kTma) {
      if (threadIdx.x != 0) return;
      ptx::mbar_arrive_expect_tx(&s.full[stage], (uint32_t)sizeof(s.in[0]));
#pragma unroll
      for (int n = 0; n < N; ++n)
        ptx::tma_load_3d(&s.in[stage][n], &maps.map[n], &s.full[stage], c0, t0 - (n == shifted), b);
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const T* at = static_cast<const T*>(x[n]) + (size_t)b * p.T * p.D + c0;
        for (int i = threadIdx.x; i < kRows * kWide; i += kGsWarps * 32) {
          const int k = i / kWide, j = i % kWide, t = t0 - (n == shifted) + k;
          T v = Pair<T>::one(0.f);
          if (t >= 0 && t < p.T && c0 + j < p.D) v = at[(size_t)t * p.D + j];
          s.in[stage][n][k][j] = v;
        }
      }
    }
  }
  template <bool kTma>
  __device__ __forceinline__ void arrived(int step) {
    if (kTma) wait(&s.full[step & 1], step, false);
    else __syncthreads();
  }
  __device__ __forceinline__ float2 token(int stage, int n, int k) const {
    return Pair<T>::get(*reinterpret_cast<const typename Pair<T>::type*>(&s.in[stage][n][group * L + k][2 * lane]));
  }
  // Two channels of a row of fp32 values (states, decays), 0 where there are none.
  __device__ __forceinline__ float2 pair_of(const float* x, size_t row) const {
    float2 v = both(0.f);
    if (x && c < p.D) v.x = x[row * p.D + c];
    if (x && c + 1 < p.D) v.y = x[row * p.D + c + 1];
    return v;
  }
  __device__ __forceinline__ void put_pair(float* x, size_t row, float2 v) const {
    if (c < p.D) x[row * p.D + c] = v.x;
    if (c + 1 < p.D) x[row * p.D + c + 1] = v.y;
  }

  __device__ __forceinline__ float4 map_of(int buf, int g) const { return s.group[buf][g * kLanes + lane]; }

  // After every group has put its map into s.group[buf] and met the others (__syncthreads): what
  // enters the tokens of the `mine`th in time, all maps being there in time order; `carry`, what
  // enters the step, moves on to the next one's.  Maps are applied one after the other, in one order.
  __device__ __forceinline__ float2 enter(int step, int mine, float2& carry) {
    const int buf = step & 1;
    float2 in = carry;
    if (size > 1) {
      float4* told = s.cta + (buf * size) * kLanes;
      if (threadIdx.x == 0 && !lost) ptx::mbar_arrive_expect_tx(&s.told[buf], size * kLanes * 16);
      if ((unsigned)group < size && !lost) {  // each group tells some of the CTAs
        float2 A = both(1.f), H = both(0.f);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float4 m = map_of(buf, g);
          A = mul2(A, make_float2(m.x, m.y));
          H = applied(m, H);
        }
        for (unsigned r = group; r < size; r += kGroups)
          tell(r, told + rank * kLanes + lane, make_float4(A.x, A.y, H.x, H.y), &s.told[buf]);
      }
      wait(&s.told[buf], step, true);
      for (unsigned r = 0; r < size; ++r) {
        if (r == rank) in = carry;
        carry = applied(told[r * kLanes + lane], carry);
      }
      for (int g = 0; g < mine; ++g) in = applied(map_of(buf, g), in);
    } else {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (g == mine) in = carry;
        carry = applied(map_of(buf, g), carry);
      }
    }
    return in;
  }
};

// A lane's two values of one token (c < D); kPairs: D is even, and both go at once.
template <typename T, bool kPairs>
__device__ __forceinline__ void store(T* at, float2 v, int c, int D) {
  if (kPairs) {
    __stcs(reinterpret_cast<typename Pair<T>::type*>(at), Pair<T>::put(v));
  } else {
    at[0] = Pair<T>::one(v.x);
    if (c + 1 < D) at[1] = Pair<T>::one(v.y);
  }
}

// ---- launches ----------------------------------------------------------------------------
// A kernel's room on each device: clusters of each size that run at once, asked of the device once.
struct Room {
  std::atomic<int> clusters[64][kGsMaxCluster + 1];  // + 1, so that 0 means not asked yet
};
void launch_config(int size, unsigned grid, int smem, cudaStream_t st, cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr) {
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGsWarps * 32);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)size;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = size > 1 ? 1 : 0;
}
template <typename K>
cudaError_t clusters_at_once(K kernel, int size, int smem, int dev, Room& room, int& clusters) {
  return ask_once(dev < 64 ? &room.clusters[dev][size] : nullptr, clusters, [&](int& n) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess && size > 1) {
      cudaLaunchConfig_t cfg;
      cudaLaunchAttribute attr;
      launch_config(size, (unsigned)size, smem, nullptr, cfg, &attr);
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    } else if (e == cudaSuccess) {
      int per_sm = 0, sms = 0;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kGsWarps * 32, (size_t)smem);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      n = per_sm * sms;
    }
    if (e != cudaSuccess) cudaGetLastError();  // reported, or the layout goes without this size
    return e;
  });
}

// Map over (D, T, B) with a box of a unit's channels and a chunk of tokens.
bool make_gs_map(CUtensorMap* m, const void* base, const GsArgs& p, bool bf16, int chunk, int wide) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)p.D * (bf16 ? 2 : 4);
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.T, (cuuint64_t)p.B};
  const cuuint64_t strides[2] = {row, row * p.T};
  const cuuint32_t box[3] = {(cuuint32_t)wide, (cuuint32_t)chunk, 1}, es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Groups of a warp, and CTAs that share a unit: those with the shortest estimate.  Units beyond the
// clusters that run at once come in turns, the last one with fewer CTAs on an SM.  A step takes 1.5 us
// (forward in bf16; backward 1.4) for a CTA alone on its SM, and kMore of that more for every other
// one there (2.1, 2.7 and 3.5; 2.1, 2.6 and 3.2); the maps' way round adds a little for every CTA of
// the cluster.  More groups a warp are narrower units of longer steps: where there are few units, or
// few channels.  (Clusters of 9 to 16, where the device allows them, ran far fewer at once.)
constexpr double kMore = 0.42, kRound = 0.01, kGroup = 0.05;

struct Choice {
  int groups, size, steps, units;
  double t;         // 0: none yet
  cudaError_t why;  // an error of a size that could not be asked about
};
template <typename T, int N, int G, typename K>
void consider(Choice& best, K kernel, const GsArgs& p, int dev, Room& room) {
  const int chunks = (p.T + kChunk<T, N, G> - 1) / kChunk<T, N, G>, wide = kGsWidth / G;
  const int units = p.B * ((p.D + wide - 1) / wide);
  for (int size = 1; size <= kGsMaxCluster && (size == 1 || size <= chunks); ++size) {
    int n = 0;
    const cudaError_t e = clusters_at_once(kernel, size, smem_bytes<T, N, G>(size), dev, room, n);
    if (e != cudaSuccess) best.why = e;
    if (e != cudaSuccess || n < 1) continue;
    const int steps = (chunks + size - 1) / size;
    auto turn = [&](int clusters) {  // in steps of a CTA alone
      const int on_sm = (clusters * size + 151) / 152;
      return steps * (1.0 + kMore * (on_sm - 1)) * (1.0 + kRound * size) * (1.0 + kGroup * (G - 1));
    };
    const double t = units / n * turn(n) + (units % n ? turn(units % n) : 0.0);
    if (best.t == 0 || t < best.t) best = Choice{G, size, steps, units, t, best.why};
  }
}
template <typename T, int N, int G, typename K>
cudaError_t launch(K kernel, GsArgs& p, const Choice& c, const void* const* x, bool tma, cudaStream_t st) {
  GsMaps<N> maps{};
  if (tma)
    for (int n = 0; n < N; ++n)
      if (!make_gs_map(&maps.map[n], x[n], p, sizeof(T) == 2, kChunk<T, N, G>, kGsWidth / G)) return cudaErrorNotSupported;
  p.cluster = c.size;
  p.steps = c.steps;
  p.tiles_d = c.units / p.B;
  if (p.part && p.cluster * p.B == 1) p.part = p.ddecay;  // a single row of partials is the sum
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_config(c.size, (unsigned)((long long)c.units * c.size), smem_bytes<T, N, G>(c.size), st, cfg, &attr);
  return cudaLaunchKernelEx(&cfg, kernel, p, maps);
}

template <template <typename, bool, int, bool> class K, typename F>
cudaError_t choose(bool bf16, bool wide, int mix, bool gate, F f) {
#define LL_GS_MIX(T, W, M) return gate ? f(K<T, W, M, true>{}) : f(K<T, W, M, false>{})
#define LL_GS_W(T, W)                                        \
  switch (mix) {                                             \
    case kMixRms: LL_GS_MIX(T, W, kMixRms);                  \
    case kMixLerp: LL_GS_MIX(T, W, kMixLerp);                \
    default: LL_GS_MIX(T, W, kMixNone);                      \
  }
  if (bf16) {
    if (wide) LL_GS_W(__nv_bfloat16, true) else LL_GS_W(__nv_bfloat16, false)
  } else {
    if (wide) LL_GS_W(float, true) else LL_GS_W(float, false)
  }
#undef LL_GS_W
#undef LL_GS_MIX
}
// TMA wants rows that begin on 16 bytes.
inline bool whole_rows(int D, bool bf16) { return D % (bf16 ? 8 : 4) == 0; }

}  // namespace
}  // namespace ll
