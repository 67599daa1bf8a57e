// Gated feed-forward block: m = act(x Wg^T) * (x Wu^T), and the gradients, on the tensor cores.
// Contracts are in include/loglinear.h.
//
// Bound by the tensor cores: 4 R D F operations forward, 8 backward.  A persistent pair of CTAs
// (cta_group::2) takes one tile of 256 x 256 at a time: each CTA loads 128 rows of A and 128 of B per
// 64 summed values (32 KB a stage, six stages; a warp for each operand: by one alone a stage took 0.23 us,
// which narrow tiles wait for, now 0.14), the first one's issuing thread feeds both SMs' tensor
// cores, and each SM's tensor memory holds 128 rows of two accumulators, so that eight warps write
// one tile out while the next is summed.  Forward, the 256 columns are 128 of Wg and the same 128 of
// Wu: a thread has a gate and its up value in one row, and only their product goes out.  With few
// rows the tiles are narrower, so that every pair has one (ffgate_api.cu).
//
// 8192 x 4096 x 11008 850 to 876 us under the power cap (1.69 to 1.74 PFLOP/s; a library product sustains 1.73) and
// 725 in a burst; gradients of 8192 x 2048 x 5632 490 to 523 us, of which the products of dm with the activation's
// derivative, a pass over memory of its own, are some 70.
//
// fp32 runs through the same kernel.  Forward every row of x and of the weights is summed over, so it may be
// scaled: two fp16 parts (hi + lo, 2^-23 of a value or 2^-39 of the row's largest) make three products, the
// one left out below 2^-22.  Backward the gradients of gate and up are summed along both their sides (x and the
// weights along one), so one scale a row would not do: all are three bf16 parts (24 bits, over all of fp32's
// range), six products, what is left out below 2^-24.  Forward with three parts took 60 us of 1003 x 1024 x 2816, with two 40 (fp32 operands' split by
// itself 9: 4 bytes read and 4 written a value).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "ffgate.cuh"
#include "ffgate_act.cuh"
#include "launch_util.cuh"
#include "tc_common.cuh"

namespace ll {
namespace {

constexpr int kGroup = 2;                 // CTAs of a tile
constexpr int kRow = 64 * 2;              // bytes of a row of a stage
constexpr int kEpiWarps = 8;
constexpr int kFfThreads = 128 + kEpiWarps * 32;
constexpr int kOutBytes = 32 * 128;       // a warp's rows on their way out
constexpr int kFfSmem = kFfStageRoom + kEpiWarps * kOutBytes + 1024 + 256;
constexpr int kBand = 8;                  // tiles of rows that run together down the columns

struct Bars {
  uint64_t full[kFfMaxStages], empty[kFfMaxStages], acc_full[2], acc_empty[2];
  uint32_t tmem;
};

// ---- the pair of CTAs ----------------------------------------------------------------------
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of the first CTA's counterpart of a place in shared memory.
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(ptx::smem_u32(p)));
  return a;
}
__device__ __forceinline__ void tma_load_pair(void* dst, const void* tmap, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(ptx::smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on both CTAs' barriers once the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          ptx::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void arrive_in_first(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_first(bar)) : "memory");
}
// Bounded (2 s); a role whose wait ran out gives up, the others follow.
__device__ __forceinline__ bool ff_wait(uint64_t* bar, uint32_t parity, unsigned* status) {
#pragma unroll 1
  for (int i = 0; i < 1024; ++i)
    if (__builtin_expect(ptx::mbar_try_wait(bar, parity), 1)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (ptx::globaltimer_ns() - t0 < kWaitNs) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
  }
  atomicExch(status, kStatusTimeout);
  return false;
}

// ---- tiles -----------------------------------------------------------------------------------
struct Tile {
  int prob, m, n, split;
  int from, to;  // its blocks of 64 summed values, of all pairs
};
// Tiles of a problem in bands of kBand row tiles, rows first: what runs at a time shares its operands
// in L2.
__device__ __forceinline__ Tile tile_at(const FfArgs& p, int t) {
  Tile x;
  x.prob = 0;
  while (x.prob + 1 < p.probs && t >= p.prob[x.prob + 1].tile0) ++x.prob;
  const FfProb& r = p.prob[x.prob];
  t -= r.tile0;
  x.split = 0;
  if (r.splits > 1) {
    x.split = t % r.splits;
    t /= r.splits;
  }
  x.from = x.split * r.share;
  x.to = min(x.from + r.share, r.pairs * r.kblocks);
  const int band = t / (kBand * r.tiles_n), m0 = band * kBand, rows = min(kBand, r.tiles_m - m0);
  t -= band * kBand * r.tiles_n;
  x.n = t / rows;
  x.m = m0 + t - x.n * rows;
  return x;
}
// Operands as the tensor cores take them, and their products, the smallest first: part `part(i) & 3` of A
// and part(i) >> 2 of B.
struct Whole {  // bf16
  using T = __nv_bfloat16;
  static constexpr int kParts = 1, kProducts = 1;
  static constexpr bool kHalf = false, kFit = false;
  static constexpr __device__ int part(int) { return 0; }
};
struct Few : Whole {  // of no more rows than one CTA takes: stages of as many as there are, and more of them
  static constexpr bool kFit = true;
};
struct Thirds {  // fp32 as three of bf16
  using T = float;
  static constexpr int kParts = 3, kProducts = 6;
  static constexpr bool kHalf = false, kFit = false;
  static constexpr __device__ int part(int i) { return (0x041582 >> (4 * i)) & 15; }
};
struct Halves {  // fp32 as two of fp16, rows scaled
  using T = float;
  static constexpr int kParts = 2, kProducts = 3;
  static constexpr bool kHalf = true, kFit = false;
  static constexpr __device__ int part(int i) { return (0x041 >> (4 * i)) & 15; }
};
// The tensor cores cut their sums off where fp32 would round (a sum over 16384 products of fp32 values
// loses 2e-5 of itself).  fp32 tiles are therefore summed in runs, which the warps that write out add up in
// registers: of one block of 64 values, whose last four instructions alone are of full size, or in two parts
// of two blocks where the sum is long.  So they stay at 1.6e-7 and 4.3e-7 of a row's norm (an fp32 sum that
// rounds every addition: 2.6e-7 over 128 values, 5.0e-7 over 512, 6.2e-7 over 8192), and every further
// block in a run adds 2.3e-7.  The adding up is what bounds the short runs: 1003 x 1024 x 2816 51.9 us with
// runs of one block, 41.7 with two, 32.7 with a whole sum.  bf16 results do not see any of it, and take a
// whole tile as one run.
template <typename O>
__device__ __forceinline__ int run_of(const FfProb& r, int left) {
  return O::kParts == 1 ? left : min(left, O::kHalf && r.kblocks > 8 ? 2 : 1);
}

// ---- values ----------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---- writing out -----------------------------------------------------------------------------
__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tmap), "r"(c0), "r"(c1),
               "r"(ptx::smem_u32(src))
               : "memory");
}
// 32 columns of the warp's 32 rows, of which each lane has one, into the warp's place (rows of 128
// bytes, swizzled as the store's map says); `at`: which 32 columns of a row of bf16.
template <typename T>
__device__ __forceinline__ void stage(uint8_t* out, const float* v, int lane, int at) {
  uint8_t* row = out + lane * 128;
  if (sizeof(T) == 2) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(row + (((4 * at + c) ^ (lane & 7)) << 4)) =
          make_uint4(pack_bf2(v[8 * c], v[8 * c + 1]), pack_bf2(v[8 * c + 2], v[8 * c + 3]),
                     pack_bf2(v[8 * c + 4], v[8 * c + 5]), pack_bf2(v[8 * c + 6], v[8 * c + 7]));
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<float4*>(row + ((c ^ (lane & 7)) << 4)) =
          make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  }
}
template <typename T>
__device__ __forceinline__ void put_eight(void* to, long long at, const float* v) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(static_cast<T*>(to) + at) =
        make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
  } else {
    float4* out = reinterpret_cast<float4*>(static_cast<T*>(to) + at);
    out[0] = make_float4(v[0], v[1], v[2], v[3]);
    out[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
// Columns col.. of the 32 rows from `row` on their way, once the place is full (the store clips what
// lies outside; a box all outside is left out).
__device__ __forceinline__ void send(const void* map, const uint8_t* out, const FfProb& r, int col, int row, int lane) {
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0 && col < r.cols && row < r.rows) {
    tma_store_2d(map, out, col, row);
    ptx::bulk_commit_group();
  }
}
__device__ __forceinline__ void place_free(int lane) {
  if (lane == 0) ptx::bulk_wait_read_all();
  __syncwarp();
}

template <typename O>
__global__ void __cluster_dims__(kGroup, 1, 1) __launch_bounds__(kFfThreads, 1)
    ff_products_kernel(const __grid_constant__ FfArgs p, const __grid_constant__ FfMaps maps) {
  using T = typename O::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_out = smem + kFfStageRoom;
  Bars& bars = *reinterpret_cast<Bars*>(s_out + kEpiWarps * kOutBytes);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const unsigned rank = cluster_rank();
  const int first = blockIdx.x / kGroup, stride = gridDim.x / kGroup;
  // a stage: the parts of A, then those of B
  const int a_bytes = O::kFit ? p.a_box * kRow : 128 * kRow, b_bytes = O::kFit ? p.b_box * kRow : 128 * kRow;
  const int stage_bytes = O::kParts * (a_bytes + b_bytes), stages = O::kFit ? p.stages : kFfStageRoom / stage_bytes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFfMaxStages; ++i) {
      ptx::mbar_init(&bars.full[i], 1);
      ptx::mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars.acc_full[i], 1);
      ptx::mbar_init(&bars.acc_empty[i], kGroup * kEpiWarps);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(ptx::smem_u32(&bars.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem;

  ptx::griddep_launch_dependents();

  if (warp == 0 || warp == 3) {
    // ---- loads: this CTA's 128 rows of A by warp 0, of B by warp 3 -----------------------------
    if (ptx::elect_one()) {
      const bool first_operand = warp == 0;
      uint8_t* const place = smem + (first_operand ? 0 : O::kParts * a_bytes);
      const int part_bytes = first_operand ? a_bytes : b_bytes;
      const uint32_t bar0 = in_first(bars.full);
      uint32_t s = 0, phase = 1;  // the wait for an empty stage passes in the first turn
      bool ok = true, turned = false;
      ptx::griddep_wait();  // operands may come from the kernel ahead; all else here waits for them
      for (int t = first; ok && t < p.tiles; t += stride) {
        const Tile x = tile_at(p, t);
        const FfProb& r = p.prob[x.prob];
        const int gated = r.gated, width = r.width, kblocks = r.kblocks;
        const int at = first_operand ? x.m * 256 + (int)rank * 128 : x.n * width + (gated ? 0 : (int)rank * 128);
        const bool mn = first_operand ? r.a_mn : r.b_mn;
        // with few rows the second CTA has none; whatever lies in their place goes into rows that nobody reads
        const bool any = !O::kFit || !first_operand || rank == 0;
        const uint32_t bytes =
            O::kParts * ((O::kFit ? 1 : kGroup) * a_bytes + kGroup * (O::kFit ? b_bytes : gated ? width * kRow : 128 * kRow));
        const int second = first_operand ? r.a[1] : r.b[1];
        const CUtensorMap* map = &maps.m[first_operand ? r.a[0] : r.b[gated ? rank : 0]];
        int k = x.from;
        if (k >= kblocks) {
          k -= kblocks;
          map = &maps.m[second];
        }
        for (int left = x.to - x.from; left > 0; --left) {
          if (!ff_wait(&bars.empty[s], phase, p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = bar0 + 8 * s;
          if (first_operand && rank == 0) ptx::mbar_arrive_expect_tx(&bars.full[s], bytes);
          uint8_t* to = place + s * stage_bytes;
#pragma unroll
          for (int part = 0; part < O::kParts; ++part, to += part_bytes) {
            if (!any) break;
            tma_load_pair(to, map, bar, mn ? at : 64 * k, mn ? 64 * k : at, part);
            if (mn) tma_load_pair(to + 64 * kRow, map, bar, at + 64, 64 * k, part);
          }
          if (++s == stages) {
            s = 0;
            phase ^= 1;
            turned = true;
          }
          if (++k == kblocks) {
            k = 0;
            map = &maps.m[second];
          }
        }
      }
      // What was asked for lands before the CTAs end, whatever their other roles gave up (bounded, 2 s in all; each
      // stage's bytes count in the first CTA, for both): the stages before s in this turn, the others in the one
      // before it.
      if (first_operand && rank == 0) {
        bool landed = true;
        for (uint32_t i = 0; landed && i < (uint32_t)stages; ++i)
          if (i < s || turned) landed = ff_wait(&bars.full[i], i < s ? phase ^ 1 : phase, p.status);
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---- products, for both CTAs ------------------------------------------------------------
    if (ptx::elect_one()) {
      uint32_t s = 0, phase = 0, n = 0;
      bool ok = true;
      const uint64_t kmaj = ptx::smem_desc_sw128(ptx::smem_u32(smem), 16, 1024);
      const uint64_t mnmaj = ptx::smem_desc_sw128(ptx::smem_u32(smem), 64 * kRow, 1024);
      for (int t = first; ok && t < p.tiles; t += stride) {
        const Tile x = tile_at(p, t);
        const FfProb& r = p.prob[x.prob];
        const int columns = r.gated ? 2 * r.width : 256;
        const uint32_t idesc =
            O::kHalf ? ptx::idesc_f16_f32(256, columns, r.a_mn, r.b_mn) : ptx::idesc_bf16_f32(256, columns, r.a_mn, r.b_mn);
        const uint64_t da = r.a_mn ? mnmaj : kmaj, db = (r.b_mn ? mnmaj : kmaj) + (O::kParts * a_bytes >> 4);
        const uint32_t sa = r.a_mn ? 128 : 2, sb = r.b_mn ? 128 : 2;  // 16 summed values, in 16 bytes
        for (int k0 = x.from, run; ok && k0 < x.to; k0 += run, ++n) {
          run = run_of<O>(r, x.to - k0);
          const uint32_t acc = n & 1, d = tmem + 256 * acc;
          if (n >= 2) ok = ff_wait(&bars.acc_empty[acc], ((n >> 1) - 1) & 1, p.status);
          if (!ok) break;
          ptx::tc_fence_after();
          for (int k = 0; k < run; ++k) {
            if (!ff_wait(&bars.full[s], phase, p.status)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int i = 0; i < O::kProducts; ++i) {
              const uint32_t at = s * (stage_bytes >> 4);
              const uint64_t pa = da + at + (O::part(i) & 3) * (a_bytes >> 4);
              const uint64_t pb = db + at + (O::part(i) >> 2) * (b_bytes >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) umma_pair(d, pa + kk * sa, pb + kk * sb, idesc, k + i + kk > 0);
            }
            commit_pair(&bars.empty[s]);
            if (++s == stages) {
              s = 0;
              phase ^= 1;
            }
          }
          if (ok) commit_pair(&bars.acc_full[acc]);
        }
      }
    }
  } else if (warp >= 4) {
    // ---- a tile's way out ---------------------------------------------------------------------
    const int e = warp - 4, quad = warp & 3, half = e >> 2;
    uint8_t* out = s_out + e * kOutBytes;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    constexpr int kPer = sizeof(T) == 2 ? 2 : 1;  // runs of 32 columns in a store
    uint32_t n = 0;
    bool ok = true;
    if (O::kHalf) ptx::griddep_wait();  // the scales
    // waits for a run's sums, and hands their place back
    auto arrive = [&] {
      ok = __all_sync(0xffffffffu, ff_wait(&bars.acc_full[n & 1], (n >> 1) & 1, p.status));
      ptx::tc_fence_after();
      return tmem + 256 * (n & 1) + lanes;
    };
    auto release = [&] {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_in_first(&bars.acc_empty[n & 1]);
      ++n;
    };
    // 32 columns `run` of a tile's output on their way
    auto put = [&](const FfProb& r, int map, const float* v, int run, int col, int row) {
      const int c = run % kPer;
      if (c == 0) place_free(lane);
      stage<T>(out, v, lane, c);
      if (c + 1 == kPer) send(&maps.m[map], out, r, col + 32 * (run + 1 - kPer), row, lane);
    };
    // 16 columns of a split tile's sums
    auto put_part = [&](const FfProb& r, const Tile& x, const float* v, int second_half, int col, int row) {
      if (row + lane >= r.rows) return;
      const long long plane = r.gated ? 2 * x.split + second_half : x.split;
      const long long at = (plane * r.rows + row + lane) * r.cols + col;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (col + 8 * h < r.cols) put_eight<float>(r.part, at + 8 * h, v + 8 * h);  // a multiple of 8
    };
    // 16 columns of a narrow tile straight out: there are few rows of them
    auto put_narrow = [&](const FfProb& r, const float* g, const float* u, int col, int row) {
      if (row + lane >= r.rows) return;
      const long long at = (long long)(row + lane) * r.cols + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (col + 8 * h >= r.cols) break;  // a multiple of 8
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = ff_act<T>(g[8 * h + j], p.act) * u[8 * h + j];
        put_eight<T>(p.m, at + 8 * h, m);
        if (p.gate) {
          put_eight<T>(p.gate, at + 8 * h, g + 8 * h);
          put_eight<T>(p.up, at + 8 * h, u + 8 * h);
        }
      }
    };
    for (int t = first; t < p.tiles; t += stride) {
      const Tile x = tile_at(p, t);
      const FfProb& r = p.prob[x.prob];
      const int row = x.m * 256 + (int)rank * 128 + quad * 32;
      // a thread's columns: up to 64 of the gate's and of up's, in 16s, or 128 in a row
      const int per = r.gated ? (r.width / 16 + 1) / 2 : 8, sixteens = r.gated && half ? r.width / 16 - per : per;
      const int from = half * 16 * per, second = r.gated ? r.width : 64;
      const int col = x.n * r.width + from;
      const bool narrow = r.gated && r.width < 128;
      if constexpr (sizeof(T) == 4) {
        // gated tiles are those of halves.  The scales of the columns lie in the warp's place until the tile goes out
        const float2* const scales = reinterpret_cast<const float2*>(out);
        float2 scale;
        if constexpr (O::kHalf) {
          place_free(lane);
          float2* const to = reinterpret_cast<float2*>(out);
#pragma unroll
          for (int c = lane; c < 64; c += 32) {
            to[c] = p.scale_gate[min(col + c, r.cols - 1)];
            to[64 + c] = p.scale_up[min(col + c, r.cols - 1)];
          }
          scale = p.scale_x[min(row + lane, r.rows - 1)];
          __syncwarp();
        }
        float v[2][64];
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i / 64][i % 64] = 0.f;
        for (int left = x.to - x.from; left > 0; left -= run_of<O>(r, left)) {
          const uint32_t d = arrive();
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float y[2][16];
            if (c >= sixteens) break;
            ptx::tmem_ld16(d + from + 16 * c, y[0]);
            ptx::tmem_ld16(d + from + second + 16 * c, y[1]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j / 16][16 * c + j % 16] += y[j / 16][j % 16];
          }
          release();
        }
        if (!ok) break;
        if constexpr (O::kHalf) {  // the rows' scales back
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            if (c / 16 >= sixteens) continue;
            const float2 g = scales[c], u = scales[64 + c];
            v[0][c] = v[0][c] * (scale.x * g.x) * (scale.y * g.y);
            v[1][c] = v[1][c] * (scale.x * u.x) * (scale.y * u.y);
          }
        }
        if (r.splits > 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i % 4 < sixteens) put_part(r, x, v[i / 4] + 16 * (i % 4), i / 4, col + (O::kHalf ? 0 : 64 * (i / 4)) + 16 * (i % 4), row);
          continue;
        }
        if (O::kHalf && narrow) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < sixteens) put_narrow(r, v[0] + 16 * c, v[1] + 16 * c, col + 16 * c, row);
          continue;
        }
        if (O::kHalf && r.out_gate >= 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) put(r, r.out_gate, v[0] + 32 * c, c, col, row);
#pragma unroll
          for (int c = 0; c < 2; ++c) put(r, r.out_up, v[1] + 32 * c, c, col, row);
        }
        if (O::kHalf) {
          ff_gated<T, 32>(v[0], v[1], p.act);
          ff_gated<T, 32>(v[0] + 32, v[1] + 32, p.act);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) put(r, r.out, v[0] + 32 * c, c, col, row);
        if (!O::kHalf) {
#pragma unroll
          for (int c = 0; c < 2; ++c) put(r, r.out, v[1] + 32 * c, 2 + c, col, row);
        }
      } else {
        const uint32_t d = arrive();
        if (!ok) break;
        if (r.splits > 1) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            if (i % 4 >= sixteens) continue;
            float v[16];
            ptx::tmem_ld16(d + from + (i / 4) * second + 16 * (i % 4), v);
            ptx::tmem_ld_wait();
            put_part(r, x, v, i / 4, col + (r.gated ? 0 : 64 * (i / 4)) + 16 * (i % 4), row);
          }
          release();
        } else if (narrow) {
#pragma unroll 1
          for (int c = 0; c < sixteens; ++c) {
            float g[16], u[16];
            ptx::tmem_ld16(d + from + 16 * c, g);
            ptx::tmem_ld16(d + second + from + 16 * c, u);
            ptx::tmem_ld_wait();
            put_narrow(r, g, u, col + 16 * c, row);
          }
          release();
        } else if (r.gated) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float g[32], u[32];
            ptx::tmem_ld32(d + from + 32 * c, g);
            ptx::tmem_ld32(d + 128 + from + 32 * c, u);
            ptx::tmem_ld_wait();
            if (c == 1 && r.out_gate < 0) release();
            ff_gated<T, 32>(g, u, p.act);
            put(r, r.out, g, c, col, row);
          }
          if (r.out_gate >= 0) {  // what the backward needs
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              float v[32];
              ptx::tmem_ld32(d + (i >> 1) * 128 + from + 32 * (i & 1), v);
              ptx::tmem_ld_wait();
              if (i == 3) release();
              put(r, i < 2 ? r.out_gate : r.out_up, v, i & 1, col, row);
            }
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            ptx::tmem_ld32(d + from + 32 * c, v);
            ptx::tmem_ld_wait();
            if (c == 3) release();
            put(r, r.out, v, c, col, row);
          }
        }
      }
    }
    if (lane == 0) ptx::bulk_wait_read_all();
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();  // both have read their tensor memory, and nothing arrives any more
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ---- operands --------------------------------------------------------------------------------
__device__ __forceinline__ void parts_of(float v, __nv_bfloat16& hi, __nv_bfloat16& mid, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float r = v - __bfloat162float(hi);
  mid = __float2bfloat16_rn(r);
  lo = __float2bfloat16_rn(r - __bfloat162float(mid));
}
// V values (4 or 8) from `at` on of the three parts, n apart.
template <int V>
__device__ __forceinline__ void put_parts(__nv_bfloat16* to, long long at, long long n, const float* v) {
  __align__(16) __nv_bfloat16 x[3][V];
#pragma unroll
  for (int j = 0; j < V; ++j) parts_of(v[j], x[0][j], x[1][j], x[2][j]);
  using W = typename std::conditional<V == 8, uint4, uint2>::type;
#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<W*>(to + i * n + at) = *reinterpret_cast<const W*>(x[i]);
}
// Counts are multiples of 8 (rows are).
__global__ void __launch_bounds__(256) ff_split_kernel(const __grid_constant__ FfSplit s) {
  const int i = blockIdx.y;
  const long long n = s.n[i];
  ptx::griddep_launch_dependents();
  for (long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; at < n; at += (long long)gridDim.x * 2048) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(s.from[i] + at));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(s.from[i] + at + 4));
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    put_parts<8>(static_cast<__nv_bfloat16*>(s.to[i]), at, n, v);
  }
}
// Rows as two fp16 parts of values scaled by a power of two that brings the largest to 2^14 .. 2^15.  What
// is lost is half a step of the low part: 2^-23 of a value, and at least half of fp16's smallest step, 2^-25,
// which is 2^-39 of a largest value of 2^14.  (Three bf16 parts lose 2^-24 of any value; with them 1003 x 1024 x
// 2816 took 60 us instead of 41.)  The scale
// goes back as two factors of half its exponent each, so that no product of factors leaves fp32's range.
// W warps a row, 16 values a lane: read once up to 4096 values, or twice, the second time from the caches.
template <int W, bool kOnce>
__global__ void __launch_bounds__(256) ff_halves_kernel(const __grid_constant__ FfHalves s) {
  __shared__ unsigned most[8];
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, at = threadIdx.x % (32 * W) * 4;
  long long row = (long long)blockIdx.x * (8 / W) + warp / W;
  int i = 0;
  while (i < 2 && row >= s.rows[i]) row -= s.rows[i++];
  const bool there = row < s.rows[i];
  const float* from = s.from[i] + row * s.D;
  float4 x[4];
  // the rows' bits as numbers: what is not negative is in order
  unsigned bits = 0;
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = base + at + 128 * W * k;
      x[k] = there && d < s.D ? *reinterpret_cast<const float4*>(from + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  for (int base = 0; base < (kOnce ? 1 : s.D); base += 512 * W) {
    load(base);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      bits = max(bits, __float_as_uint(fmaxf(fmaxf(fabsf(x[k].x), fabsf(x[k].y)), fmaxf(fabsf(x[k].z), fabsf(x[k].w)))));
  }
  bits = __reduce_max_sync(0xffffffffu, bits);
  if (W > 1) {
    if ((threadIdx.x & 31) == 0) most[warp] = bits;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) bits = max(bits, most[warp / W * W + k]);
  }
  if (!there) return;
  // rows of zeros, and with infinities (NaN whatever the scale): any scale; below 2^-112 a smaller one
  const int e = bits == 0 ? 0 : min(14 + 127 - (int)(bits >> 23), 126), h = e >> 1;
  auto power = [](int k) { return __int_as_float((127 + k) << 23); };
  const float f0 = power(h), f1 = power(e - h);
  if (at == 0) s.scale[i][row] = make_float2(power(-h), power(h - e));
  __half* to = static_cast<__half*>(s.to[i]) + row * s.D;
  const long long n = s.rows[i] * s.D;
  for (int base = 0; base < (kOnce ? 1 : s.D); base += 512 * W) {
    if (!kOnce) load(base);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = base + at + 128 * W * k;
      if (d >= s.D) break;
      const float v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      __align__(8) __half hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y = v[j] * f0 * f1;
        hi[j] = __float2half_rn(y);
        lo[j] = __float2half_rn(y - __half2float(hi[j]));
      }
      *reinterpret_cast<uint2*>(to + d) = *reinterpret_cast<const uint2*>(hi);
      *reinterpret_cast<uint2*>(to + n + d) = *reinterpret_cast<const uint2*>(lo);
    }
  }
}
// The gradients of gate and up, as the products take them: in bf16 rounded to one part, which makes the weights'
// and x's gradients off by 2.3e-3 of their norm instead of 1.7e-3: two independent roundings instead of one.  A second
// part would be twice the products, another 437 us at 8192 x 2048 x 5632.  (bf16 in 32 registers, so that all 16 CTAs
// of an SM run in two full turns: in 40 the SMs were done apart, and the pairs of CTAs of the products behind them
// began apart, 504 -> 546 us for 8831 x 552 x 10768.)
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 8 : 5) ff_act_bwd_kernel(const T* dm, const T* gate, const T* up, __nv_bfloat16* dgate,
                                                         __nv_bfloat16* dup, long long n, int act) {
  constexpr int V = sizeof(T) == 2 ? 8 : 4;
  ptx::griddep_launch_dependents();
  for (long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * V; at < n; at += (long long)gridDim.x * 256 * V) {
    const uint4 rd = __ldcs(reinterpret_cast<const uint4*>(dm + at)), rg = __ldcs(reinterpret_cast<const uint4*>(gate + at)),
                ru = __ldcs(reinterpret_cast<const uint4*>(up + at));
    const uint32_t d[4] = {rd.x, rd.y, rd.z, rd.w}, g[4] = {rg.x, rg.y, rg.z, rg.w}, u[4] = {ru.x, ru.y, ru.z, ru.w};
    float a[V], b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      auto value = [&](const uint32_t* w) {
        if (sizeof(T) == 4) return __uint_as_float(w[j % 4]);
        return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
      };
      const float2 f = ff_act_and_slope<T>(value(g), act);
      a[j] = value(d) * value(u) * f.y;
      b[j] = value(d) * f.x;
    }
    if (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(dgate + at) = make_uint4(pack_bf2(a[0], a[1]), pack_bf2(a[2], a[3]), pack_bf2(a[4 % V], a[5 % V]),
                                                         pack_bf2(a[6 % V], a[7 % V]));
      *reinterpret_cast<uint4*>(dup + at) = make_uint4(pack_bf2(b[0], b[1]), pack_bf2(b[2], b[3]), pack_bf2(b[4 % V], b[5 % V]),
                                                       pack_bf2(b[6 % V], b[7 % V]));
    } else {
      put_parts<4>(dgate, at, n, a);
      put_parts<4>(dup, at, n, b);
    }
  }
}
// The sums of split tiles in order, and what comes after them.  Four values a thread; counts are
// multiples of 8.
template <typename T>
__global__ void __launch_bounds__(256) ff_join_kernel(const __grid_constant__ FfJoin j) {
  const auto& r = j.prob[blockIdx.y];
  const long long step = j.gated ? 2 * r.n : r.n;
  ptx::griddep_wait();
  for (long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * 4; at < r.n; at += (long long)gridDim.x * 1024) {
    float v[2][4] = {};
    for (int s = 0; s < r.splits; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h && !j.gated) break;
        const float4 x = __ldcs(reinterpret_cast<const float4*>(r.part + s * step + h * r.n + at));
        v[h][0] += x.x, v[h][1] += x.y, v[h][2] += x.z, v[h][3] += x.w;
      }
    auto put = [&](void* to, const float* x) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(static_cast<T*>(to) + at) = make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
      else
        *reinterpret_cast<float4*>(static_cast<T*>(to) + at) = make_float4(x[0], x[1], x[2], x[3]);
    };
    if (j.gated) {
      if (j.gate) {
        put(j.gate, v[0]);
        put(j.up, v[1]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[0][i] = ff_act<T>(v[0][i], j.act) * v[1][i];
    }
    put(r.out, v[0]);
  }
}
unsigned grid_for(long long n, int per) {
  const long long ctas = (n + per - 1) / per;
  return (unsigned)(ctas < 152 * 16 ? ctas : 152 * 16);
}

}  // namespace

bool ff_operand_map(CUtensorMap* m, const void* base, long long inner, long long outer, int parts, bool mn_major, int rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)parts};
  const cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)inner * outer * 2};
  const cuuint32_t box[3] = {64, mn_major ? 64u : (cuuint32_t)rows, 1}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool ff_output_map(CUtensorMap* m, const void* base, long long cols, long long rows, bool bf16) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {bf16 ? 64u : 32u, 32}, es[2] = {1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename O>
static cudaError_t launch_products(const FfArgs& p, const FfMaps& maps, bool behind, cudaStream_t st) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(ff_products_kernel<O>, kFfSmem);
  if (e != cudaSuccess) return e;
  const unsigned grid = kGroup * (unsigned)(p.tiles < 152 / kGroup ? p.tiles : 152 / kGroup);
  if (behind) return launch_ahead(ff_products_kernel<O>, dim3(grid), kFfThreads, kFfSmem, st, p, maps);
  ff_products_kernel<O><<<grid, kFfThreads, kFfSmem, st>>>(p, maps);
  return cudaGetLastError();
}
cudaError_t launch_ff_products(const FfArgs& p, const FfMaps& maps, FfOperands kind, bool behind, cudaStream_t st) {
  const cudaError_t e = kind == FfOperands::kWhole    ? p.stages ? launch_products<Few>(p, maps, behind, st)
                                                                 : launch_products<Whole>(p, maps, behind, st)
                        : kind == FfOperands::kThirds ? launch_products<Thirds>(p, maps, behind, st)
                                                      : launch_products<Halves>(p, maps, behind, st);
  if (e == cudaSuccess) note_launch();
  return e;
}
cudaError_t launch_ff_join(const FfJoin& j, bool bf16, cudaStream_t st) {
  long long most = 0;
  for (int i = 0; i < j.probs; ++i) most = j.prob[i].n > most ? j.prob[i].n : most;
  const dim3 grid(grid_for(most, 1024), j.probs);
  const cudaError_t e = launch_ahead(bf16 ? ff_join_kernel<__nv_bfloat16> : ff_join_kernel<float>, grid, 256, 0, st, j);
  if (e == cudaSuccess) note_launch();
  return e;
}
cudaError_t launch_ff_split(const FfSplit& s, cudaStream_t st) {
  long long most = 0;
  for (int i = 0; i < s.tensors; ++i) most = s.n[i] > most ? s.n[i] : most;
  ff_split_kernel<<<dim3(grid_for(most, 2048), s.tensors), 256, 0, st>>>(s);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}
cudaError_t launch_ff_halves(const FfHalves& s, cudaStream_t st) {
  const long long rows = s.rows[0] + s.rows[1] + s.rows[2];
  auto grid = [&](int warps) { return (unsigned)((rows * warps + 7) / 8); };
  if (s.D <= 512) ff_halves_kernel<1, true><<<grid(1), 256, 0, st>>>(s);
  else if (s.D <= 1024) ff_halves_kernel<2, true><<<grid(2), 256, 0, st>>>(s);
  else if (s.D <= 2048) ff_halves_kernel<4, true><<<grid(4), 256, 0, st>>>(s);
  else if (s.D <= 4096) ff_halves_kernel<8, true><<<grid(8), 256, 0, st>>>(s);
  else ff_halves_kernel<8, false><<<grid(8), 256, 0, st>>>(s);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}
cudaError_t launch_ff_act_bwd(const void* dm, const void* gate, const void* up, void* dgate, void* dup, long long n, int act,
                              bool bf16, cudaStream_t st) {
  auto* dg = static_cast<__nv_bfloat16*>(dgate);
  auto* du = static_cast<__nv_bfloat16*>(dup);
  if (bf16) {
    using T = __nv_bfloat16;
    ff_act_bwd_kernel<T><<<grid_for(n, 2048), 256, 0, st>>>(static_cast<const T*>(dm), static_cast<const T*>(gate),
                                                            static_cast<const T*>(up), dg, du, n, act);
  } else {
    ff_act_bwd_kernel<float><<<grid_for(n, 1024), 256, 0, st>>>(static_cast<const float*>(dm), static_cast<const float*>(gate),
                                                                static_cast<const float*>(up), dg, du, n, act);
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ll
