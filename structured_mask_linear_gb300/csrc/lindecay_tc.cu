// Tensor-core (tcgen05 / TMEM / TMA) kernels of the linear attention with a decay per head
// (the scan of lindecay.cuh) for bf16 tensors with widths up to 128, multiples of 8.
//
// One persistent CTA per SM walks units of work (a head's 64 output columns over one
// segment of the sequence) and, inside a unit, 128-token chunks in scan order.  The state
// R (a x 64) stays in registers between chunks, so each chunk's X, Y and Z are read once
// and its output written once.  Widths are padded to 64 or 128 by TMA's zero fill; columns
// past a width are clipped by the TMA store.
//
// Per chunk, in fp32 tensor-memory accumulators:
//     S  = X Yᵀ                    128 x 128 x a
//     Ob = X R                     128 x 64 x a     (R rounded to bf16)
//     D  = Yᵀ (Zhi + Zlo)          a x 64 x 128     (w_j Z_j as two bf16 parts)
//     Oa = P Z                     128 x 64 x 128   (P = S g^|i-j| masked, rounded to bf16)
// and out_i = Oa_i + g^(i'+sh) Ob_i, R <- g^nv R + D.
//
// Roundings: X, Y, Z enter exactly.  P and R enter their products as bf16, each an error of
// the size of out's own rounding to bf16 (independent, so out's relative error is about
// sqrt 2 of the rounding alone).  w_j Z_j enters as a high and a low bf16 part (16
// significant bits, relative error below 2^-17): the states are fp32 outputs, and an error
// made in one chunk stays in them.  R itself is carried in fp32.
//
// Warp roles (512 threads, 16 warps; 128 registers a thread):
//   warp 0      one thread issues the TMA loads, kStages chunks ahead
//   warp 1      one thread issues the MMAs, S one chunk ahead of the rest
//   warps 4-7   P: reads S, writes P over it in tensor memory (bf16, row t in lane t)
//   warps 8-11  state: w Z hi / lo, R's update, R's bf16 image for the next Ob
//   warps 12-15 output: Oa, Ob -> out, staged and stored by TMA
// Every mbarrier wait is bounded (wait_bar); one that runs out records LL_ERR_TIMEOUT and
// ends its role, the others follow by their own limits.
#include "lindecay.cuh"
#include "tc_common.cuh"

namespace ll {

namespace {

constexpr int kThreads = 512;
constexpr int kC = kLinChunk;
constexpr int kZBytes = kC * kLinTile * 2;  // 16 KB: 128 tokens x 64 columns, bf16
constexpr int kMisc = 1024;

template <int KA>
struct Lay {
  static constexpr int kX = kC * KA * 2;
  static constexpr int kStage = 2 * kX + kZBytes;  // X, Y, Z (in this order)
  static constexpr int kStages = KA == 64 ? 3 : 2;
  static constexpr int kZt = kStages * kStage;     // w Z: high part, low part
  static constexpr int kImg = kZt + 2 * kZBytes;   // R as bf16: KA rows x 128 bytes
  static constexpr int kOut = kImg + KA * 128;     // out tile on its way out
  static constexpr int kMiscOff = kOut + kZBytes;
  static constexpr int kBytes = kMiscOff + kMisc + 1024;  // + alignment
};
static_assert(Lay<128>::kBytes <= 232448, "shared memory");

struct LinMaps {
  CUtensorMap m[kLinProbs][4];  // X, Y, Z (loads), out (stores)
};

// Tensor-memory columns: S of even and odd chunks (P over their first 64, Oa in the last
// 64), Ob of even and odd chunks, D.
constexpr uint32_t kColS = 0, kColOb = 256, kColD = 384;

// The chunks a CTA works on, in order; every role walks the same sequence.
struct Walk {
  const LinArgs& p;
  bool state_only;
  int u;             // unit
  LinUnit x;
  int nh, hi;        // heads of the unit, current one
  int lo, hi_c, n;   // valid chunks [lo, hi_c) of the segment, their number
  int len;           // valid tokens of the batch row
  int k;             // index of the current chunk in scan order
  __device__ __forceinline__ Walk(const LinArgs& a, bool s) : p(a), state_only(s), u((int)blockIdx.x) { enter(); }
  __device__ __forceinline__ int total() const { return state_only ? p.sunits : p.units; }
  __device__ __forceinline__ bool live() const { return u < total(); }
  __device__ __forceinline__ void enter() {
    if (!live()) return;
    x = state_only ? lin_state_unit(p, u) : lin_unit(p, u);
    const LinProb& r = p.pr[x.prob];
    nh = (state_only || r.oh == p.H) ? 1 : p.hpg;
    hi = 0;
    len = lin_len(p, x.b);
    lo = x.seg * p.L;
    hi_c = min(min(lo + p.L, p.NC), (len + kC - 1) / kC);
    n = max(0, hi_c - lo);
    k = 0;
  }
  __device__ __forceinline__ int head() const { return x.oh * nh + hi; }
  __device__ __forceinline__ int chunk() const { return p.pr[x.prob].rev ? hi_c - 1 - k : lo + k; }
  __device__ __forceinline__ int valid() const { return min(kC, len - chunk() * kC); }
  // one (unit, head) at a time: the chunks of a run are k = 0 .. n - 1
  __device__ __forceinline__ void next_run() {
    k = 0;
    if (++hi == nh) {
      u += (int)gridDim.x;
      enter();
    }
  }
};

// Per-CTA barriers (in shared memory)
struct Bars {
  uint64_t full[3], empty[3], s_full[2], p_ready[2], o_full[2], o_empty[2], z_ready, r_ready, d_full, fin;
  uint32_t tmem;
};

__device__ __forceinline__ bool lin_wait(uint64_t* bar, uint32_t parity, const LinArgs& p) {
  if (wait_bar(bar, parity)) return true;
  atomicExch(p.status, kStatusTimeout);
  return false;
}
// The same for a role of whole warps: every lane continues or none.
__device__ __forceinline__ bool lin_wait_warp(uint64_t* bar, uint32_t parity, const LinArgs& p) {
  return __all_sync(0xffffffffu, lin_wait(bar, parity, p));
}

template <int KA, bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 1) lin_tc_kernel(const __grid_constant__ LinMaps maps,
                                                             const __grid_constant__ LinArgs p) {
  using S = Lay<KA>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + S::kMiscOff);
  float* s_cf = reinterpret_cast<float*>(smem + S::kMiscOff + 256);  // 32
  float* s_dt = s_cf + 32;                                           // 64
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      ptx::mbar_init(&bars.full[i], 1);
      ptx::mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars.s_full[i], 1);
      ptx::mbar_init(&bars.p_ready[i], 128);
      ptx::mbar_init(&bars.o_full[i], 1);
      ptx::mbar_init(&bars.o_empty[i], 128);
    }
    ptx::mbar_init(&bars.z_ready, 128);
    ptx::mbar_init(&bars.r_ready, 128);
    ptx::mbar_init(&bars.d_full, 1);
    ptx::mbar_init(&bars.fin, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&bars.tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tb = bars.tmem;

  if (tid == 0) {
    // ---- loads --------------------------------------------------------------------------
    uint32_t it = 0;
    bool ok = true;
    for (Walk w(p, kStateOnly); ok && w.live(); w.next_run()) {
      const LinProb& r = p.pr[w.x.prob];
      const CUtensorMap* m = maps.m[w.x.prob];
      const int h = w.head(), g = h / p.hpg;
      const int hx = r.xh == p.H ? h : g, hy = r.yh == p.H ? h : g, hz = r.zh == p.H ? h : g;
      for (; w.k < w.n; ++w.k, ++it) {
        const uint32_t s = it % S::kStages;
        if (it >= (uint32_t)S::kStages && !lin_wait(&bars.empty[s], ((it / S::kStages) & 1) ^ 1, p)) {
          ok = false;
          break;
        }
        uint8_t* st = smem + s * S::kStage;
        const int t0 = w.chunk() * kC;
        ptx::mbar_arrive_expect_tx(&bars.full[s], kStateOnly ? S::kX + kZBytes : S::kStage);
#pragma unroll
        for (int c = 0; c < KA / 64; ++c) {
          if (!kStateOnly) ptx::tma_load_4d(st + c * 16384, &m[0], &bars.full[s], 64 * c, hx, t0, w.x.b);
          ptx::tma_load_4d(st + S::kX + c * 16384, &m[1], &bars.full[s], 64 * c, hy, t0, w.x.b);
        }
        ptx::tma_load_4d(st + 2 * S::kX, &m[2], &bars.full[s], kLinTile * w.x.tile, hz, t0, w.x.b);
      }
    }
    if (!ok)  // let the copies in flight land before the CTA ends (bounded)
      for (uint32_t j = it >= (uint32_t)S::kStages ? it - S::kStages : 0; j < it; ++j)
        wait_bar(&bars.full[j % S::kStages], (j / S::kStages) & 1);
  } else if (tid == 32) {
    // ---- MMAs ---------------------------------------------------------------------------
    uint32_t n = 0;  // chunks of this CTA
    for (Walk w(p, kStateOnly); w.live(); w.next_run()) n += w.n;
    const uint32_t s0 = ptx::smem_u32(smem);
    const uint32_t img = s0 + S::kImg, zt = s0 + S::kZt;
    auto issue_s = [&](uint32_t it) -> bool {
      const uint32_t st = it % S::kStages, bf = it & 1;
      if (!lin_wait(&bars.full[st], (it / S::kStages) & 1, p)) return false;
      if (it >= 2 && !lin_wait(&bars.o_empty[bf], ((it >> 1) & 1) ^ 1, p)) return false;
      ptx::tc_fence_after();
      const uint32_t x0 = s0 + st * S::kStage, y0 = x0 + S::kX;
      const uint32_t idesc = ptx::idesc_bf16_f32(128, 128, 0, 0);
#pragma unroll
      for (int kk = 0; kk < KA / 16; ++kk) {
        const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
        ptx::umma_f16(tb + kColS + 128 * bf, ptx::smem_desc_sw128(x0 + off, 16, 1024),
                      ptx::smem_desc_sw128(y0 + off, 16, 1024), idesc, kk > 0);
      }
      ptx::umma_commit(&bars.s_full[bf]);
      return true;
    };
    bool ok = kStateOnly || n == 0 || issue_s(0);
    for (uint32_t it = 0; ok && it < n; ++it) {
      const uint32_t st = it % S::kStages, bf = it & 1, par = it & 1;
      const uint32_t x0 = s0 + st * S::kStage, y0 = x0 + S::kX, z0 = x0 + 2 * S::kX;
      if (!kStateOnly) {
        if (it + 1 < n && !issue_s(it + 1)) break;
        if (!lin_wait(&bars.r_ready, par, p)) break;
        ptx::tc_fence_after();
        const uint32_t idesc = ptx::idesc_bf16_f32(128, 64, 0, 1);
#pragma unroll
        for (int kk = 0; kk < KA / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          ptx::umma_f16(tb + kColOb + 64 * bf, ptx::smem_desc_sw128(x0 + off, 16, 1024),
                        ptx::smem_desc_sw128(img + kk * 2048, 1024, 1024), idesc, kk > 0);
        }
      }
      if (!lin_wait(&bars.z_ready, par, p)) break;
      ptx::tc_fence_after();
      // D: A = Yᵀ (M = 128, both MN-major).  With a padded to 64 the second 64 rows of A
      // read Z's tile that follows Y (LBO 16 KB): lanes 64..127 of D are never read.
      const uint32_t idesc_d = ptx::idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk)
          ptx::umma_f16(tb + kColD, ptx::smem_desc_sw128(y0 + kk * 2048, 16384, 1024),
                        ptx::smem_desc_sw128(zt + part * kZBytes + kk * 2048, 1024, 1024), idesc_d, part + kk > 0);
      ptx::umma_commit(&bars.d_full);
      if (!kStateOnly) {
        if (!lin_wait(&bars.p_ready[bf], (it >> 1) & 1, p)) break;
        ptx::tc_fence_after();
        const uint32_t idesc = ptx::idesc_bf16_f32(128, 64, 0, 1);
        const uint32_t tp = tb + kColS + 128 * bf;
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk)
          ptx::umma_f16_tmem_a(tp + 64, tp + kk * 8, ptx::smem_desc_sw128(z0 + kk * 2048, 1024, 1024), idesc, kk > 0);
        ptx::umma_commit(&bars.o_full[bf]);
      }
      ptx::umma_commit(&bars.empty[st]);
    }
  } else if (!kStateOnly && warp >= 4 && warp < 8) {
    // ---- P ------------------------------------------------------------------------------
    const int quad = warp - 4;
    const uint32_t loff = (uint32_t)(quad * 32) << 16;
    uint32_t it = 0;
    bool ok = true;
    for (Walk w(p, false); ok && w.live(); w.next_run()) {
      if (w.n == 0) continue;
      const bool rev = p.pr[w.x.prob].rev != 0;
      const float l2 = lin_log2_decay(p.log_a, w.head());
      // g^(j - i) tables over 32 keys: off the diagonal 32-group g^|i-j| is the product of a
      // factor of the row and group (to the group's nearest key) and one of the key, both
      // <= 1; on it the power of the lag itself, 0 where the lag is negative.
      ptx::named_bar_sync(1, 128);
      if (quad == 0) {
        s_cf[lane] = exp2f(l2 * (float)(rev ? lane : 31 - lane));
      } else if (quad < 3) {
        const int x = (quad - 1) * 32 + lane;  // key - row + 31
        const int d = rev ? x - 31 : 31 - x;
        s_dt[x] = d < 0 ? 0.f : exp2f(l2 * (float)d);
      }
      ptx::named_bar_sync(1, 128);
      const float* dt = s_dt + 31 - lane;
      for (; w.k < w.n; ++w.k, ++it) {
        const uint32_t bf = it & 1;
        const int nv = w.valid();
        if (!lin_wait_warp(&bars.s_full[bf], (it >> 1) & 1, p)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t ts = tb + kColS + 128 * bf + loff;
#pragma unroll 1
        for (int cg = 0; cg < 4; ++cg) {
          uint32_t pk[16];
          if (cg == quad || (cg < quad) != rev) {
            float sv[32];
            ptx::tmem_ld32(ts + cg * 32, sv);
            if (cg == quad) {
              ptx::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float f = dt[j];
                sv[j] = f != 0.f ? sv[j] * f : 0.f;
              }
            } else {
              const float rf = exp2f(l2 * (float)(rev ? 32 * (cg - quad) - lane : 32 * (quad - cg) + lane - 31));
              const float4* c4 = reinterpret_cast<const float4*>(s_cf);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int j4 = 0; j4 < 8; ++j4) {
                const float4 c = c4[j4];
                sv[4 * j4] *= rf * c.x;
                sv[4 * j4 + 1] *= rf * c.y;
                sv[4 * j4 + 2] *= rf * c.z;
                sv[4 * j4 + 3] *= rf * c.w;
              }
            }
            if (rev && nv < 32 * cg + 32) {  // keys past the row's length (warp-uniform)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (32 * cg + j >= nv) sv[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(sv[2 * j], sv[2 * j + 1]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = 0u;
          }
          // packed columns 16 cg ..: they held S of keys below 32 cg, all read before
          ptx::tmem_st16(ts + cg * 16, pk);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bars.p_ready[bf]);
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // ---- state --------------------------------------------------------------------------
    // Thread r of the role: token r of the chunk for w Z, row r of R.
    const int row = tid - 256, quad = warp - 8, rot = row & 7;
    const uint32_t td = tb + kColD + ((uint32_t)(quad * 32) << 16);
    uint8_t* zhi = smem + S::kZt + row * 128;
    uint8_t* img = smem + S::kImg + row * 128;
    const bool holds = row < KA;  // warp-uniform: this thread has a row of R
    uint32_t it = 0;
    bool ok = true;
    float R[kLinTile];
    auto write_image = [&]() {
      if (holds) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(img + ((c ^ rot) << 4)) =
              make_uint4(pack_bf16(R[8 * c], R[8 * c + 1]), pack_bf16(R[8 * c + 2], R[8 * c + 3]),
                         pack_bf16(R[8 * c + 4], R[8 * c + 5]), pack_bf16(R[8 * c + 6], R[8 * c + 7]));
        ptx::fence_proxy_async_smem();
      }
      ptx::mbar_arrive(&bars.r_ready);
    };
    for (Walk w(p, kStateOnly); ok && w.live(); w.next_run()) {
      const LinProb& r = p.pr[w.x.prob];
      const bool rev = r.rev != 0;
      const int h = w.head();
      const size_t bh = (size_t)w.x.b * p.H + h;
      const int c0 = kLinTile * w.x.tile;
      const int nc = min(kLinTile, r.b - c0);  // columns of this tile, a multiple of 8
      const float l2 = lin_log2_decay(p.log_a, h);
      float* seg = r.seg ? r.seg + (((bh * r.tiles + w.x.tile) * p.nseg + w.x.seg) * r.a + row) * kLinTile : nullptr;
#pragma unroll
      for (int j = 0; j < kLinTile; ++j) R[j] = 0.f;
      if (!kStateOnly && row < r.a) {
        if (p.nseg > 1) {
#pragma unroll
          for (int j = 0; j < kLinTile; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(seg + j);
            R[j] = x.x;
            R[j + 1] = x.y;
            R[j + 2] = x.z;
            R[j + 3] = x.w;
          }
        } else if (r.init) {
          const float* in = r.init + bh * r.a * r.b + (size_t)row * r.init_rs + (size_t)c0 * r.init_cs;
#pragma unroll
          for (int j = 0; j < kLinTile; ++j)
            if (j < nc) R[j] = in[(size_t)j * r.init_cs];
        }
      }
      if (!kStateOnly && w.n > 0) write_image();
      for (; w.k < w.n; ++w.k, ++it) {
        const uint32_t s = it % S::kStages;
        const int nv = w.valid();
        uint8_t* y0 = smem + s * S::kStage + S::kX + row * 128;
        uint8_t* z0 = smem + s * S::kStage + 2 * S::kX + row * 128;
        if (!lin_wait_warp(&bars.full[s], (it / S::kStages) & 1, p)) {
          ok = false;
          break;
        }
        if (row < nv) {
          const float wt = exp2f(l2 * (float)(rev ? row + 1 : nv - 1 - row));
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int off = (c ^ rot) << 4;
            uint4 x = *reinterpret_cast<const uint4*>(z0 + off), y;
            __nv_bfloat162* hx = reinterpret_cast<__nv_bfloat162*>(&x);
            __nv_bfloat162* hy = reinterpret_cast<__nv_bfloat162*>(&y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 f = __bfloat1622float2(hx[e]);
              f.x *= wt;
              f.y *= wt;
              hx[e] = __floats2bfloat162_rn(f.x, f.y);
              const float2 rr = __bfloat1622float2(hx[e]);
              hy[e] = __floats2bfloat162_rn(f.x - rr.x, f.y - rr.y);
            }
            *reinterpret_cast<uint4*>(zhi + off) = x;
            *reinterpret_cast<uint4*>(zhi + kZBytes + off) = y;
          }
        } else {
          // past the row's length: whatever the padding holds must not reach a product
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            *reinterpret_cast<uint4*>(zhi + (c << 4)) = zero;
            *reinterpret_cast<uint4*>(zhi + kZBytes + (c << 4)) = zero;
            *reinterpret_cast<uint4*>(z0 + (c << 4)) = zero;
#pragma unroll
            for (int d = 0; d < KA / 64; ++d) *reinterpret_cast<uint4*>(y0 + d * 16384 + (c << 4)) = zero;
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bars.z_ready);
        if (!lin_wait_warp(&bars.d_full, it & 1, p)) {
          ok = false;
          break;
        }
        if (holds) {
          ptx::tc_fence_after();
          const float dec = exp2f(l2 * (float)nv);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float d[32];
            ptx::tmem_ld32(td + 32 * q, d);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) R[32 * q + j] = dec * R[32 * q + j] + d[j];
          }
          ptx::tc_fence_before();
        }
        if (!kStateOnly && w.k + 1 < w.n) write_image();  // Ob of this chunk has completed (before D)
      }
      if (!ok) break;
      if (row < r.a) {
        if (kStateOnly) {
#pragma unroll
          for (int j = 0; j < kLinTile; j += 4)
            *reinterpret_cast<float4*>(seg + j) = make_float4(R[j], R[j + 1], R[j + 2], R[j + 3]);
        } else if (r.fin && w.x.seg == (rev ? 0 : p.nseg - 1)) {
          float* out = r.fin + (bh * r.a + row) * r.b + c0;
#pragma unroll
          for (int j = 0; j < kLinTile; j += 4)
            if (j < nc) *reinterpret_cast<float4*>(out + j) = make_float4(R[j], R[j + 1], R[j + 2], R[j + 3]);
        }
      }
    }
  } else if (!kStateOnly && warp >= 12) {
    // ---- output -------------------------------------------------------------------------
    const int row = tid - 384, quad = warp - 12, rot = row & 7;
    const uint32_t loff = (uint32_t)(quad * 32) << 16;
    uint8_t* stage = smem + S::kOut;
    float4* scr = reinterpret_cast<float4*>(p.scratch) + (size_t)blockIdx.x * p.L * (kC * kLinTile / 4) + row;
    uint32_t it = 0;
    bool ok = true;
    for (Walk w(p, false); ok && w.live(); w.next_run()) {
      const LinProb& r = p.pr[w.x.prob];
      const bool rev = r.rev != 0;
      const float l2 = lin_log2_decay(p.log_a, w.head());
      const bool first = w.hi == 0, last = w.hi + 1 == w.nh;
      const int c0 = kLinTile * w.x.tile;
      for (; w.k < w.n; ++w.k, ++it) {
        const uint32_t bf = it & 1;
        const int nv = w.valid(), ch = w.chunk();
        // sums over a group's heads: 16 float4 per row, consecutive rows side by side
        float4* sc = scr + (size_t)w.k * (kC * kLinTile / 4);
        const bool in = row < nv;
        const float wo = exp2f(l2 * (float)(rev ? nv - 1 - row : row + 1));
        if (!lin_wait_warp(&bars.o_full[bf], (it >> 1) & 1, p)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (last) {
          if (row == 0) ptx::bulk_wait_read_all();  // the previous tile has left the staging area
          ptx::named_bar_sync(2, 128);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float oa[32], ob[32];
          ptx::tmem_ld32(tb + kColS + 128 * bf + 64 + 32 * q + loff, oa);
          ptx::tmem_ld32(tb + kColOb + 64 * bf + 32 * q + loff, ob);
          ptx::tmem_ld_wait();
          if (q == 1) {
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bars.o_empty[bf]);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) oa[j] = in ? oa[j] + wo * ob[j] : 0.f;
          if (!first) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 y = sc[(8 * q + j) * kC];
              oa[4 * j] += y.x;
              oa[4 * j + 1] += y.y;
              oa[4 * j + 2] += y.z;
              oa[4 * j + 3] += y.w;
            }
          }
          if (!last) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sc[(8 * q + j) * kC] = make_float4(oa[4 * j], oa[4 * j + 1], oa[4 * j + 2], oa[4 * j + 3]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(stage + row * 128 + (((4 * q + c) ^ rot) << 4)) =
                  make_uint4(pack_bf16(oa[8 * c], oa[8 * c + 1]), pack_bf16(oa[8 * c + 2], oa[8 * c + 3]),
                             pack_bf16(oa[8 * c + 4], oa[8 * c + 5]), pack_bf16(oa[8 * c + 6], oa[8 * c + 7]));
          }
        }
        if (last) {
          ptx::fence_proxy_async_smem();
          ptx::named_bar_sync(2, 128);
          if (row == 0) {
            ptx::tma_store_4d(&maps.m[w.x.prob][3], stage, c0, w.x.oh, ch * kC, w.x.b);
            ptx::bulk_commit_group();
          }
        }
      }
      if (ok && last) {  // chunks past the row's length: zeros
        const int t1 = min(p.T, min((w.x.seg + 1) * p.L, p.NC) * kC);
        const int nv8 = min(kLinTile, r.b - c0) / 8;
        for (int t = max(w.lo, w.lo + w.n) * kC + row; t < t1; t += kC) {
          uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(r.out) +
                                              (((size_t)w.x.b * p.T + t) * r.oh + w.x.oh) * r.b + c0);
          for (int c = 0; c < nv8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    if (row == 0) ptx::bulk_wait_read_all();
  }
  // join; on a timeout the MMAs issued may still run: give them a bounded wait
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) {
    if (*reinterpret_cast<volatile unsigned*>(p.status) == kStatusTimeout) {
      if (lane == 0) {
        ptx::umma_commit(&bars.fin);
        wait_bar(&bars.fin, 0);
      }
      __syncwarp();
    }
    ptx::tmem_dealloc(tb, 512);
  }
}

bool lin_map(CUtensorMap* m, const void* base, int inner, int count, int T, int B) {
  return make_map(m, base, inner, count, T, B);
}

template <int KA>
cudaError_t launch_ka(LinArgs& p, const LinMaps& maps, int ctas, cudaStream_t st) {
  constexpr int smem = Lay<KA>::kBytes;
  cudaError_t e;
  if (p.nseg > 1) {
    if ((e = cudaFuncSetAttribute(lin_tc_kernel<KA, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
        cudaSuccess)
      return e;
    lin_tc_kernel<KA, true><<<min(ctas, p.sunits), kThreads, smem, st>>>(maps, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    note_launch();
    if ((e = launch_lin_scan(p, st)) != cudaSuccess) return e;
  }
  if ((e = cudaFuncSetAttribute(lin_tc_kernel<KA, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
      cudaSuccess)
    return e;
  lin_tc_kernel<KA, false><<<min(ctas, p.units), kThreads, smem, st>>>(maps, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  note_launch();
  return cudaSuccess;
}

}  // namespace

bool lin_is_wide(int a) { return a > 64; }

// Every scan of p pads a to the same width (64 or 128).
cudaError_t launch_lin_tc(LinArgs& p, int ctas, cudaStream_t st) {
  LinMaps maps;
  for (int i = 0; i < p.nprob; ++i) {
    const LinProb& r = p.pr[i];
    if (!lin_map(&maps.m[i][0], r.X, r.a, r.xh, p.T, p.B) || !lin_map(&maps.m[i][1], r.Y, r.a, r.yh, p.T, p.B) ||
        !lin_map(&maps.m[i][2], r.Z, r.b, r.zh, p.T, p.B) || !lin_map(&maps.m[i][3], r.out, r.b, r.oh, p.T, p.B))
      return cudaErrorInvalidValue;
  }
  for (int i = p.nprob; i < kLinProbs; ++i)
    for (int j = 0; j < 4; ++j) maps.m[i][j] = maps.m[0][j];
  return lin_is_wide(p.pr[0].a) ? launch_ka<128>(p, maps, ctas, st) : launch_ka<64>(p, maps, ctas, st);
}

}  // namespace ll
