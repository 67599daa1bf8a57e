// Kernels of the linear attention with a decay per head (the scan of lindecay.cuh) beside the
// tensor-core one: the prefix over segment totals, the fp32 scan, the single-token step.
#include <cuda_runtime.h>

#include "launch_util.cuh"
#include "lindecay.cuh"
#include "ptx.cuh"

namespace ll {

namespace {

// ---------------------------------------------------------------------------------
// lin_scan: segment totals -> the state at each segment's start, in place, in scan order:
// prefix_{s+1} = g^(tokens of s) prefix_s + total_s, prefix_0 = the start state or 0.  One
// thread per float4 of a (head, column tile); its loads do not depend on the running sum
// and are issued eight at a time, a batch ahead.
// ---------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) lin_scan_kernel(const __grid_constant__ LinArgs p) {
  ptx::launch_dependents();
  ptx::wait_for_prerequisites();  // launched while the totals are still being made
  const LinProb& r = p.pr[blockIdx.y];
  const int n4 = r.a * (kLinTile / 4);
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= (long long)r.nsplit * r.nh * n4) return;
  const int q = (int)(e % n4), uh = (int)(e / n4);
  LinItem x;
  x.prob = blockIdx.y;
  x.unit = r.split0 + uh / r.nh;
  lin_locate(p, x);
  const int tile = x.tile, b = x.b, h = x.oh * r.nh + uh % r.nh, bh = b * p.H + h;
  const int row = q / (kLinTile / 4), c = q % (kLinTile / 4) * 4;
  const int len = lin_len(p, b), span = p.L * p.chunk;
  const float l2 = lin_log2_decay(p.log_a, h);
  float4* s4 = reinterpret_cast<float4*>(r.seg) + (size_t)uh * p.nseg * n4 + q;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r.init && kLinTile * tile + c < r.b) {  // b is a multiple of 8: whole float4s
    const float* in =
        r.init + (size_t)bh * r.a * r.b + (size_t)row * r.init_rs + (size_t)(kLinTile * tile + c) * r.init_cs;
    acc = make_float4(in[0], in[r.init_cs], in[2 * (size_t)r.init_cs], in[3 * (size_t)r.init_cs]);
  }
  const int last = p.nseg - 1;
  constexpr int kBatch = 8;
  float4 now[kBatch], next[kBatch];
  auto fetch = [&](int i0, float4(&to)[kBatch]) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k < last) to[k] = s4[(size_t)(i0 + k) * n4];
  };
  fetch(0, now);
  for (int i0 = 0; i0 <= last; i0 += kBatch) {
    fetch(i0 + kBatch, next);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k;
      if (i <= last) {
        s4[(size_t)i * n4] = acc;
        // tokens of segment i: in sequence order it starts at chunk i L, or ends there from the end
        const int t0 = r.rev ? max(0, p.NC - (i + 1) * p.L) * p.chunk : i * span;
        const int t1 = r.rev ? (p.NC - i * p.L) * p.chunk : t0 + span;
        const float d = exp2f(l2 * (float)max(0, min(len, t1) - t0));
        acc.x = d * acc.x + now[k].x;
        acc.y = d * acc.y + now[k].y;
        acc.z = d * acc.z + now[k].z;
        acc.w = d * acc.w + now[k].w;
      }
      now[k] = next[k];
    }
  }
}

// ---------------------------------------------------------------------------------
// lin_f32: the scan in fp32, one CTA per item (a head's 64 output columns, or those of a
// whole group, over a unit or a segment), 64-token chunks in two buffers filled by cp.async.
//
// The products need fp32's accuracy, which the tensor cores give in three steps: a value is
// split into its first 11 significant bits (hi) and the rest (lo, exact, of which 11 bits
// enter), and a b = hi_a hi_b + hi_a lo_b + lo_a hi_b is accumulated in fp32; what is left
// out is of the order of 2^-22 |a b|.  The operands lie in shared memory as fp32 (tcgen05
// would need them there in 16 or 11 bits, both parts: twice the space) and are split in
// registers, so the warp-level instruction (m16n8k8) is used.
//
// Tile strides make the fragment loads free of bank conflicts: 8 mod 32 for operands that
// run along a row with k (two values at a time), 4 mod 32 for those that run along a row with
// n.  Y does both and has the second: its two-value loads take two turns.
//
// Bound: the instructions around the products.  Each step of 8 along k loads and splits eight
// values a lane for six products; the schedulers issue in half of the cycles, the tensor cores
// work in 30 % (their rate for this instruction: 294 TFLOP/s measured), the barriers between a
// chunk's four products take most of the rest.  A padded batch of 3 x 1501 tokens, 8 heads of
// 128 and 64: 78 us (138 with the products on the CUDA cores); 20000 tokens, 4 heads of 128 and
// 128: 300 us.
// ---------------------------------------------------------------------------------
constexpr int kF = 512;
constexpr int kC32 = kLinChunk32;
constexpr int kLdX = 136, kLdY = 132, kLdZ = 68, kLdP = 72;
struct F32Smem {
  float X[2][kC32 * kLdX];
  float Y[2][kC32 * kLdY];
  float Z[2][kC32 * kLdZ];
  float R[128 * kLdZ];
  float P[kC32 * kLdP];
  float pw[kC32 + 1];  // g^d
};

// x = hi + lo for a pair: hi is x rounded to tf32's 11 significant bits.
__device__ __forceinline__ void split_tf32(float2 x, uint32_t& h0, uint32_t& l0, uint32_t& h1, uint32_t& l1) {
  h0 = (__float_as_uint(x.x) + 0x1000u) & 0xffffe000u;
  h1 = (__float_as_uint(x.y) + 0x1000u) & 0xffffe000u;
  const float2 lo = ptx::fma2(make_float2(__uint_as_float(h0), __uint_as_float(h1)), make_float2(-1.f, -1.f), x);
  l0 = __float_as_uint(lo.x);
  l1 = __float_as_uint(lo.y);
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// acc (16 x 16, two n-tiles of 8) += A B over k = k0 .. k1 - 1 (multiples of 8), by one warp:
// A(m, k) = a[m sam + k sak], B(k, n) = b[k sbk + n sbn] wk(k); kA, kB: sak, sbk are 1.  The
// instruction's k = t and t + 4 are the tile's k = 2t and 2t + 1, on both sides, so that they lie
// next to each other in a row.
constexpr int kNt = 2;
template <bool kA, bool kB, typename W>
__device__ __forceinline__ void warp_mma(float (&acc)[kNt][4], const float* a, int sam, int sak, const float* b, int sbk,
                                         int sbn, int k0, int k1, W wk) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  // The instruction's own accumulation truncates: at most four steps add up in it before
  // they are added to acc in fp32 arithmetic.
  for (int kb = k0; kb < k1; kb += 32) {
    float part[kNt][4] = {};
    const int ke = min(kb + 32, k1);
#pragma unroll 4
    for (int k = kb; k < ke; k += 8) {
      uint32_t ah[4], al[4], bh[kNt][2], bl[kNt][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* p = a + (g + 8 * i) * sam + (k + 2 * t) * sak;
        const float2 x = kA ? *reinterpret_cast<const float2*>(p) : make_float2(p[0], p[sak]);
        split_tf32(x, ah[i], al[i], ah[2 + i], al[2 + i]);
      }
      const float w0 = wk(k + 2 * t), w1 = wk(k + 2 * t + 1);
#pragma unroll
      for (int j = 0; j < kNt; ++j) {
        const float* p = b + (k + 2 * t) * sbk + (8 * j + g) * sbn;
        const float2 x = kB ? *reinterpret_cast<const float2*>(p) : make_float2(p[0], p[sbk]);
        split_tf32(make_float2(w0 * x.x, w1 * x.y), bh[j][0], bl[j][0], bh[j][1], bl[j][1]);
      }
#pragma unroll
      for (int j = 0; j < kNt; ++j) mma_tf32(part[j], al, bh[j]);
#pragma unroll
      for (int j = 0; j < kNt; ++j) mma_tf32(part[j], ah, bl[j]);
#pragma unroll
      for (int j = 0; j < kNt; ++j) mma_tf32(part[j], ah, bh[j]);
    }
#pragma unroll
    for (int j = 0; j < kNt; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] += part[j][e];
  }
}
struct NoWeight {
  __device__ __forceinline__ float operator()(int) const { return 1.f; }
};

template <bool kStateOnly>
__global__ void __launch_bounds__(kF, 1) lin_f32_kernel(const __grid_constant__ LinArgs p) {
  extern __shared__ float4 smem4[];
  F32Smem& sm = *reinterpret_cast<F32Smem*>(smem4);
  if (kStateOnly) ptx::launch_dependents();
  else ptx::wait_for_prerequisites();  // segments' start states
  const int tid = threadIdx.x, warp = tid >> 5, g = (tid & 31) >> 2, t4 = tid & 3;
  const int wm = (warp & 3) * 16, wn = (warp >> 2) * 8 * kNt;  // this warp's part of a 64 x 64 tile
  int head0 = 0;
  const LinItem x =
      kStateOnly ? lin_state_item(p, (int)blockIdx.x, &head0) : lin_item(p, (int)blockIdx.x);
  const LinProb& r = p.pr[x.prob];
  const bool rev = r.rev != 0;
  const int sh = rev ? 0 : 1;
  const int a = r.a, b = r.b, c0 = kLinTile * x.tile, nc = min(kLinTile, b - c0);
  const int len = lin_len(p, x.b), cv = (len + kC32 - 1) / kC32;
  int first, step;
  const int n = lin_visit(p, x, cv, &first, &step);
  const float* Xg = static_cast<const float*>(r.X);
  const float* Yg = static_cast<const float*>(r.Y);
  const float* Zg = static_cast<const float*>(r.Z);
  float* out = static_cast<float*>(r.out);
  for (int hi_h = head0; hi_h < (kStateOnly ? head0 + 1 : r.nh); ++hi_h) {
    const int h = x.oh * r.nh + hi_h, grp = h / p.hpg;
    const int hx = r.xh == p.H ? h : grp, hy = r.yh == p.H ? h : grp, hz = r.zh == p.H ? h : grp;
    const size_t bh = (size_t)x.b * p.H + h;
    const float l2 = lin_log2_decay(p.log_a, h);
    float* seg = kStateOnly || x.from == kLinSeg ? lin_seg(p, x, hi_h) : nullptr;
    // rows of X, Y, Z of one chunk, by cp.async; zeros past the row's length (whatever lies
    // there must not reach a product) and past Z's columns
    auto load = [&](int k, int s) {
      const int ch = first + step * k;
      const int nv = min(kC32, len - ch * kC32);
      const size_t t0 = (size_t)x.b * p.T + (size_t)ch * kC32;
      const int a4 = a / 4;
      for (int e = tid; e < kC32 * a4; e += kF) {
        const int t = e / a4, c = e % a4 * 4;
        float* y = sm.Y[s] + t * kLdY + c;
        float* xx = sm.X[s] + t * kLdX + c;
        if (t < nv) {
          ptx::cp_async16(y, Yg + ((t0 + t) * r.yh + hy) * a + c);
          if (!kStateOnly) ptx::cp_async16(xx, Xg + ((t0 + t) * r.xh + hx) * a + c);
        } else {
          *reinterpret_cast<float4*>(y) = make_float4(0.f, 0.f, 0.f, 0.f);
          if (!kStateOnly) *reinterpret_cast<float4*>(xx) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      for (int e = tid; e < kC32 * (kLinTile / 4); e += kF) {
        const int t = e / (kLinTile / 4), c = e % (kLinTile / 4) * 4;
        float* z = sm.Z[s] + t * kLdZ + c;
        if (t < nv && c < nc) ptx::cp_async16(z, Zg + ((t0 + t) * r.zh + hz) * b + c0 + c);
        else *reinterpret_cast<float4*>(z) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      ptx::cp_async_commit();
    };
    __syncthreads();
    if (n > 0) load(0, 0);
    // R, rows a .. up to a multiple of 16 zero; and the columns of X and Y up to one of 8 are
    // all there (a is one)
    for (int e = tid; e < 128 * kLinTile; e += kF) {
      const int i = e / kLinTile, j = e % kLinTile;
      float v = 0.f;
      if (!kStateOnly && i < a) {
        if (seg) v = seg[e];
        else if (r.init && j < nc) v = r.init[bh * a * b + (size_t)i * r.init_rs + (size_t)(c0 + j) * r.init_cs];
      }
      sm.R[i * kLdZ + j] = v;
    }
    if (tid <= kC32) sm.pw[tid] = exp2f(l2 * (float)tid);
    for (int k = 0; k < n; ++k) {
      const int s = k & 1, ch = first + step * k;
      const int nv = min(kC32, len - ch * kC32);
      const size_t t0 = (size_t)x.b * p.T + (size_t)ch * kC32;
      if (k + 1 < n) {
        load(k + 1, s ^ 1);
        ptx::cp_async_wait_group<1>();
      } else {
        ptx::cp_async_wait_group<0>();
      }
      __syncthreads();
      const float *X = sm.X[s], *Y = sm.Y[s], *Z = sm.Z[s];
      // what a short call can do without: rows and keys past the length, R while it is zero and
      // R when nothing reads it any more (without states, 36 tokens: 17.5 -> 13.2 us, 3: 13.4 -> 8.0)
      const int nk = (nv + 7) & ~7;
      const bool zero = k == 0 && !seg && !r.init, last = k + 1 == n && !(r.fin && x.to == kLinInit);
      float acc[kNt][4];
      auto clear = [&]() {
#pragma unroll
        for (int j = 0; j < kNt; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
      };
      if (!kStateOnly) {
        clear();
        // S, only where some key of the warp's 16 x 16 part counts
        const bool some = wm < nv && wn < nv && (rev ? wn + 8 * kNt > wm : wn <= wm + 15);
        if (some) warp_mma<true, true>(acc, X + wm * kLdX, kLdX, 1, Y + wn * kLdY, 1, kLdY, 0, a, NoWeight());
#pragma unroll
        for (int j = 0; j < kNt; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = wm + g + 8 * (e >> 1), col = wn + 8 * j + 2 * t4 + (e & 1);
            const int d = rev ? col - row : row - col;
            sm.P[row * kLdP + col] = d >= 0 ? acc[j][e] * sm.pw[d] : 0.f;
          }
        // X R, its rows scaled, then P Z on top
        clear();
        if (wm < nv && !zero) warp_mma<true, false>(acc, X + wm * kLdX, kLdX, 1, sm.R + wn, kLdZ, 1, 0, a, NoWeight());
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = wm + g + 8 * (e >> 1);
          const float w = row < nv ? sm.pw[rev ? nv - 1 - row : row + sh] : 0.f;
#pragma unroll
          for (int j = 0; j < kNt; ++j) acc[j][e] *= w;
        }
        __syncthreads();  // P complete; R has been read
        if (wm < nv)
          warp_mma<true, false>(acc, sm.P + wm * kLdP, kLdP, 1, Z + wn, kLdZ, 1, rev ? wm : 0,
                                rev ? nk : min(nk, wm + 16), NoWeight());
#pragma unroll
        for (int j = 0; j < kNt; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = wm + g + 8 * e, col = wn + 8 * j + 2 * t4;
            if (ch * kC32 + t >= p.T || col >= nc) continue;
            float2* o = reinterpret_cast<float2*>(out + ((t0 + t) * r.oh + x.oh) * b + c0 + col);
            float2 v = t < nv ? make_float2(acc[j][2 * e], acc[j][2 * e + 1]) : make_float2(0.f, 0.f);
            if (hi_h > 0) {  // heads of the group add up, in order
              const float2 y = *o;
              v = make_float2(v.x + y.x, v.y + y.y);
            }
            *o = v;
          }
      }
      // R <- g^nv R + Yᵀ (w Z), 16 x 16 parts handed out to the warps
      const float dec = sm.pw[nv];
      const float* pw = sm.pw;
      // rows of Z past the length are zero: any weight will do there
      auto wz = [&](int t) { return pw[rev ? t + 1 : max(nv - 1 - t, 0)]; };
      for (int tile = warp; (kStateOnly || !last) && tile < (a + 15) / 16 * (kLinTile / (8 * kNt)); tile += kF / 32) {
        const int m0 = tile / (kLinTile / (8 * kNt)) * 16, n0 = tile % (kLinTile / (8 * kNt)) * 8 * kNt;
        float* R = sm.R + (m0 + g) * kLdZ + n0 + 2 * t4;
#pragma unroll
        for (int j = 0; j < kNt; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = dec * R[8 * (e >> 1) * kLdZ + 8 * j + (e & 1)];
        if (nk == kC32) warp_mma<false, false>(acc, Y + m0, 1, kLdY, Z + n0, kLdZ, 1, 0, kC32, wz);
        else warp_mma<false, false>(acc, Y + m0, 1, kLdY, Z + n0, kLdZ, 1, 0, nk, wz);
#pragma unroll
        for (int j = 0; j < kNt; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) R[8 * (e >> 1) * kLdZ + 8 * j + (e & 1)] = acc[j][e];
      }
      __syncthreads();  // the buffers are free, R is complete
    }
    __syncthreads();
    if (kStateOnly) {
      for (int e = tid; e < a * kLinTile; e += kF) seg[e] = sm.R[e / kLinTile * kLdZ + e % kLinTile];
    } else if (r.fin && x.to == kLinInit) {
      for (int e = tid; e < a * nc; e += kF)
        r.fin[(bh * a + e / nc) * b + c0 + e % nc] = sm.R[e / nc * kLdZ + e % nc];
    }
  }
  if (!kStateOnly) {  // chunks past the row's length: zeros
    int t0;
    const int t1 = lin_past(p, x, cv, &t0), n4 = nc / 4;
    for (int e = tid;; e += kF) {
      const int t = t0 + e / n4;
      if (t >= t1) break;
      *reinterpret_cast<float4*>(out + (((size_t)x.b * p.T + t) * r.oh + x.oh) * b + c0 + e % n4 * 4) =
          make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// ---------------------------------------------------------------------------------
// lin_step: one token.  S <- g S + k vᵀ, o = Sᵀ q, one pass over the fp32 states, which is
// all it costs (2 x 4 dk dv bytes per head against a few hundred for the rest).  A CTA
// takes 32 columns of a head's state: its threads load them (8 float4 columns x 16 rows at
// a time, up to 8 loads in flight a thread) before anything waits for q and k.  64 users of
// 48 heads of 128 and 64: 33.6 us, 6.05 TB/s, 89 % of the copy rate; one user 2.1 us.
// ---------------------------------------------------------------------------------
constexpr int kStepT = 128;
constexpr int kStepRows = kStepT / 8;
constexpr int kStepIter = 128 / kStepRows;

template <typename TIn>
__global__ void __launch_bounds__(kStepT) lin_step_kernel(LinStepArgs d) {
  __shared__ float qs[128], ks[128];
  __shared__ float4 red[kStepT / 32][8];
  const int tid = threadIdx.x;
  const int tiles = (d.dv + 31) / 32;
  const int bh = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int b = bh / d.H, h = bh % d.H;
  const int c = tile * 32 + (tid & 7) * 4, r0 = tid >> 3;
  const bool col = c < d.dv;  // dv is a multiple of 8: whole float4s
  float* S = d.states + (size_t)bh * d.dk * d.dv + c;
  float4 s[kStepIter];
#pragma unroll
  for (int i = 0; i < kStepIter; ++i) {
    const int row = r0 + i * kStepRows;
    if (col && row < d.dk) s[i] = *reinterpret_cast<const float4*>(S + (size_t)row * d.dv);
  }
  const size_t qk = ((size_t)b * (d.H / d.hpg) + h / d.hpg) * d.dk;
  if (tid < d.dk) {
    qs[tid] = ll_load(static_cast<const TIn*>(d.q), qk + tid);
    ks[tid] = ll_load(static_cast<const TIn*>(d.k), qk + tid);
  }
  const float g = exp2f(lin_log2_decay(d.log_a, h));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const size_t vo = (size_t)bh * d.dv + c;
  if (col) {
    const TIn* vp = static_cast<const TIn*>(d.v);
    v = make_float4(ll_load(vp, vo), ll_load(vp, vo + 1), ll_load(vp, vo + 2), ll_load(vp, vo + 3));
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kStepIter; ++i) {
    const int row = r0 + i * kStepRows;
    if (col && row < d.dk) {
      const float k = ks[row], q = qs[row];
      float4 x = s[i];
      x.x = g * x.x + k * v.x;
      x.y = g * x.y + k * v.y;
      x.z = g * x.z + k * v.z;
      x.w = g * x.w + k * v.w;
      *reinterpret_cast<float4*>(S + (size_t)row * d.dv) = x;
      acc.x += q * x.x;
      acc.y += q * x.y;
      acc.z += q * x.z;
      acc.w += q * x.w;
    }
  }
#pragma unroll
  for (int off = 8; off < 32; off <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
  }
  if ((tid & 31) < 8) red[tid >> 5][tid & 7] = acc;
  __syncthreads();
  if (tid < 8 && col) {
    float4 o = red[0][tid];
#pragma unroll
    for (int w = 1; w < kStepT / 32; ++w) {
      o.x += red[w][tid].x;
      o.y += red[w][tid].y;
      o.z += red[w][tid].z;
      o.w += red[w][tid].w;
    }
    TIn* op = static_cast<TIn*>(d.o);
    ll_store(op, vo, o.x);
    ll_store(op, vo + 1, o.y);
    ll_store(op, vo + 2, o.z);
    ll_store(op, vo + 3, o.w);
  }
}

}  // namespace

// A launch that may start while the kernel before it ends.
static cudaLaunchConfig_t dependent_launch(dim3 grid, int threads, int smem, cudaStream_t st, cudaLaunchAttribute* at) {
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

cudaError_t launch_lin_scan(const LinArgs& p, cudaStream_t st) {
  long long most = 0;
  for (int i = 0; i < p.nprob; ++i) {
    const long long n = (long long)p.pr[i].nsplit * p.pr[i].nh * p.pr[i].a * (kLinTile / 4);
    most = n > most ? n : most;
  }
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = dependent_launch(dim3((unsigned)((most + 255) / 256), p.nprob), 256, 0, st, at);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lin_scan_kernel, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_lin_f32(LinArgs& p, cudaStream_t st) {
  cudaError_t e;
  constexpr int smem = sizeof(F32Smem);
  if (p.nseg > 1) {
    static SmemLimit limit;
    if ((e = limit.raise(lin_f32_kernel<true>, smem)) != cudaSuccess) return e;
    lin_f32_kernel<true><<<p.sitems, kF, smem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    note_launch();
    if ((e = launch_lin_scan(p, st)) != cudaSuccess) return e;
  }
  static SmemLimit limit;
  if ((e = limit.raise(lin_f32_kernel<false>, smem)) != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  cudaLaunchConfig_t cfg = dependent_launch(dim3(p.items), kF, smem, st, at);
  if (p.nseg == 1) cfg.numAttrs = 0;
  if ((e = cudaLaunchKernelEx(&cfg, lin_f32_kernel<false>, p)) == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_lin_step(const LinStepArgs& d, bool bf16, cudaStream_t st) {
  const unsigned grid = (unsigned)(d.B * d.H * ((d.dv + 31) / 32));
  if (bf16) lin_step_kernel<__nv_bfloat16><<<grid, kStepT, 0, st>>>(d);
  else lin_step_kernel<float><<<grid, kStepT, 0, st>>>(d);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ll
