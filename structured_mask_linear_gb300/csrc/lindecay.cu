// CUDA-core kernels of the linear attention with a decay per head (the scan of
// lindecay.cuh): the prefix over segment totals, the fp32 scan, and the single-token step.
#include <cuda_runtime.h>

#include "launch_util.cuh"
#include "lindecay.cuh"

namespace ll {

namespace {

// ---------------------------------------------------------------------------------
// lin_scan: segment totals -> the state at each segment's start, in place, in scan order:
// prefix_{s+1} = g^(tokens of s) prefix_s + total_s, prefix_0 = the start state or 0.  One
// thread per float4 of a (head, column tile); its loads do not depend on the running sum
// and are issued eight at a time, a batch ahead.
// ---------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) lin_scan_kernel(const __grid_constant__ LinArgs p) {
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
// lin_f32: the scan in fp32, one CTA per unit (a head's 64 output columns, or those of a
// whole group, over one segment), 64-token chunks.  X and Z sit in shared memory by token,
// Y transposed, R by row; the four products of a chunk run on the CUDA cores from there.
// ---------------------------------------------------------------------------------
constexpr int kF = 256;
constexpr int kC32 = kLinChunk32;
constexpr int kLd = 68;  // row stride of 64-wide tiles
struct F32Smem {
  float Yt[128 * kLd];
  float R[128 * kLd];
  float X[kC32 * 132];
  float Z[kC32 * kLd];
  float Zw[kC32 * kLd];
  float P[kC32 * kLd];
  float pw[kC32 + 1];  // g^d
};

template <bool kStateOnly>
__global__ void __launch_bounds__(kF, 1) lin_f32_kernel(const __grid_constant__ LinArgs p) {
  extern __shared__ float4 smem4[];
  F32Smem& sm = *reinterpret_cast<F32Smem*>(smem4);
  const int tid = threadIdx.x;
  int head0 = 0;
  const LinItem x =
      kStateOnly ? lin_state_item(p, (int)blockIdx.x, &head0) : lin_item(p, (int)blockIdx.x);
  const LinProb& r = p.pr[x.prob];
  const bool rev = r.rev != 0;
  const int sh = rev ? 0 : 1;
  const int a = r.a, b = r.b, c0 = kLinTile * x.tile, nc = min(kLinTile, b - c0);
  const int ldx = a + 4;
  const int len = lin_len(p, x.b), cv = (len + kC32 - 1) / kC32;
  int first, step;
  const int n = lin_visit(p, x, cv, &first, &step);
  const float* Xg = static_cast<const float*>(r.X);
  const float* Yg = static_cast<const float*>(r.Y);
  const float* Zg = static_cast<const float*>(r.Z);
  float* out = static_cast<float*>(r.out);
  for (int hi_h = head0; hi_h < (kStateOnly ? head0 + 1 : r.nh); ++hi_h) {
    const int h = x.oh * r.nh + hi_h, g = h / p.hpg;
    const int hx = r.xh == p.H ? h : g, hy = r.yh == p.H ? h : g, hz = r.zh == p.H ? h : g;
    const size_t bh = (size_t)x.b * p.H + h;
    const float l2 = lin_log2_decay(p.log_a, h);
    float* seg = kStateOnly || x.from == kLinSeg ? lin_seg(p, x, hi_h) : nullptr;
    __syncthreads();
    for (int e = tid; e < a * kLinTile; e += kF) {
      const int i = e / kLinTile, j = e % kLinTile;
      float v = 0.f;
      if (!kStateOnly) {
        if (seg) v = seg[e];
        else if (r.init && j < nc) v = r.init[bh * a * b + (size_t)i * r.init_rs + (size_t)(c0 + j) * r.init_cs];
      }
      sm.R[i * kLd + j] = v;
    }
    if (tid <= kC32) sm.pw[tid] = exp2f(l2 * (float)tid);
    for (int k = 0; k < n; ++k) {
      const int ch = first + step * k;
      const int nv = min(kC32, len - ch * kC32);
      const size_t t0 = (size_t)x.b * p.T + (size_t)ch * kC32;
      __syncthreads();
      const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!kStateOnly)
        for (int e = tid; e < kC32 * (a / 4); e += kF) {
          const int t = e / (a / 4), c = e % (a / 4) * 4;
          *reinterpret_cast<float4*>(sm.X + t * ldx + c) =
              t < nv ? *reinterpret_cast<const float4*>(Xg + ((t0 + t) * r.xh + hx) * a + c) : zero4;
        }
      for (int e = tid; e < kC32 * (a / 4); e += kF) {
        const int t = e % kC32, c = e / kC32 * 4;
        const float4 y = t < nv ? *reinterpret_cast<const float4*>(Yg + ((t0 + t) * r.yh + hy) * a + c) : zero4;
        sm.Yt[c * kLd + t] = y.x;
        sm.Yt[(c + 1) * kLd + t] = y.y;
        sm.Yt[(c + 2) * kLd + t] = y.z;
        sm.Yt[(c + 3) * kLd + t] = y.w;
      }
      for (int e = tid; e < kC32 * (kLinTile / 4); e += kF) {
        const int t = e / (kLinTile / 4), c = e % (kLinTile / 4) * 4;
        const float4 z =
            (t < nv && c < nc) ? *reinterpret_cast<const float4*>(Zg + ((t0 + t) * r.zh + hz) * b + c0 + c) : zero4;
        const float w = t < nv ? sm.pw[rev ? t + 1 : nv - 1 - t] : 0.f;
        *reinterpret_cast<float4*>(sm.Z + t * kLd + c) = z;
        *reinterpret_cast<float4*>(sm.Zw + t * kLd + c) = make_float4(w * z.x, w * z.y, w * z.z, w * z.w);
      }
      __syncthreads();
      if (!kStateOnly) {
        smem_mm(kC32, kC32, a, sm.X, ldx, 1, sm.Yt, kLd, tid, kF, [&](int m0, int n0, float(&acc)[4][4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float4 v;
            float* o = &v.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int d = rev ? n0 + j - m0 - i : m0 + i - n0 - j;
              o[j] = d >= 0 ? acc[i][j] * sm.pw[d] : 0.f;
            }
            *reinterpret_cast<float4*>(sm.P + (m0 + i) * kLd + n0) = v;
          }
        });
        // X R: the 16 x 16 output tiles are one per thread, the same one in both products
        float it[4][4];
        smem_mm(kC32, kLinTile, a, sm.X, ldx, 1, sm.R, kLd, tid, kF, [&](int m0, int, float(&acc)[4][4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = m0 + i;
            const float w = t < nv ? sm.pw[rev ? nv - 1 - t : t + sh] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) it[i][j] = w * acc[i][j];
          }
        });
        __syncthreads();
        smem_mm_r(
            kC32, kLinTile, kC32, sm.P, kLd, 1, sm.Z, kLd, tid, kF,
            [&](int m0, int, int& kb, int& ke) {
              if (rev) kb = m0;
              else ke = m0 + 4;
            },
            [&](int m0, int n0, float(&acc)[4][4]) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int t = m0 + i;
                if (ch * kC32 + t >= p.T || n0 >= nc) continue;
                float4* o = reinterpret_cast<float4*>(out + ((t0 + t) * r.oh + x.oh) * b + c0 + n0);
                float4 v = t < nv ? make_float4(acc[i][0] + it[i][0], acc[i][1] + it[i][1], acc[i][2] + it[i][2],
                                                acc[i][3] + it[i][3])
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                if (hi_h > 0) {  // heads of the group add up, in order
                  const float4 y = *o;
                  v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
                }
                *o = v;
              }
            });
      }
      const float dec = sm.pw[nv];
      smem_mm(a, kLinTile, kC32, sm.Yt, kLd, 1, sm.Zw, kLd, tid, kF, [&](int m0, int n0, float(&acc)[4][4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& R = sm.R[(m0 + i) * kLd + n0 + j];
            R = dec * R + acc[i][j];
          }
      });
    }
    __syncthreads();
    if (kStateOnly) {
      for (int e = tid; e < a * kLinTile; e += kF) seg[e] = sm.R[e / kLinTile * kLd + e % kLinTile];
    } else if (r.fin && x.to == kLinInit) {
      for (int e = tid; e < a * nc; e += kF)
        r.fin[(bh * a + e / nc) * b + c0 + e % nc] = sm.R[e / nc * kLd + e % nc];
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
// a time, up to 8 loads in flight a thread) before anything waits for q and k.
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

cudaError_t launch_lin_scan(const LinArgs& p, cudaStream_t st) {
  long long most = 0;
  for (int i = 0; i < p.nprob; ++i) {
    const long long n = (long long)p.pr[i].nsplit * p.pr[i].nh * p.pr[i].a * (kLinTile / 4);
    most = n > most ? n : most;
  }
  lin_scan_kernel<<<dim3((unsigned)((most + 255) / 256), p.nprob), 256, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
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
  lin_f32_kernel<false><<<p.items, kF, smem, st>>>(p);
  if ((e = cudaGetLastError()) == cudaSuccess) note_launch();
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
