// The norms around a block, fused with its gate and the residual scale, and their gradients.
//
// Per row (token) of D values, rms over groups of `group` values for the block's output and
// over the whole row for the residual stream:
//     n  = y rsqrt(mean_group(y²) + eps) w_post
//     x' = x + scale act(gate) n
//     h  = x' rsqrt(mean(x'²) + eps) w_pre
// with x, gate, w_post, scale and the (w_pre, h) pair each optional.  Gradients, given dx'
// and dh (r1, r2 the two rsqrt):
//     u   = dh w_pre,       dx = dx' + r2 (u - x' r2² mean(u x')),   dw_pre = sum dh x' r2
//     dm  = dx scale,       dscale = sum dx act(gate) n,             dgate = dm n act'(gate)
//     dn  = dm act(gate),   dw_post = sum dn y r1
//     un  = dn w_post,      dy = r1 (un - y r1² mean_group(un y))
// All sums are fp32; values are rounded once, where they are stored.  h is the norm of x'
// before x' is rounded; the gradients take x' as stored.  Only normalised values (y r1, x' r2)
// are multiplied by a further rsqrt: its square or cube alone leaves fp32's range where a row
// is zeros or tiny (eps = 1e-30: r1 = 1e15) or huge, while the gradient does not.
//
// Both directions are bound by memory: each activation is read once and written once.
// 32768 rows of 4096 in bf16, every part: forward 230 us, 5.85 TB/s, 86 % of the copy rate;
// 16384 rows: backward 215 us, 5.0 TB/s, 74 % (the rest is a step's reductions, which overlap
// the other CTA's copies only in part).  A row alone takes 2.9 us forwards, 7 backwards.
#include <cuda_runtime.h>

#include "blocknorm.cuh"
#include "launch_util.cuh"
#include "ptx.cuh"

namespace ll {

namespace {

// Eight consecutive values as four fp32 pairs (packed arithmetic, ptx::mul2 and so on).
struct F8 {
  float2 v[4];
};
using ptx::add2;
using ptx::fma2;
using ptx::mul2;
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
__device__ __forceinline__ F8 fill8(float c) { return {{pair(c), pair(c), pair(c), pair(c)}}; }
// The same as they lie in memory: kept so until they are used.
struct RawF {
  float4 a, b;
};
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  using type = RawF;
};
template <>
struct Raw<__nv_bfloat16> {
  using type = uint4;
};
__device__ __forceinline__ F8 unpack8(const uint4& x) {
  F8 r;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return r;
}
__device__ __forceinline__ F8 unpack8(const RawF& x) {
  return {{make_float2(x.a.x, x.a.y), make_float2(x.a.z, x.a.w), make_float2(x.b.x, x.b.y), make_float2(x.b.z, x.b.w)}};
}
__device__ __forceinline__ uint4 raw8(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ RawF raw8(const float* p) {
  return {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
}
template <typename T>
__device__ __forceinline__ F8 load8(const T* p) {
  return unpack8(raw8(p));
}
__device__ __forceinline__ void store8(float* p, const F8& x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
}
__device__ __forceinline__ uint32_t pack2(float2 a) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x.v[0]), pack2(x.v[1]), pack2(x.v[2]), pack2(x.v[3]));
}
// The eight columns of a thread's vector: side by side, or where rows are not whole vectors
// (D no multiple of 8, so that they start anywhere) `step` apart, so that the threads of a row
// read neighbours; those from D on are 0.
template <bool kOdd>
struct Eight {
  int c, step, D;
  __device__ __forceinline__ Eight(int i, int t, int tpr, int D) : c(kOdd ? i * 8 * tpr + t : (i * tpr + t) * 8), step(tpr), D(D) {}
  __device__ __forceinline__ bool any() const { return c < D; }
  __device__ __forceinline__ uint4 raw(const __nv_bfloat16* p) const {
    if constexpr (!kOdd) {
      return raw8(p + c);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p) + c + 2 * e * step;
        const uint32_t lo = c + 2 * e * step < D ? q[0] : 0u, hi = c + (2 * e + 1) * step < D ? q[step] : 0u;
        w[e] = lo | hi << 16;
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ RawF raw(const float* p) const {
    if constexpr (!kOdd) {
      return raw8(p + c);
    } else {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = c + e * step < D ? p[c + e * step] : 0.f;
      return {make_float4(w[0], w[1], w[2], w[3]), make_float4(w[4], w[5], w[6], w[7])};
    }
  }
  template <typename T>
  __device__ __forceinline__ F8 load(const T* p) const {
    return unpack8(raw(p));
  }
  __device__ __forceinline__ F8 weight(const float* w) const { return w ? load(w) : fill8(1.f); }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const F8& x) const {
    if constexpr (!kOdd) {
      store8(p + c, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e * step < D) ll_store(p, c + e * step, e & 1 ? x.v[e >> 1].y : x.v[e >> 1].x);
    }
  }
};
__device__ __forceinline__ float sum8(const F8& x) {
  const float2 s = add2(add2(x.v[0], x.v[1]), add2(x.v[2], x.v[3]));
  return s.x + s.y;
}

// 1 / (1 + e^-x) for a pair: one exp2 and one reciprocal each.  The exponent's rounding, half a
// unit of x log2(e), is the result's relative error where e^-x is large: measured 2.5 x 2^-23
// from -5 up, 8 down to -15, 15 to -30, 32 to -87; in absolute terms below 2^-23 everywhere.  e^-x
// may reach infinity, whose reciprocal is 0.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 t = mul2(x, pair(-1.4426950408889634f));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = add2(e, pair(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return r;
}
// The gate's activation, fixed at compile time: kNoGate for a norm without one.
constexpr int kNoGate = -1;
template <int kAct>
__device__ __forceinline__ float2 act_of2(float2 g) {
  if (kAct == BN_IDENTITY) return g;
  const float2 s = sigmoid2(g);
  return kAct == BN_SILU ? mul2(g, s) : s;
}
// act(g) and its derivative
template <int kAct>
__device__ __forceinline__ void act_grad2(float2 g, float2& a, float2& d) {
  if (kAct == BN_IDENTITY) {
    a = g;
    d = pair(1.f);
    return;
  }
  const float2 s = sigmoid2(g), q = fma2(s, pair(-1.f), pair(1.f));
  if (kAct == BN_SILU) {
    a = mul2(g, s);
    d = fma2(a, q, s);  // s + g s (1 - s)
  } else {
    a = s;
    d = mul2(s, q);
  }
}
__device__ __forceinline__ float act_of(int act, float g) {
  const float2 x = make_float2(g, 0.f);
  return act == BN_SILU ? act_of2<BN_SILU>(x).x : act == BN_SIGMOID ? act_of2<BN_SIGMOID>(x).x : g;
}
__device__ __forceinline__ float2 act_grad(int act, float g) {
  float2 a, d;
  if (act == BN_SILU) act_grad2<BN_SILU>(make_float2(g, 0.f), a, d);
  else if (act == BN_SIGMOID) act_grad2<BN_SIGMOID>(make_float2(g, 0.f), a, d);
  else act_grad2<BN_IDENTITY>(make_float2(g, 0.f), a, d);
  return make_float2(a.x, d.x);
}

// Sum over the aligned groups of `width` lanes (a power of two) that hold a value each.
__device__ __forceinline__ float lanes_sum(float x, int width) {
  for (int o = width >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Sums over the tpr threads of a row (tpr a power of two >= 32, rows aligned in the CTA).
// `red` holds K floats a warp; the caller lets a barrier pass before using it again.
template <int K>
__device__ __forceinline__ void row_sum(float (&x)[K], int tpr, float* red) {
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = lanes_sum(x[k], 32);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, n = tpr >> 5, w0 = warp & ~(n - 1);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) red[warp * K + k] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float s = 0.f;
    for (int w = 0; w < n; ++w) s += red[(w0 + w) * K + k];
    x[k] = s;
  }
}

// ---------------------------------------------------------------------------------
// bn_fwd: up to 512 threads a row, each with NV vectors of 8 values that stay in registers
// between the two norms, so nothing is read twice.  Small rows share a CTA.  gl: lanes per
// group of y's norm, 0: the whole row (kOdd: D is no multiple of 8).
// ---------------------------------------------------------------------------------
template <typename T, int NV, int kAct, bool kOdd>
__global__ void __launch_bounds__(512) bn_fwd_kernel(const __grid_constant__ BnArgs p, int tpr, int gl) {
  using R8 = typename Raw<T>::type;
  __shared__ float red1[16], red2[16];
  const int t = threadIdx.x & (tpr - 1);
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < p.rows;
  const size_t base = (size_t)row * p.D;
  const T* X = static_cast<const T*>(p.x);
  const T* Y = static_cast<const T*>(p.y);
  const T* Gt = static_cast<const T*>(p.gate);
  R8 yr[NV], xr[NV], gr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Eight<kOdd> c(i, t, tpr, p.D);
    const bool on = live && c.any();
    yr[i] = on && Y ? c.raw(Y + base) : R8{};
    xr[i] = on && X ? c.raw(X + base) : R8{};
    gr[i] = on && kAct != kNoGate ? c.raw(Gt + base) : R8{};
  }
  F8 x[NV];
  if (Y) {
    float ss[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      F8 y = unpack8(yr[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) y.v[e] = mul2(y.v[e], y.v[e]);
      ss[i] = sum8(y);
    }
    if (gl) {
#pragma unroll
      for (int i = 0; i < NV; ++i) ss[i] = lanes_sum(ss[i], gl);
    } else {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) s[0] += ss[i];
      row_sum(s, tpr, red1);
#pragma unroll
      for (int i = 0; i < NV; ++i) ss[i] = s[0];
    }
    T* XN = static_cast<T*>(p.x_new);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Eight<kOdd> c(i, t, tpr, p.D);
      x[i] = unpack8(xr[i]);
      if (!live || !c.any()) continue;
      const float r = rsqrtf(ss[i] * p.inv_group + p.eps);
      const F8 w = c.weight(p.w_post), sc = c.weight(p.scale), y = unpack8(yr[i]), g = unpack8(gr[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 m = mul2(mul2(y.v[e], pair(r)), w.v[e]);
        if (kAct != kNoGate) m = mul2(m, act_of2<kAct>(g.v[e]));
        x[i].v[e] = fma2(sc.v[e], m, x[i].v[e]);
      }
      c.store(XN + base, x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = unpack8(xr[i]);
  }
  if (!p.h) return;
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    F8 q;
#pragma unroll
    for (int e = 0; e < 4; ++e) q.v[e] = mul2(x[i].v[e], x[i].v[e]);
    s[0] += sum8(q);
  }
  row_sum(s, tpr, red2);
  const float r = rsqrtf(s[0] * p.inv_D + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Eight<kOdd> c(i, t, tpr, p.D);
    if (!live || !c.any()) continue;
    const F8 w = c.weight(p.w_pre);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i].v[e] = mul2(mul2(x[i].v[e], pair(r)), w.v[e]);
    c.store(static_cast<T*>(p.h) + base, x[i]);
  }
}

// ---------------------------------------------------------------------------------
// bn_bwd: persistent CTAs, two per SM (one for rows that need 512 threads), blockDim / tpr
// rows at a time.  Rows are contiguous, so a step's rows of each input are one bulk copy
// into a ring of stages in shared memory; the reductions of one step overlap the copies of
// the next ones and the other CTA's arithmetic.  The weights' gradients stay in registers
// over a CTA's rows and go out once, the row slots combined in shared memory; bn_reduce adds
// the CTAs' partials in order.  Rows that are not whole vectors (kOdd) cannot be copied that
// way: they are read where they lie, the second and third time from L1 (37317 rows of 222 in
// bf16: 94 us, of which memory needs 20; value by value with a CTA per row 489).
// ---------------------------------------------------------------------------------
constexpr int kBwdMaxT = 512;
constexpr int kBwdMaxStages = 8;

// Which arguments there are, where that is known at compile time: all of them (the joint
// between two blocks), or dx_new, y and w_post alone (a norm per head, with or without a
// gate).  kAny looks at the pointers, for every other combination.
enum { kJoint, kHeads, kAny };

template <typename T, int NV, int kAct, int kArgs, bool kOdd>
__global__ void __launch_bounds__(kBwdMaxT) bn_bwd_kernel(const __grid_constant__ BnArgs p, int tpr, int gl, int stages) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(8) uint64_t full[kBwdMaxStages];
  ptx::launch_dependents();
  __shared__ float red1[3 * (kBwdMaxT / 32)], red2[kBwdMaxT / 32];
  const int tid = threadIdx.x, t = tid & (tpr - 1), slot = tid / tpr, R = blockDim.x / tpr;
  const T* in[5] = {static_cast<const T*>(p.dh), static_cast<const T*>(p.x), static_cast<const T*>(p.dx_new),
                    static_cast<const T*>(p.y), static_cast<const T*>(p.gate)};
  const bool has_pre = kArgs == kAny ? p.dh != nullptr : kArgs == kJoint;
  const bool has_dxn = kArgs != kAny || p.dx_new, has_y = kArgs != kAny || p.y;
  const bool has_dx = kArgs == kAny ? p.dx != nullptr : kArgs == kJoint;
  using C8 = Eight<kOdd>;
  auto w_pre = [&](const C8& c) { return kArgs == kJoint ? c.load(p.w_pre) : c.weight(p.w_pre); };
  auto w_post = [&](const C8& c) { return kArgs != kAny ? c.load(p.w_post) : c.weight(p.w_post); };
  auto scale = [&](const C8& c) {
    return kArgs == kJoint ? c.load(p.scale) : kArgs == kHeads ? fill8(1.f) : c.weight(p.scale);
  };
  const size_t arr = (size_t)R * p.D * sizeof(T);  // one array of a stage
  int nin = 0, at[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) at[k] = in[k] ? nin++ : 0;
  const long long steps = (p.rows + R - 1) / R;
  auto load = [&](long long step, int st) {
    const long long r0 = step * R;
    const int n = (int)(p.rows - r0 < R ? p.rows - r0 : R);
    const uint32_t bytes = (uint32_t)(n * (size_t)p.D * sizeof(T));
    ptx::mbar_arrive_expect_tx(&full[st], bytes * nin);
#pragma unroll
    for (int k = 0; k < 5; ++k)
      if (in[k]) ptx::bulk_load(sm + ((size_t)st * nin + at[k]) * arr, in[k] + (size_t)r0 * p.D, bytes, &full[st]);
  };
  if (!kOdd && tid == 0) {
    for (int i = 0; i < stages; ++i) ptx::mbar_init(&full[i], 1);
    ptx::fence_mbar_init();
    for (int i = 0; i < stages; ++i)
      if ((long long)blockIdx.x + (long long)i * gridDim.x < steps)
        load((long long)blockIdx.x + (long long)i * gridDim.x, i);
  }
  __syncthreads();
  F8 apre[NV], apost[NV], ascale[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) apre[i] = apost[i] = ascale[i] = fill8(0.f);
  long long it = 0;
  for (long long step = blockIdx.x; step < steps; step += gridDim.x, ++it) {
    const int st = kOdd ? 0 : (int)(it % stages);
    const long long row = step * R + slot;
    const bool live = row < p.rows;
    if (!kOdd) {
      bool ok = bn_wait(&full[st], (uint32_t)(it / stages) & 1);
      if (!ok) atomicExch(p.status, (unsigned)LL_ERR_TIMEOUT);
      if (!__syncthreads_and(ok)) {
        if (tid == 0)  // let the other copies in flight land (bounded)
          for (int i = 0; i < stages; ++i) bn_wait(&full[i], (uint32_t)((it + (i - st + stages) % stages) / stages) & 1);
        return;
      }
    }
    const T* a = reinterpret_cast<const T*>(sm + (size_t)st * nin * arr) + (size_t)slot * p.D;
    const size_t arre = arr / sizeof(T);
    const size_t here = (size_t)row * p.D;
    const T *aH = kOdd ? in[0] + here : a + at[0] * arre, *aX = kOdd ? in[1] + here : a + at[1] * arre,
            *aD = kOdd ? in[2] + here : a + at[2] * arre, *aY = kOdd ? in[3] + here : a + at[3] * arre,
            *aG = kOdd ? in[4] + here : a + at[4] * arre;
    float s3[3] = {0.f, 0.f, 0.f}, sg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const C8 c(i, t, tpr, p.D);
      sg[i] = 0.f;
      if (!live || !c.any()) continue;
      if (has_pre) {
        const F8 x = c.load(aX), dh = c.load(aH), w = w_pre(c);
        float2 xx = mul2(x.v[0], x.v[0]), ux = mul2(mul2(dh.v[0], w.v[0]), x.v[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          xx = fma2(x.v[e], x.v[e], xx);
          ux = fma2(mul2(dh.v[e], w.v[e]), x.v[e], ux);
        }
        s3[0] += xx.x + xx.y;
        s3[1] += ux.x + ux.y;
      }
      if (has_y) {
        const F8 y = c.load(aY);
        float2 yy = mul2(y.v[0], y.v[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) yy = fma2(y.v[e], y.v[e], yy);
        sg[i] = yy.x + yy.y;
        s3[2] += sg[i];
      }
    }
    if (gl) {
#pragma unroll
      for (int i = 0; i < NV; ++i) sg[i] = lanes_sum(sg[i], gl);
    }
    row_sum(s3, tpr, red1);
    const float r2 = rsqrtf(s3[0] * p.inv_D + p.eps), c2 = -(r2 * s3[1] * p.inv_D) * r2;
    float se[NV], r1[NV];
    F8 un[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const C8 c(i, t, tpr, p.D);
      se[i] = 0.f;
      r1[i] = rsqrtf((gl ? sg[i] : s3[2]) * p.inv_group + p.eps);
      un[i] = fill8(0.f);
      if (!live || !c.any()) continue;
      F8 dx = has_dxn ? c.load(aD) : fill8(0.f);
      if (has_pre) {
        const F8 x = c.load(aX), dh = c.load(aH), w = w_pre(c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 xn = mul2(x.v[e], pair(r2));
          apre[i].v[e] = fma2(dh.v[e], xn, apre[i].v[e]);
          dx.v[e] = fma2(mul2(dh.v[e], pair(r2)), w.v[e], fma2(xn, pair(c2), dx.v[e]));
        }
      }
      if (has_dx) c.store(static_cast<T*>(p.dx) + here, dx);
      if (has_y) {
        const F8 w = w_post(c), sc = scale(c), y = c.load(aY);
        F8 dg;
        const F8 g = kAct != kNoGate ? c.load(aG) : fill8(0.f);
        float2 s = pair(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 yn = mul2(y.v[e], pair(r1[i])), n = mul2(yn, w.v[e]);
          float2 dn = mul2(dx.v[e], sc.v[e]);
          if (kAct != kNoGate) {
            float2 av, ad;
            act_grad2<kAct>(g.v[e], av, ad);
            if (kArgs != kHeads) ascale[i].v[e] = fma2(mul2(dx.v[e], av), n, ascale[i].v[e]);
            dg.v[e] = mul2(mul2(dn, n), ad);
            dn = mul2(dn, av);
          } else {
            if (kArgs != kHeads) ascale[i].v[e] = fma2(dx.v[e], n, ascale[i].v[e]);
          }
          apost[i].v[e] = fma2(dn, yn, apost[i].v[e]);
          un[i].v[e] = mul2(dn, w.v[e]);
          s = fma2(un[i].v[e], yn, s);
        }
        se[i] = s.x + s.y;
        if (kAct != kNoGate) c.store(static_cast<T*>(p.dgate) + here, dg);
      }
    }
    if (gl) {
#pragma unroll
      for (int i = 0; i < NV; ++i) se[i] = lanes_sum(se[i], gl);
    } else {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) s[0] += se[i];
      row_sum(s, tpr, red2);
#pragma unroll
      for (int i = 0; i < NV; ++i) se[i] = s[0];
    }
    if (has_y) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const C8 c(i, t, tpr, p.D);
        if (!live || !c.any()) continue;
        const float k = -r1[i] * se[i] * p.inv_group;
        const F8 y = c.load(aY);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          un[i].v[e] = fma2(mul2(y.v[e], pair(r1[i])), pair(k), mul2(un[i].v[e], pair(r1[i])));
        c.store(static_cast<T*>(p.dy) + here, un[i]);
      }
    }
    __syncthreads();  // every thread has read the stage (and red1, red2)
    if (!kOdd && tid == 0 && step + (long long)stages * gridDim.x < steps) load(step + (long long)stages * gridDim.x, st);
  }
  // partial sums of this CTA, the row slots combined in slot order
  const bool asked[3] = {p.dw_pre != nullptr, p.dw_post != nullptr, p.dscale != nullptr};
  float* part = p.part + (size_t)blockIdx.x * 3 * p.D;
  float* acc = reinterpret_cast<float*>(sm);  // 3 x D: the ring is free (every copy was waited for)
  for (int s = 0; s < R; ++s) {
    __syncthreads();
    if (slot != s) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const C8 c(i, t, tpr, p.D);
      if (!c.any()) continue;
      const F8* from[3] = {&apre[i], &apost[i], &ascale[i]};
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (!asked[k]) continue;
        F8 x = *from[k];
        if (s) {
          const F8 y = c.load(acc + k * p.D);
#pragma unroll
          for (int e = 0; e < 4; ++e) x.v[e] = add2(y.v[e], x.v[e]);
        }
        c.store(acc + k * p.D, x);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (asked[k])
      for (int c = tid; c < p.D; c += blockDim.x) part[k * p.D + c] = acc[k * p.D + c];
}

// Sums of the CTAs' partials, in order: 32 columns x 32 slices of the parts per CTA, so that
// a thread's few loads are in flight at once.  blockIdx.y counts the gradients asked for.
constexpr int kSlices = 32;
constexpr int kPerSlice = (kBnMaxParts + kSlices - 1) / kSlices;
__global__ void __launch_bounds__(32 * kSlices) bn_reduce_kernel(const __grid_constant__ BnArgs p, int nparts) {
  __shared__ float red[kSlices][33];
  float* const outs[3] = {p.dw_pre, p.dw_post, p.dscale};
  int which = -1;
  for (int i = 0, n = (int)blockIdx.y; i < 3; ++i)
    if (outs[i] && n-- == 0) which = i;
  ptx::wait_for_prerequisites();  // launched while the partials are still being made
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int per = (nparts + kSlices - 1) / kSlices, p0 = sl * per;
  float x[kPerSlice], s = 0.f;
#pragma unroll
  for (int i = 0; i < kPerSlice; ++i)
    x[i] = c < p.D && i < per && p0 + i < nparts ? p.part[((size_t)(p0 + i) * 3 + which) * p.D + c] : 0.f;
#pragma unroll
  for (int i = 0; i < kPerSlice; ++i) s += x[i];
  red[sl][lane] = s;
  __syncthreads();
  if (sl == 0 && c < p.D) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s += red[i][lane];
    outs[which][c] = s;
  }
}

// ---------------------------------------------------------------------------------
// Any D up to kBnMaxD and any group that divides it, for the groups that are neither the row
// nor whole vectors of a power of two, and those of one value: a CTA per row, values one by
// one.  The rsqrt of each group stays in shared memory; inputs are read again for each step
// (from L1 or L2).
// ---------------------------------------------------------------------------------
constexpr int kAnyT = 256;

__device__ __forceinline__ float block_sum(float x, float* red) {
  x = lanes_sum(x, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kAnyT / 32; ++w) s += red[w];
  return s;
}
// out[k] = sum over group k of f(column), for every group of the row: by the whole CTA for
// one group, else a warp per group.
template <typename F>
__device__ __forceinline__ void group_sums(int D, int group, float* out, float* red, F f) {
  const int n = D / group;
  if (n == 1) {
    float s = 0.f;
    for (int c = threadIdx.x; c < D; c += kAnyT) s += f(c);
    s = block_sum(s, red);
    if (threadIdx.x == 0) out[0] = s;
  } else {
    for (int k = threadIdx.x >> 5; k < n; k += kAnyT / 32) {
      float s = 0.f;
      for (int c = threadIdx.x & 31; c < group; c += 32) s += f(k * group + c);
      s = lanes_sum(s, 32);
      if ((threadIdx.x & 31) == 0) out[k] = s;
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kAnyT) bn_fwd_any_kernel(const __grid_constant__ BnArgs p) {
  extern __shared__ float s_grp[];
  __shared__ float red[kAnyT / 32];
  const size_t base = (size_t)blockIdx.x * p.D;
  const T *X = static_cast<const T*>(p.x), *Y = static_cast<const T*>(p.y), *Gt = static_cast<const T*>(p.gate);
  if (Y)
    group_sums(p.D, p.group, s_grp, red, [&](int c) {
      const float y = ll_load(Y, base + c);
      return y * y;
    });
  auto value = [&](int c) {
    float x = X ? ll_load(X, base + c) : 0.f;
    if (Y) {
      float m = ll_load(Y, base + c) * rsqrtf(s_grp[c / p.group] * p.inv_group + p.eps);
      if (p.w_post) m *= p.w_post[c];
      if (Gt) m *= act_of(p.act, ll_load(Gt, base + c));
      x += p.scale ? p.scale[c] * m : m;
    }
    return x;
  };
  float s = 0.f;
  // x' may be written over x or y only after h has been formed: the values are read again
  for (int c = threadIdx.x; c < p.D; c += kAnyT) {
    const float x = value(c);
    s += x * x;
  }
  s = block_sum(s, red);
  const float r = rsqrtf(s * p.inv_D + p.eps);
  for (int c = threadIdx.x; c < p.D; c += kAnyT) {
    const float x = value(c);
    if (Y) ll_store(static_cast<T*>(p.x_new), base + c, x);
    if (p.h) ll_store(static_cast<T*>(p.h), base + c, p.w_pre ? x * r * p.w_pre[c] : x * r);
  }
}

template <typename T>
__global__ void __launch_bounds__(kAnyT) bn_bwd_any_kernel(const __grid_constant__ BnArgs p) {
  extern __shared__ float s_dyn[];
  __shared__ float red[kAnyT / 32];
  const int ng = p.D / p.group;
  float *acc = s_dyn;                       // 3 x D weight gradients of this CTA's rows
  float *s_y = acc + 3 * p.D, *s_e = s_y + ng;  // per group: sum y², sum un y
  const T *H = static_cast<const T*>(p.dh), *X = static_cast<const T*>(p.x), *Dn = static_cast<const T*>(p.dx_new),
          *Y = static_cast<const T*>(p.y), *Gt = static_cast<const T*>(p.gate);
  for (int c = threadIdx.x; c < 3 * p.D; c += kAnyT) acc[c] = 0.f;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const size_t base = (size_t)row * p.D;
    __syncthreads();
    float a = 0.f, b = 0.f;
    if (H)
      for (int c = threadIdx.x; c < p.D; c += kAnyT) {
        const float x = ll_load(X, base + c), u = ll_load(H, base + c) * (p.w_pre ? p.w_pre[c] : 1.f);
        a += x * x;
        b += u * x;
      }
    a = block_sum(a, red);
    b = block_sum(b, red);
    const float r2 = rsqrtf(a * p.inv_D + p.eps), c2 = r2 * b * p.inv_D;
    if (Y)
      group_sums(p.D, p.group, s_y, red, [&](int c) {
        const float y = ll_load(Y, base + c);
        return y * y;
      });
    auto dx_of = [&](int c) {
      float dx = Dn ? ll_load(Dn, base + c) : 0.f;
      if (H) {
        const float u = ll_load(H, base + c) * (p.w_pre ? p.w_pre[c] : 1.f);
        // a single value: the two terms are equal but for eps, which is all that is left
        dx += p.D == 1 ? r2 * p.eps * r2 * (r2 * u) : r2 * (u - ll_load(X, base + c) * r2 * c2);
      }
      return dx;
    };
    auto un_of = [&](int c) {
      float d = dx_of(c) * (p.scale ? p.scale[c] : 1.f);
      if (Gt) d *= act_of(p.act, ll_load(Gt, base + c));
      return p.w_post ? d * p.w_post[c] : d;
    };
    if (Y) group_sums(p.D, p.group, s_e, red, [&](int c) { return un_of(c) * ll_load(Y, base + c); });
    for (int c = threadIdx.x; c < p.D; c += kAnyT) {
      const float dx = dx_of(c);
      if (H) acc[c] += ll_load(H, base + c) * (ll_load(X, base + c) * r2);
      float dy = 0.f, dg = 0.f;
      if (Y) {
        const int k = c / p.group;
        const float r1 = rsqrtf(s_y[k] * p.inv_group + p.eps), y = ll_load(Y, base + c), yn = y * r1;
        const float n = p.w_post ? yn * p.w_post[c] : yn;
        const float2 ac = Gt ? act_grad(p.act, ll_load(Gt, base + c)) : make_float2(1.f, 0.f);
        const float dm = p.scale ? dx * p.scale[c] : dx;
        acc[p.D + c] += dm * ac.x * yn;
        acc[2 * p.D + c] += dx * ac.x * n;
        dg = dm * n * ac.y;
        dy = p.group == 1 ? r1 * p.eps * r1 * (r1 * un_of(c)) : r1 * (un_of(c) - yn * (r1 * s_e[k] * p.inv_group));
      }
      if (p.dx) ll_store(static_cast<T*>(p.dx), base + c, dx);
      if (Gt) ll_store(static_cast<T*>(p.dgate), base + c, dg);
      if (Y) ll_store(static_cast<T*>(p.dy), base + c, dy);
    }
  }
  __syncthreads();
  float* part = p.part + (size_t)blockIdx.x * 3 * p.D;
  for (int c = threadIdx.x; c < 3 * p.D; c += kAnyT) part[c] = acc[c];
}

int ceil_pow2(int x) {
  int r = 1;
  while (r < x) r <<= 1;
  return r;
}
// Lanes per group of y's norm when groups lie inside a warp's vectors; 0: the whole row is
// one group; -1: neither.
int group_lanes(const BnArgs& p) {
  if (p.D == 1 || (p.y && p.group == 1)) return -1;  // the gradient of one value alone has its own form
  if (!p.y || p.group == p.D) return 0;
  const int n = p.group / 8;
  return p.group % 8 == 0 && n <= 32 && (n & (n - 1)) == 0 ? n : -1;
}

template <int N>
struct Int {
  static constexpr int value = N;
};
// f(Int<the gate's activation>)
template <typename F>
void with_act(const BnArgs& p, F f) {
  if (!p.gate) f(Int<kNoGate>());
  else if (p.act == BN_SILU) f(Int<BN_SILU>());
  else if (p.act == BN_SIGMOID) f(Int<BN_SIGMOID>());
  else f(Int<BN_IDENTITY>());
}

template <typename T>
cudaError_t fwd(const BnArgs& p, cudaStream_t st) {
  const int gl = group_lanes(p), nvec = (p.D + 7) / 8;
  if (gl < 0) {
    const int smem = p.y ? p.D / p.group * 4 : 0;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(bn_fwd_any_kernel<T>, kBnMaxGroups * 4);
    if (e != cudaSuccess) return e;
    bn_fwd_any_kernel<T><<<(unsigned)p.rows, kAnyT, smem, st>>>(p);
    return cudaGetLastError();
  }
  // With many rows, four vectors a thread (two in fp32): fewer threads a row, more rows on
  // an SM at a time.  With few, one, for the shortest way through a row, and where rows are not
  // whole vectors, for their single loads (20000 rows of 1119 in bf16: 143 us with one, 190
  // with four; 37317 of 222: 33 us, of which memory needs 12).
  int nv = p.D % 8 == 0 && p.rows >= 4 * 152 && nvec >= 64 ? (sizeof(T) == 2 && nvec >= 128 ? 4 : 2) : 1;
  while (nvec > 512 * nv) nv *= 2;
  int tpr = ceil_pow2((nvec + nv - 1) / nv);
  tpr = tpr < 32 ? 32 : tpr;
  const int threads = tpr < 128 ? 128 : tpr, R = threads / tpr;
  const unsigned grid = (unsigned)((p.rows + R - 1) / R);
  with_act(p, [&](auto act) {
    constexpr int kAct = decltype(act)::value;
    auto launch = [&](auto odd) {
      constexpr bool kOdd = decltype(odd)::value;
      if (nv == 1) bn_fwd_kernel<T, 1, kAct, kOdd><<<grid, threads, 0, st>>>(p, tpr, gl);
      else if (nv == 2) bn_fwd_kernel<T, 2, kAct, kOdd><<<grid, threads, 0, st>>>(p, tpr, gl);
      else bn_fwd_kernel<T, 4, kAct, kOdd><<<grid, threads, 0, st>>>(p, tpr, gl);
    };
    if (p.D % 8) launch(Int<1>());
    else launch(Int<0>());
  });
  return cudaGetLastError();
}

template <typename T, int NV>
cudaError_t bwd_fast(const BnArgs& p, const BnBwdPlan& pl, int gl, cudaStream_t st) {
  const int nin = (p.dh ? 2 : 0) + (p.dx_new ? 1 : 0) + (p.y ? 1 : 0) + (p.gate ? 1 : 0);
  const size_t stage = (size_t)nin * (pl.threads / pl.tpr) * p.D * sizeof(T), acc = (size_t)3 * p.D * 4;
  const bool odd = p.D % 8 != 0;
  int stages = odd ? 0 : (int)((size_t)pl.smem / stage);
  stages = stages > kBwdMaxStages ? kBwdMaxStages : stages;
  const size_t smem = stage * stages > acc ? stage * stages : acc;
  const bool base = p.dx_new && p.y && p.w_post;
  const int args = base && p.dh && p.w_pre && p.scale && p.dx ? kJoint : base && !p.dh && !p.scale && !p.dx ? kHeads : kAny;
  cudaError_t e = cudaSuccess;
  with_act(p, [&](auto act) {
    constexpr int kAct = decltype(act)::value;
    auto launch = [&](auto kernel, SmemLimit& limit) {
      if ((e = limit.raise(kernel, kBnBwdSmem)) != cudaSuccess) return;
      kernel<<<pl.ctas, pl.threads, smem, st>>>(p, pl.tpr, gl, stages);
      e = cudaGetLastError();
    };
    static SmemLimit limits[4];
    if (odd) return launch(bn_bwd_kernel<T, NV, kAct, kAny, true>, limits[3]);
    if constexpr (kAct == kNoGate || kAct == BN_SILU) {  // the activations in use have their own kernels
      if (args == kJoint) return launch(bn_bwd_kernel<T, NV, kAct, kJoint, false>, limits[0]);
      if (args == kHeads) return launch(bn_bwd_kernel<T, NV, kAct, kHeads, false>, limits[1]);
    }
    launch(bn_bwd_kernel<T, NV, kAct, kAny, false>, limits[2]);
  });
  return e;
}

template <typename T>
cudaError_t bwd(const BnArgs& p, cudaStream_t st) {
  const int gl = group_lanes(p);
  const BnBwdPlan pl = bn_bwd_plan(p, sizeof(T) == 2);
  cudaError_t e;
  if (!pl.fast) {
    const int smem = (3 * p.D + 2 * (p.D / p.group)) * 4;
    static SmemLimit limit;
    e = limit.raise(bn_bwd_any_kernel<T>, (3 * kBnMaxD + 2 * kBnMaxGroups) * 4);
    if (e != cudaSuccess) return e;
    bn_bwd_any_kernel<T><<<pl.ctas, kAnyT, smem, st>>>(p);
    e = cudaGetLastError();
  } else {
    e = pl.nv == 1 ? bwd_fast<T, 1>(p, pl, gl, st) : bwd_fast<T, 2>(p, pl, gl, st);
  }
  if (e != cudaSuccess) return e;
  note_launch();
  if (p.dw_pre || p.dw_post || p.dscale) {
    const int outs = (p.dw_pre ? 1 : 0) + (p.dw_post ? 1 : 0) + (p.dscale ? 1 : 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.D + 31) / 32, outs);
    cfg.blockDim = dim3(32 * kSlices);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, bn_reduce_kernel, p, pl.ctas)) != cudaSuccess) return e;
    note_launch();
  }
  return cudaSuccess;
}

}  // namespace

// Which backward kernel runs and on how many CTAs (each leaves a partial of the weights'
// gradients in the workspace).
BnBwdPlan bn_bwd_plan(const BnArgs& p, bool bf16) {
  BnBwdPlan pl{};
  const int nvec = (p.D + 7) / 8, e = bf16 ? 2 : 4;
  pl.nv = nvec <= (p.D % 8 ? 256 : 32) ? 1 : 2;
  pl.tpr = ceil_pow2((nvec + pl.nv - 1) / pl.nv);
  pl.tpr = pl.tpr < 32 ? 32 : pl.tpr;
  pl.threads = pl.tpr <= 256 ? 256 : 512;
  // two CTAs an SM where the rows of a step leave room for two of them, else one
  const long long stage = 5LL * (pl.threads / pl.tpr) * p.D * e;
  const int per_sm = pl.threads == 256 && 2 * stage <= kBnBwdSmem ? 2 : 1;
  pl.smem = kBnBwdSmem / per_sm;
  pl.fast = nvec <= 1024 && group_lanes(p) >= 0 && stage <= pl.smem;
  const long long steps = pl.fast ? (p.rows + pl.threads / pl.tpr - 1) / (pl.threads / pl.tpr) : p.rows;
  const int most = pl.fast ? 152 * per_sm : kBnMaxParts;
  pl.ctas = (int)(steps < most ? steps : most);
  return pl;
}

cudaError_t launch_bn_fwd(const BnArgs& p, bool bf16, cudaStream_t st) {
  const cudaError_t e = bf16 ? fwd<__nv_bfloat16>(p, st) : fwd<float>(p, st);
  if (e == cudaSuccess) note_launch();
  return e;
}
cudaError_t launch_bn_bwd(const BnArgs& p, bool bf16, cudaStream_t st) {
  return bf16 ? bwd<__nv_bfloat16>(p, st) : bwd<float>(p, st);
}

}  // namespace ll
