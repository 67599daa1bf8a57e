// Gated recurrence over channels: h_t = a_t h_{t-1} + n(a_t) sigmoid(i_t) x_t with
// a_t = exp(-decay sigmoid(r_t)); the gradients; one token.  Contracts are in include/loglinear.h.
//
// Bytes: 8 a value forward in bf16 (x, r, i in, h out), 16 backward.  Everything is read once.  A unit
// is 64, 32 or 16 channels of a sequence; a cluster of 1 to 8 CTAs walks it in steps, each CTA with a
// run of tokens, a warp's lanes in 1, 2 or 4 groups with 7 to 15 tokens each.  A step's tokens come by
// TMA while the step before is worked on.  Every group makes the map of its tokens, keeping
// (a_t, u_t) in registers; the CTAs write their maps into one another's shared memory; then each knows
// what enters its tokens and the next step, and applies it.
//
// At 4 x 8192 x 2560 139 us forward (4.8 TB/s, 71 % of a copy's rate) and 254 backward (5.3, 78 %), in fp32 222
// and 444 (both 89 %); 100003 tokens of 2048 channels 398 (4.1, 61 %).  What bounds bf16: waiting.  35
// instructions a value forward (77 us of the 139 if they were issued without a pause) on 16 warps an SM,
// the special functions' unit 38 % busy (three exponentials, two reciprocals, a root), and the maps' way round,
// some 1300 cycles a step that only the SM's other CTAs fill.  Rows that are not whole 16 bytes are copied value by
// value between barriers: 4 x 8192 x 2562 706 and 1203 us.  Measured on the way there (the first of these): chunks of a sequence handed on through flags
// in global memory 402 us; clusters with a barrier for every step (it waits for the stores to global
// memory too) and loads into registers 243; tokens by TMA and maps by asynchronous stores 174; four
// CTAs of four warps instead of two of eight 141.  Both sigmoids by one reciprocal of their product
// 152 instead of 155: not worth capped exponents.  Narrower units where channels or units are few:
// 50000 tokens of 64 channels 169 -> 50 us, 26060 of 13 x 24 93 -> 37, the long document 440 -> 398.
#include "gatescan_walk.cuh"

namespace ll {
namespace {

// ---- forward -----------------------------------------------------------------------------
template <typename T, bool kTma, int M, bool kGate, int G>
__global__ void __launch_bounds__(kGsWarps * 32, 4)
    gs_fwd_kernel(const __grid_constant__ GsArgs p, const __grid_constant__ GsMaps<2 + kGate> maps) {
  constexpr int N = 2 + kGate, L = kTokens<T, N, G>;
  extern __shared__ __align__(128) unsigned char raw[];
  Walk<T, N, G, 2> w(*reinterpret_cast<Shared<T, N, G>*>(raw), p);
  const float2 decay = not_below_0(w.pair_of(p.decay, 0));
  float2 carry = w.pair_of(p.state_in, w.b);
  const void* const from[3] = {p.r, p.x, p.i};

  const int stride = (int)w.size * kChunk<T, N, G>;
  int t0 = (int)w.rank * kChunk<T, N, G>;
  if (kTma) {
    w.template fetch<kTma>(maps, from, 0, t0, -1);
    if (w.steps > 1) w.template fetch<kTma>(maps, from, 1, t0 + stride, -1);
  }
  for (int step = 0; step < w.steps; ++step, t0 += stride) {
    const int stage = kTma ? step & 1 : 0, t = t0 + w.group * L, there = w.len - t;
    if (!kTma) w.template fetch<kTma>(maps, from, 0, t0, -1);
    w.template arrived<kTma>(step);
    float2 A = both(0.f), H = both(0.f), a[L], u[L];
#pragma unroll
    for (int k = 0; k < L; ++k) {
      const float2 z = mul2(decay, sigmoid_of(exp_minus<T>(w.token(stage, 0, k))));
      const float2 m = loss_of<T>(z);
      a[k] = kept_of(m);
      u[k] = mixed<M>(m, w.token(stage, 1, k));
      if (kGate) u[k] = mul2(u[k], sigmoid_of(exp_minus<T>(w.token(stage, N - 1, k))));
      A = add2(A, z);
      H = fma2(a[k], H, u[k]);
    }
    if (there < L) {  // past the length the map is the identity
      A = H = both(0.f);
#pragma unroll
      for (int k = 0; k < L; ++k) {
        if (k < there) {
          A = add2(A, mul2(decay, sigmoid_of(exp_minus<T>(w.token(stage, 0, k)))));
        } else {
          a[k] = both(1.f);
          u[k] = both(0.f);
        }
        H = fma2(a[k], H, u[k]);
      }
    }
    // the decay over the group's tokens as one exponential of the sum
    A = exp_minus<float>(A);
    w.s.group[step & 1][threadIdx.x] = make_float4(A.x, A.y, H.x, H.y);
    __syncthreads();
    if (kTma && step + 2 < w.asked) w.template fetch<kTma>(maps, from, stage, t0 + 2 * stride, -1);
    float2 h = w.enter(step, w.group, carry);
    T* out = static_cast<T*>(p.h) + ((size_t)w.b * p.T + t) * p.D + w.c;
    if (there >= L) {
      if (w.c < p.D) {
#pragma unroll
        for (int k = 0; k < L; ++k) {
          h = fma2(a[k], h, u[k]);
          store<T, kTma>(out, h, w.c, p.D);
          out += p.D;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < L; ++k) {
        h = fma2(a[k], h, u[k]);
        if (t + k < p.T && w.c < p.D) store<T, kTma>(out, k < there ? h : both(0.f), w.c, p.D);
        out += p.D;
      }
    }
  }
  w.template leave<kTma>();
  if (p.state_out && w.rank == 0 && w.group == 0) w.put_pair(p.state_out, w.b, carry);
}

// ---- one token ---------------------------------------------------------------------------
template <typename T, bool kPairs, int M, bool kGate>
__global__ void __launch_bounds__(128) gs_step_kernel(GsStepArgs p) {
  using W = typename Pair<T>::type;
  const long long at = ((long long)blockIdx.x * 128 + threadIdx.x) * (kPairs ? 2 : 1);
  if (at >= p.n) return;
  const int c = (int)(at % p.D);
  auto values = [&](const void* x) {
    const T* v = static_cast<const T*>(x) + at;
    return kPairs ? Pair<T>::get(*reinterpret_cast<const W*>(v)) : both((float)*v);
  };
  auto floats = [&](const float* x) { return kPairs ? *reinterpret_cast<const float2*>(x) : both(*x); };
  const float2 st = floats(p.states + at), decay = not_below_0(floats(p.decay + c));
  const float2 m = loss_of<T>(mul2(decay, sigmoid_of(exp_minus<T>(values(p.r)))));
  float2 u = mixed<M>(m, values(p.x));
  if (kGate) u = mul2(u, sigmoid_of(exp_minus<T>(values(p.i))));
  const float2 h = fma2(kept_of(m), st, u);
  if (kPairs) *reinterpret_cast<float2*>(p.states + at) = h;
  else p.states[at] = h.x;
  T* out = static_cast<T*>(p.h) + at;
  if (kPairs) *reinterpret_cast<W*>(out) = Pair<T>::put(h);
  else *out = Pair<T>::one(h.x);
}

template <typename T, bool kTma, int M, bool kGate>
struct Forward {
  static cudaError_t run(GsArgs& p, cudaStream_t st) {
    constexpr int N = 2 + kGate;
    static Room room[3];
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const void* const x[] = {p.r, p.x, p.i};
    Choice c{};
    consider<T, N, 1>(c, gs_fwd_kernel<T, kTma, M, kGate, 1>, p, dev, room[0]);
    if constexpr (kTma) {
      consider<T, N, 2>(c, gs_fwd_kernel<T, kTma, M, kGate, 2>, p, dev, room[1]);
      consider<T, N, 4>(c, gs_fwd_kernel<T, kTma, M, kGate, 4>, p, dev, room[2]);
    }
    if (c.t == 0) return c.why != cudaSuccess ? c.why : cudaErrorInvalidConfiguration;
    if constexpr (kTma) {
      if (c.groups == 2) return launch<T, N, 2>(gs_fwd_kernel<T, kTma, M, kGate, 2>, p, c, x, true, st);
      if (c.groups == 4) return launch<T, N, 4>(gs_fwd_kernel<T, kTma, M, kGate, 4>, p, c, x, true, st);
    }
    return launch<T, N, 1>(gs_fwd_kernel<T, kTma, M, kGate, 1>, p, c, x, kTma, st);
  }
};
template <typename T, bool kPairs, int M, bool kGate>
struct Step {
  static cudaError_t run(const GsStepArgs& p, unsigned grid, cudaStream_t st) {
    gs_step_kernel<T, kPairs, M, kGate><<<grid, 128, 0, st>>>(p);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_gs_fwd(GsArgs p, bool bf16, cudaStream_t st) {
  const cudaError_t e = choose<Forward>(bf16, whole_rows(p.D, bf16), p.mix, p.i != nullptr, [&](auto k) { return k.run(p, st); });
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_gs_step(const GsStepArgs& p, int mix, bool bf16, cudaStream_t st) {
  const int v = p.D % 2 == 0 ? 2 : 1;
  const unsigned grid = (unsigned)((p.n / v + 127) / 128);
  const cudaError_t e = choose<Step>(bf16, v == 2, mix, p.i != nullptr, [&](auto k) { return k.run(p, grid, st); });
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ll
