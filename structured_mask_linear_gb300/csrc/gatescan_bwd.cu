// Gated recurrence: the gradients.  Contracts are in include/loglinear.h; how a cluster walks a unit
// stands in gatescan.cu.
#include "gatescan_walk.cuh"

namespace ll {
namespace {

// ---- backward ----------------------------------------------------------------------------
// The adjoint runs the same scan from the last token: with c what comes in from the token after,
// g_t = dh_t + c and a_t g_t goes on: the map (a_t, a_t dh_t).  Chunks and groups are counted from
// the end; the groups of a CTA have their tokens in memory's order all the same.
template <typename T, bool kTma, int M, bool kGate, int G>
__global__ void __launch_bounds__(kGsWarps * 32, sizeof(T) == 2 ? 4 : 2)
    gs_bwd_kernel(const __grid_constant__ GsArgs p, const __grid_constant__ GsMaps<4 + kGate> maps) {
  constexpr int N = 4 + kGate, L = kTokens<T, N, G>;
  extern __shared__ __align__(128) unsigned char raw[];
  Walk<T, N, G, 1> w(*reinterpret_cast<Shared<T, N, G>*>(raw), p);
  const int turn = w.kGroups - 1 - w.group;  // place in the scan
  ptx::griddep_launch_dependents();
  const float2 given = w.pair_of(p.decay, 0), decay = not_below_0(given), minus = mul2(decay, both(-1.f));
  float2 carry = w.pair_of(p.dstate_out, w.b), dsum = both(0.f);
  const void* const from[5] = {p.r, p.dh, p.x, p.h_in, p.i};  // h: of the token before

  const int stride = (int)w.size * kChunk<T, N, G>;
  int t0 = (w.steps * (int)w.size - 1 - (int)w.rank) * kChunk<T, N, G>;
  if (kTma) w.template fetch<kTma>(maps, from, 0, t0, 3);
  for (int step = 0; step < w.steps; ++step, t0 -= stride) {
    const int stage = kTma ? step & 1 : 0, t = t0 + w.group * L, there = w.len - t;
    if (!kTma) {
      __syncthreads();
      w.template fetch<kTma>(maps, from, 0, t0, 3);
    }
    w.template arrived<kTma>(step);
    float2 A = both(0.f), H = both(0.f), e[L], m[L];
#pragma unroll
    for (int k = L - 1; k >= 0; --k) {
      e[k] = exp_minus<T>(w.token(stage, 0, k));
      const float2 z = mul2(decay, sigmoid_of(e[k]));
      m[k] = loss_of<T>(z);
      A = add2(A, z);
      H = mul2(kept_of(m[k]), add2(w.token(stage, 1, k), H));
    }
    if (there < L) {  // past the length the map is the identity
      A = H = both(0.f);
#pragma unroll
      for (int k = L - 1; k >= 0; --k) {
        if (k >= there) continue;
        A = add2(A, mul2(decay, sigmoid_of(e[k])));
        H = mul2(kept_of(m[k]), add2(w.token(stage, 1, k), H));
      }
    }
    A = exp_minus<float>(A);
    w.s.group[step & 1][turn * w.kLanes + w.lane] = make_float4(A.x, A.y, H.x, H.y);
    __syncthreads();
    // the stage of the step before: all have left it
    if (kTma && step + 1 < w.asked) w.template fetch<kTma>(maps, from, stage ^ 1, t0 - stride, 3);
    float2 c = w.enter(step, turn, carry);
    const size_t last = ((size_t)w.b * p.T + t + L - 1) * p.D + w.c;
    T *ox = static_cast<T*>(p.dx) + last, *orr = static_cast<T*>(p.dr) + last, *oi = kGate ? static_cast<T*>(p.di) + last : nullptr;
    // token k's own chain, from g and the state before it
    auto token = [&](int k) {
      const float2 sg = sigmoid_of(e[k]), a = kept_of(m[k]), x = w.token(stage, 2, k);
      const float2 g = add2(w.token(stage, 1, k), c);
      float2 before = w.token(stage, 3, k);
      if (t + k == 0) before = w.pair_of(p.state_in, w.b);
      float2 dla = mul2(a, before);  // of log a, for each of g
      float2 gate = both(1.f), gx = x, di = both(0.f);
      if (kGate) {
        const float2 ei = exp_minus<T>(w.token(stage, N - 1, k));
        gate = sigmoid_of(ei);
        gx = mul2(gate, x);
        di = rest_of(ei, gate);
      }
      // n, and its derivative with respect to log a; where n is 0 it multiplies a sigmoid of 0
      float2 n = both(1.f);
      if (M == kMixLerp) {
        n = m[k];
        dla = fma2(mul2(a, both(-1.f)), gx, dla);
      } else if (M == kMixRms) {
        const float2 n2 = power_of(m[k]), rn = make_float2(inverse_root(n2.x), inverse_root(n2.y));
        n = mul2(n2, rn);
        dla = fma2(mul2(mul2(a, mul2(a, both(-1.f))), rn), gx, dla);
      }
      const float2 gn = mul2(g, n), ds = mul2(mul2(dla, g), sg);
      dsum = fma2(ds, both(-1.f), dsum);
      c = mul2(a, g);
      if (w.c >= p.D) return;
      store<T, kTma>(ox, mul2(gn, gate), w.c, p.D);
      store<T, kTma>(orr, mul2(mul2(ds, minus), rest_of(e[k], sg)), w.c, p.D);
      if (kGate) store<T, kTma>(oi, mul2(mul2(gn, gx), di), w.c, p.D);
    };
    auto down = [&] {
      ox -= p.D;
      orr -= p.D;
      if (kGate) oi -= p.D;
    };
    if (there >= L) {
#pragma unroll
      for (int k = L - 1; k >= 0; --k) {
        token(k);
        down();
      }
    } else {
#pragma unroll
      for (int k = L - 1; k >= 0; --k) {
        if (k < there) {
          token(k);
        } else if (t + k < p.T && w.c < p.D) {
          store<T, kTma>(ox, both(0.f), w.c, p.D);
          store<T, kTma>(orr, both(0.f), w.c, p.D);
          if (kGate) store<T, kTma>(oi, both(0.f), w.c, p.D);
        }
        down();
      }
    }
  }
  w.template leave<kTma>();
  if (p.dstate_in && w.rank == 0 && turn == 0) w.put_pair(p.dstate_in, w.b, carry);
  if (p.part) {
    __syncthreads();
    float2* sums = reinterpret_cast<float2*>(&w.s.group[0][0]);
    sums[turn * w.kLanes + w.lane] = make_float2(given.x < 0.f ? 0.f : dsum.x, given.y < 0.f ? 0.f : dsum.y);
    __syncthreads();
    if (turn == 0) {
      float2 sum = both(0.f);
#pragma unroll
      for (int i = 0; i < w.kGroups; ++i) sum = add2(sum, sums[i * w.kLanes + w.lane]);
      w.put_pair(p.part, (size_t)w.rank * p.B + w.b, sum);
    }
  }
}

// ddecay: the sum over the tiles' partials, in a fixed order.  32 channels by 32 threads each.
__global__ void __launch_bounds__(1024) gs_sum_kernel(const float* part, float* out, long long rows, int D) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  ptx::griddep_wait();
  float acc = 0.f;
  if (c < D)
    for (long long r = w; r < rows; r += 32) acc += part[r * D + c];
  s[w][lane] = acc;
  __syncthreads();
  if (w == 0 && c < D) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) sum += s[k][lane];
    out[c] = sum;
  }
}

template <typename T, bool kTma, int M, bool kGate>
struct Backward {
  static cudaError_t run(GsArgs& p, cudaStream_t st) {
    constexpr int N = 4 + kGate;
    static Room room[3];
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const void* const x[] = {p.r, p.dh, p.x, p.h_in, p.i};
    Choice c{};
    consider<T, N, 1>(c, gs_bwd_kernel<T, kTma, M, kGate, 1>, p, dev, room[0]);
    if constexpr (kTma) {
      consider<T, N, 2>(c, gs_bwd_kernel<T, kTma, M, kGate, 2>, p, dev, room[1]);
      consider<T, N, 4>(c, gs_bwd_kernel<T, kTma, M, kGate, 4>, p, dev, room[2]);
    }
    if (c.t == 0) return c.why != cudaSuccess ? c.why : cudaErrorInvalidConfiguration;
    if constexpr (kTma) {
      if (c.groups == 2) return launch<T, N, 2>(gs_bwd_kernel<T, kTma, M, kGate, 2>, p, c, x, true, st);
      if (c.groups == 4) return launch<T, N, 4>(gs_bwd_kernel<T, kTma, M, kGate, 4>, p, c, x, true, st);
    }
    return launch<T, N, 1>(gs_bwd_kernel<T, kTma, M, kGate, 1>, p, c, x, kTma, st);
  }
};

}  // namespace

cudaError_t launch_gs_bwd(GsArgs p, bool bf16, cudaStream_t st) {
  float* const part = p.part;
  cudaError_t e = choose<Backward>(bf16, whole_rows(p.D, bf16), p.mix, p.i != nullptr, [&](auto k) { return k.run(p, st); });
  if (e != cudaSuccess) return e;
  note_launch();
  if (!p.ddecay || p.part != part) return cudaSuccess;
  e = launch_ahead(gs_sum_kernel, dim3((p.D + 31) / 32), 1024, 0, st, p.part, p.ddecay, (long long)p.cluster * p.B, p.D);
  if (e == cudaSuccess) note_launch();
  return e;
}


}  // namespace ll
