// The gated feed-forward block's activations and their derivatives, in fp32.  T: the type of what comes of
// them, whose steps say how exact the exponentials have to be.
#pragma once

#include <cuda_bf16.h>

#include "../../include/loglinear.h"

namespace ll {

// sigmoid(x), and 1 - sigmoid(x) as exactly: the difference would lose the slope of a gate that is wide open
// (at 10 a thousandth of it, from 17 on all).
struct FfSigmoid {
  float s, rest;
};
__device__ __forceinline__ float ff_reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ FfSigmoid ff_sigmoid(float x) {
  if constexpr (sizeof(T) == 2) {
    // the exponent unit's own, |x| 2^-24 relative: well below a step of bf16
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    const float s = ff_reciprocal(1.f + e);
    return {s, e < 1.f ? e * s : 1.f - s};
  } else {
    const float e = expf(-fabsf(x)), larger = ff_reciprocal(1.f + e), smaller = e * larger;
    return x >= 0.f ? FfSigmoid{larger, smaller} : FfSigmoid{smaller, larger};
  }
}
template <typename T>
__device__ __forceinline__ float ff_act(float x, int act) {
  switch (act) {
    case FF_SILU: return x * ff_sigmoid<T>(x).s;
    case FF_SIGMOID: return ff_sigmoid<T>(x).s;
    case FF_GELU: return 0.5f * x * erfcf(x * -0.70710678118654752f);
    default: return x;
  }
}
// g = act(g) u.  The choice comes first: made for every value among its instructions it took longer than they.
template <typename T, int N>
__device__ __forceinline__ void ff_gated(float* g, const float* u, int act) {
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < N; ++j) g[j] = f(g[j]) * u[j];
  };
  switch (act) {
    case FF_SILU: each([](float x) { return ff_act<T>(x, FF_SILU); }); break;
    case FF_SIGMOID: each([](float x) { return ff_act<T>(x, FF_SIGMOID); }); break;
    case FF_GELU: each([](float x) { return ff_act<T>(x, FF_GELU); }); break;
    default: each([](float x) { return x; });
  }
}
// act(x) and its derivative.
template <typename T>
__device__ __forceinline__ float2 ff_act_and_slope(float x, int act) {
  switch (act) {
    case FF_SILU: {
      const FfSigmoid g = ff_sigmoid<T>(x);
      return make_float2(x * g.s, g.s * fmaf(x, g.rest, 1.f));
    }
    case FF_SIGMOID: {
      const FfSigmoid g = ff_sigmoid<T>(x);
      return make_float2(g.s, g.s * g.rest);
    }
    case FF_GELU: {
      const float c = 0.5f * erfcf(x * -0.70710678118654752f), z = -0.5f * x * x;
      return make_float2(x * c, fmaf(x * 0.3989422804014327f, sizeof(T) == 2 ? __expf(z) : expf(z), c));
    }
    default: return make_float2(x, 1.f);
  }
}

}  // namespace ll
