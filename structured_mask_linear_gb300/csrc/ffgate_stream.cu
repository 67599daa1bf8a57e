// Gated feed-forward block for few rows (single tokens): every weight is read once, straight into
// registers.  Contracts are in include/loglinear.h.
//
// Bound by memory: 2 F D weights, against 2 operations a weight and row.  A CTA has 16 of the F
// columns of both projections and its warps share the sum over D, so that 4 KB a warp, 96 an SM, are
// on their way at a time (two such runs a warp: 1 row of 4096 x 11008 33 us against 28.8).  bf16: mma.sync with 16 columns as its rows and the tokens as its columns
// (what the instruction takes per weight matters here, not its rate: 16 rows are a few per cent of
// what the tensor cores can do).  The summed index is permuted: a lane's 16 bytes are eight
// consecutive values, the operands' four pairs, of weights and tokens alike.  fp32: products and
// sums of fp32, two columns a warp.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ffgate.cuh"
#include "ffgate_act.cuh"

namespace ll {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 16;  // of F, per CTA

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 read(const __nv_bfloat16* row, int k, int D) {
  return k < D ? __ldcs(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ void finish(const FfStream& p, long long row, int f, float g, float u) {
  const long long at = row * p.F + f;
  auto put = [&](void* x, float v) {
    if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(x)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(x)[at] = v;
  };
  put(p.m, ff_act<T>(g, p.act) * u);
  if (p.gate) {
    put(p.gate, g);
    put(p.up, u);
  }
}

// kTiles: of 8 tokens.
template <int kTiles>
__global__ void __launch_bounds__(kWarps * 32, 3) ff_stream_bf16_kernel(FfStream p) {
  __shared__ float4 s_part[kWarps][2][kTiles][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int f0 = blockIdx.x * kCols + g;
  const __nv_bfloat16* w[2][2];  // columns f0 and f0 + 8 of each projection; a column past F reads the first
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long f = f0 + 8 * h < p.F ? f0 + 8 * h : 0;
    w[0][h] = static_cast<const __nv_bfloat16*>(p.w_gate) + f * p.D;
    w[1][h] = static_cast<const __nv_bfloat16*>(p.w_up) + f * p.D;
  }
  float acc[2][kTiles][4];
#pragma unroll
  for (int i = 0; i < 2 * kTiles * 4; ++i) (&acc[0][0][0])[i] = 0.f;
  const __nv_bfloat16* x0 = static_cast<const __nv_bfloat16*>(p.x);

  for (int k0 = warp * 64; k0 < p.D; k0 += kWarps * 64) {
    uint4 a[2][2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[c][i][h] = read(w[i][h], k0 + 32 * c + 8 * t, p.D);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = k0 + 32 * c + 8 * t;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        const int row = 8 * j + g;
        uint4 b = make_uint4(0, 0, 0, 0);
        if (row < p.rows && k < p.D) b = __ldg(reinterpret_cast<const uint4*>(x0 + (long long)row * p.D + k));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma(acc[i][j], a[c][i][0].x, a[c][i][1].x, a[c][i][0].y, a[c][i][1].y, b.x, b.y);
          mma(acc[i][j], a[c][i][0].z, a[c][i][1].z, a[c][i][0].w, a[c][i][1].w, b.z, b.w);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
      s_part[warp][i][j][lane] = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
  __syncthreads();
  // the warps' sums in order; a value is (column g or g + 8, token 8 j + 2 t or the next)
  const float* parts = reinterpret_cast<const float*>(&s_part[0][0][0][0]);
  for (int v = threadIdx.x; v < kTiles * 128; v += kWarps * 32) {
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < kWarps; ++q) sum[i] += parts[((q * 2 + i) * kTiles * 128) + v];
    const int e = v & 3, at = (v >> 2) & 31, j = v >> 7;
    const int f = blockIdx.x * kCols + (at >> 2) + 8 * (e >> 1), row = 8 * j + 2 * (at & 3) + (e & 1);
    if (f < p.F && row < p.rows) finish<__nv_bfloat16>(p, row, f, sum[0], sum[1]);
  }
}

// kRows tokens; a warp has two columns.
template <int kRows>
__global__ void __launch_bounds__(kWarps * 32) ff_stream_f32_kernel(FfStream p) {
  const int lane = threadIdx.x & 31, f0 = blockIdx.x * kCols + 2 * (threadIdx.x >> 5);
  if (f0 >= p.F) return;  // F is even
  const float* w[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[0][h] = static_cast<const float*>(p.w_gate) + (long long)(f0 + h) * p.D;
    w[1][h] = static_cast<const float*>(p.w_up) + (long long)(f0 + h) * p.D;
  }
  float acc[2][2][kRows];
#pragma unroll
  for (int i = 0; i < 4 * kRows; ++i) (&acc[0][0][0])[i] = 0.f;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 4 * lane; k0 < p.D; k0 += 256) {
    float4 a[2][2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          a[c][i][h] = k0 + 128 * c < p.D ? __ldcs(reinterpret_cast<const float4*>(w[i][h] + k0 + 128 * c)) : zero;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float4 b = zero;
        if (r < p.rows && k0 + 128 * c < p.D)
          b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + (long long)r * p.D + k0 + 128 * c));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& s = acc[i][h][r];
            s = fmaf(a[c][i][h].x, b.x, s);
            s = fmaf(a[c][i][h].y, b.y, s);
            s = fmaf(a[c][i][h].z, b.z, s);
            s = fmaf(a[c][i][h].w, b.w, s);
          }
      }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float s[2] = {acc[0][h][r], acc[1][h][r]};
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
        s[1] += __shfl_xor_sync(0xffffffffu, s[1], o);
      }
      if (lane == 0 && r < p.rows) finish<float>(p, r, f0 + h, s[0], s[1]);
    }
}

}  // namespace

cudaError_t launch_ff_stream(const FfStream& p, bool bf16, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.F + kCols - 1) / kCols);
  const int threads = kWarps * 32;
  if (bf16) {
    if (p.rows <= 8) ff_stream_bf16_kernel<1><<<grid, threads, 0, st>>>(p);
    else ff_stream_bf16_kernel<2><<<grid, threads, 0, st>>>(p);
  } else {
    if (p.rows <= 1) ff_stream_f32_kernel<1><<<grid, threads, 0, st>>>(p);
    else if (p.rows <= 2) ff_stream_f32_kernel<2><<<grid, threads, 0, st>>>(p);
    else if (p.rows <= 4) ff_stream_f32_kernel<4><<<grid, threads, 0, st>>>(p);
    else ff_stream_f32_kernel<8><<<grid, threads, 0, st>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ll
