// Linear attention with one constant decay per head: shared declarations of its kernels.
//
// Every direction is the same scan.  For token vectors X_t, Y_t (width a) and Z_t (width b)
// of a head with decay g = exp(log_a[h]),
//     out_t = X_t . R_t,   R_t = sum over s <= t of g^(t-s) Y_s Z_sᵀ  (+ the decayed start),
// or the same with time reversed.  The forward is (q, k, v); its gradients are
//     dq: (dO, v, k) forwards,   dk: (v, dO, q) backwards,   dv: (k, q, dO) backwards,
// with the start state transposed where X and Z have changed places.
//
// Chunked form over C tokens with i' the index of a token in the scan's own direction, nv
// the number of valid tokens of the chunk and sh = 1 forwards, 0 backwards:
//     out_i = sum over valid pairs in the chunk g^|i-j| (X_i . Y_j) Z_j + g^(i'+sh) X_i R
//     R    <- g^nv R + sum_j g^(nv-sh-j') Y_j Z_jᵀ
// Forwards R is the state after the token before the chunk; backwards it is the state's
// gradient at the last token before the chunk (in scan order) including that token's own
// decay, so that the gradient of the final state enters undecayed and the gradient of the
// first state comes out as R.
#pragma once

#include "ll_internal.cuh"

namespace ll {

constexpr int kLinChunk = 128;  // tokens per chunk of the tensor-core kernels
constexpr int kLinChunk32 = 64; // tokens per chunk of the fp32 kernels
constexpr int kLinTile = 64;    // columns of Z (and out) per unit of work
constexpr int kLinProbs = 3;

// One scan.  Head counts: a tensor with `G` heads is read at h / hpg, one with H heads at h.
// An output with G heads is the sum over the heads of the group.
struct LinProb {
  const void* X;
  const void* Y;
  const void* Z;
  void* out;
  int xh, yh, zh, oh;        // head counts of X, Y, Z, out
  int a, b;                  // widths of X and Y, of Z and out
  int rev;                   // 1: time runs backwards
  const float* init;         // NULL (zero), or start states: element (i, j) of head bh at
  int init_rs, init_cs;      // init[bh * a * b + i * init_rs + j * init_cs]
  float* fin;                // NULL, or end states (B*H, a, b)
  float* seg;                // (B*H, tiles, nseg, a, 64) segment totals, then start states
  int tiles;                 // ceil(b / 64)
  int unit0, sunit0;         // first unit of this scan in the output and the state pass
};

struct LinArgs {
  int B, T, H, hpg;
  int chunk;        // tokens per chunk
  int NC;           // chunks over T
  int nseg, L;      // segments per head, chunks per segment
  int nprob;
  int units, sunits;
  const float* log_a;   // (H)
  const int* lengths;   // NULL or (B)
  float* scratch;       // per CTA: sums over a group's heads, L * 128 * 64 fp32
  unsigned* status;
  LinProb pr[kLinProbs];
};

// log2 of the decay per token.  log_a above 0 counts as 0; below -1000 (where g is 0 in
// fp32) as -1000, so that 0 * log_a stays 0.  NaN stays NaN.
__device__ __forceinline__ float lin_log2_decay(const float* log_a, int h) {
  float x = log_a[h];
  x = x > 0.f ? 0.f : x < -1000.f ? -1000.f : x;
  return x * 1.4426950408889634f;
}
// valid tokens of batch row b
__device__ __forceinline__ int lin_len(const LinArgs& p, int b) {
  if (!p.lengths) return p.T;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.T ? p.T : n;
}

// A unit of work: columns 64 tile .. of out head oh of batch row b over one segment.
struct LinUnit {
  int prob, b, oh, tile, seg;
};
__device__ __forceinline__ LinUnit lin_unit(const LinArgs& p, int u) {
  LinUnit x;
  x.prob = 0;
  while (x.prob + 1 < p.nprob && u >= p.pr[x.prob + 1].unit0) ++x.prob;
  const LinProb& r = p.pr[x.prob];
  u -= r.unit0;
  x.seg = u % p.nseg;
  u /= p.nseg;
  x.tile = u % r.tiles;
  u /= r.tiles;
  x.oh = u % r.oh;
  x.b = u / r.oh;
  return x;
}
// The state pass runs over single heads and every segment but the scan's last.
__device__ __forceinline__ LinUnit lin_state_unit(const LinArgs& p, int u) {
  LinUnit x;
  x.prob = 0;
  while (x.prob + 1 < p.nprob && u >= p.pr[x.prob + 1].sunit0) ++x.prob;
  const LinProb& r = p.pr[x.prob];
  u -= r.sunit0;
  x.seg = u % (p.nseg - 1) + (r.rev ? 1 : 0);
  u /= p.nseg - 1;
  x.tile = u % r.tiles;
  u /= r.tiles;
  x.oh = u % p.H;
  x.b = u / p.H;
  return x;
}

bool lin_is_wide(int a);  // the tensor-core kernels pad a to 64 or 128
cudaError_t launch_lin_tc(LinArgs& p, int ctas, cudaStream_t st);
cudaError_t launch_lin_f32(LinArgs& p, cudaStream_t st);
cudaError_t launch_lin_scan(const LinArgs& p, cudaStream_t st);

struct LinStepArgs {
  int B, H, hpg, dk, dv;
  const void* q;
  const void* k;
  const void* v;
  const float* log_a;
  void* o;
  float* states;
};
cudaError_t launch_lin_step(const LinStepArgs& d, bool bf16, cudaStream_t st);

}  // namespace ll
