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
  int tiles;                 // ceil(b / 64)
  int nh;                    // heads summed into one output head (1 or hpg)
  int unit0;                 // units of the scans before this one
  int split0, nsplit;        // first unit (of this scan) that is cut into segments, their number
  int sunit0;                // work items of the state pass before this scan's
  float* seg;                // (nsplit, nh, nseg, a, 64): segment totals, then start states
};

// A unit is the 64 output columns of a tile, for one output head and batch row, over the
// whole sequence.  The first `nwhole` units (over all scans) are one work item each; the
// others are cut into nseg segments of L chunks, whose start states a pass over Y and Z
// and a prefix over the segments provide.
struct LinArgs {
  int B, T, H, hpg;
  int chunk;            // tokens per chunk
  int NC;               // chunks over T
  int nseg, L;
  int nwhole, items, sitems;  // work items of the output and of the state pass
  int sub;              // grouped outputs: chunks that one head runs before the next one does
  int nprob;
  const float* log_a;   // (H)
  const int* lengths;   // NULL or (B)
  float* scratch;       // grouped outputs, per CTA: sub * 128 * 64 sums, hpg * 128 * 64 states
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

// A work item: columns 64 tile .. of out head oh of batch row b over chunks [lo, hi).
struct LinItem {
  int prob, unit, b, oh, tile;
  int seg, lo, hi;
};
__device__ __forceinline__ void lin_locate(const LinArgs& p, LinItem& x) {
  const LinProb& r = p.pr[x.prob];
  x.tile = x.unit % r.tiles;
  x.oh = x.unit / r.tiles % r.oh;
  x.b = x.unit / r.tiles / r.oh;
  x.lo = x.seg * p.L;
  x.hi = min(x.lo + p.L, p.NC);
}
__device__ __forceinline__ LinItem lin_item(const LinArgs& p, int u) {
  LinItem x;
  const bool whole = u < p.nwhole;
  x.seg = whole ? 0 : (u - p.nwhole) % p.nseg;
  if (!whole) u = p.nwhole + (u - p.nwhole) / p.nseg;
  x.prob = 0;
  while (x.prob + 1 < p.nprob && u >= p.pr[x.prob + 1].unit0) ++x.prob;
  x.unit = u - p.pr[x.prob].unit0;
  lin_locate(p, x);
  if (whole) x.hi = p.NC;
  return x;
}
// An item of the state pass: one head `hi` of a unit, one segment (all but the scan's last).
__device__ __forceinline__ LinItem lin_state_item(const LinArgs& p, int u, int* head) {
  LinItem x;
  x.prob = 0;
  while (x.prob + 1 < p.nprob && u >= p.pr[x.prob + 1].sunit0) ++x.prob;
  const LinProb& r = p.pr[x.prob];
  u -= r.sunit0;
  x.seg = u % (p.nseg - 1) + (r.rev ? 1 : 0);
  u /= p.nseg - 1;
  *head = u % r.nh;
  x.unit = r.split0 + u / r.nh;
  lin_locate(p, x);
  return x;
}
// Where head `hi` (of the output's group) of a unit keeps its segment's state.
__device__ __forceinline__ float* lin_seg(const LinArgs& p, const LinItem& x, int hi) {
  const LinProb& r = p.pr[x.prob];
  return r.seg + (((size_t)(x.unit - r.split0) * r.nh + hi) * p.nseg + x.seg) * r.a * kLinTile;
}
__device__ __forceinline__ bool lin_is_split(const LinArgs& p, const LinItem& x) {
  return x.unit >= p.pr[x.prob].split0;
}
// Whether the item reaches the scan's end (and so leaves the end state).
__device__ __forceinline__ bool lin_is_last(const LinArgs& p, const LinItem& x) {
  return p.pr[x.prob].rev ? x.lo == 0 : x.hi == p.NC;
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
