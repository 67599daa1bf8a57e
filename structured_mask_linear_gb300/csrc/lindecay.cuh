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
  int unit0, nunits;         // units of the scans before this one, and its own
  long long pos0, cost;      // wrapped: where the scan's units start on the line, cost per chunk
  int split0, nsplit;        // segmented: first unit (of this scan) that is cut, number of those
  int sunit0;                // work items of the state pass before this scan's
  float* seg;                // (nsplit, nh, nseg, a, 64): segment totals, then start states
};

// A unit is the 64 output columns of a tile, for one output head and batch row, over the
// whole sequence.  Persistent CTAs share the units out in one of two ways.
//
// Wrapped (turn > 0): the units lie end to end on a line of costs that is cut into one
// piece of length `turn` per CTA.  (Units that read the same X and Y, neighbours in their
// numbering, are dealt to `abreast` CTAs that keep step, one line for each, so that what
// one of them loads is in L2 for the others.)  A unit that a cut divides is run in two parts: its first
// chunks by the CTA behind the cut, as that CTA's first item, its last chunks by the CTA
// before the cut, as that one's last item.  No unit is longer than a turn, so the first
// part ends before the second has to start; the state goes over through `hand`, a flag
// says when.  The launch is cooperative (all CTAs run at the same time).
//
// Segmented (turn == 0): the first `nwhole` units (over all scans) are one work item each;
// the others are cut into nseg segments of L chunks, whose start states a pass over Y and Z
// and a prefix over the segments provide.  Items are dealt out round robin.
struct LinArgs {
  int B, T, H, hpg;
  int chunk;            // tokens per chunk
  int NC;               // chunks over T
  long long turn, total;  // wrapped: length of a CTA's piece, and of the line
  int abreast;
  float* hand;            // (CTAs, hpg, 128, 64): the state that CTA m's first item leaves
  unsigned* flag;         // (CTAs), zero at launch
  int nseg, L;
  int nwhole, items, sitems;  // work items of the output and of the state pass
  int sub;              // grouped outputs: chunks that one head runs before the next one does
  int keep;             // states that wait for their heads' next turn: hpg, 0 where there is but one
  int nprob;
  const float* log_a;   // (H)
  const int* lengths;   // NULL or (B)
  float* scratch;       // heads in turns, per CTA: sub * 128 * 64 sums, keep * 128 * 64 states
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

// A work item: columns 64 tile .. of out head oh of batch row b over chunks k0 .. k1 - 1 in
// the scan's order (chunk k is the k-th from the end where time runs backwards).
enum { kLinInit = 0, kLinSeg, kLinHand, kLinNone };  // where a state comes from, or goes to
struct LinItem {
  int prob, unit, b, oh, tile;
  int seg, k0, k1;
  int from, to, slot;  // start state: init, segment or hand; end state: none, fin (init) or hand
};
__device__ __forceinline__ void lin_locate(const LinArgs& p, LinItem& x) {
  const LinProb& r = p.pr[x.prob];
  x.tile = x.unit % r.tiles;
  x.oh = x.unit / r.tiles % r.oh;
  x.b = x.unit / r.tiles / r.oh;
}
// Item u of the segmented form.
__device__ __forceinline__ LinItem lin_item(const LinArgs& p, int u) {
  LinItem x;
  const bool whole = u < p.nwhole;
  x.seg = whole ? 0 : (u - p.nwhole) % p.nseg;
  if (!whole) u = p.nwhole + (u - p.nwhole) / p.nseg;
  x.prob = 0;
  while (x.prob + 1 < p.nprob && u >= p.pr[x.prob + 1].unit0) ++x.prob;
  x.unit = u - p.pr[x.prob].unit0;
  lin_locate(p, x);
  x.k0 = whole ? 0 : x.seg * p.L;
  x.k1 = whole ? p.NC : min(x.k0 + p.L, p.NC);
  x.from = whole ? kLinInit : kLinSeg;
  x.to = x.k1 == p.NC ? kLinInit : kLinNone;
  x.slot = 0;
  return x;
}
// Item j of CTA m in the wrapped form; false after its last one.
__device__ __forceinline__ bool lin_wrapped_item(const LinArgs& p, int m, int j, LinItem& x) {
  const int lane = m % p.abreast;
  const long long s = (m / p.abreast) * p.turn, e = min(s + p.turn, p.total);
  if (s >= p.total) return false;
  // the unit (of this CTA's line) that position s falls into, then j further
  x.prob = 0;
  while (x.prob + 1 < p.nprob && s >= p.pr[x.prob + 1].pos0) ++x.prob;
  int u = (int)((s - p.pr[x.prob].pos0) / (p.pr[x.prob].cost * p.NC)) + j;
  while (u >= p.pr[x.prob].nunits / p.abreast) {
    u -= p.pr[x.prob].nunits / p.abreast;
    if (++x.prob == p.nprob) return false;
  }
  const LinProb& r = p.pr[x.prob];
  const long long at = r.pos0 + u * r.cost * p.NC;
  if (at >= e) return false;
  x.unit = u * p.abreast + lane;
  lin_locate(p, x);
  x.seg = 0;
  x.k0 = 0;
  x.k1 = p.NC;
  x.from = x.to = kLinInit;
  x.slot = m;
  if (at < s) {  // cut before this CTA: the first chunks (all, if the part before the cut is empty)
    x.k1 = p.NC - (int)((s - at) / r.cost);
    if (x.k1 < p.NC) x.to = kLinHand;
  } else if (at + r.cost * p.NC > e) {  // cut behind it: the last chunks
    x.k0 = p.NC - (int)((e - at) / r.cost);
    x.from = kLinHand;
    x.slot = m + p.abreast;
    if (x.k0 == p.NC) return false;
  }
  return true;
}
// An item of the state pass: one head `hi` of a unit, one segment (all but the last).
__device__ __forceinline__ LinItem lin_state_item(const LinArgs& p, int u, int* head) {
  LinItem x;
  x.prob = 0;
  while (x.prob + 1 < p.nprob && u >= p.pr[x.prob + 1].sunit0) ++x.prob;
  const LinProb& r = p.pr[x.prob];
  u -= r.sunit0;
  x.seg = u % (p.nseg - 1);
  u /= p.nseg - 1;
  *head = u % r.nh;
  x.unit = r.split0 + u / r.nh;
  lin_locate(p, x);
  x.k0 = x.seg * p.L;
  x.k1 = x.k0 + p.L;
  x.from = x.to = kLinNone;
  x.slot = 0;
  return x;
}
// Where head `hi` (of the output's group) of a unit keeps its segment's state.
__device__ __forceinline__ float* lin_seg(const LinArgs& p, const LinItem& x, int hi) {
  const LinProb& r = p.pr[x.prob];
  return r.seg + (((size_t)(x.unit - r.split0) * r.nh + hi) * p.nseg + x.seg) * r.a * kLinTile;
}
// The item's chunks that hold tokens: the first one (in sequence order) that the scan
// visits, its direction, and how many.  cv = chunks that the row's length reaches.
__device__ __forceinline__ int lin_visit(const LinArgs& p, const LinItem& x, int cv, int* first, int* step) {
  if (!p.pr[x.prob].rev) {
    *first = x.k0;
    *step = 1;
    return max(0, min(x.k1, cv) - x.k0);
  }
  const int k = max(x.k0, p.NC - cv);
  *first = p.NC - 1 - k;
  *step = -1;
  return max(0, x.k1 - k);
}
// The item's tokens past the row's length: from `*t0` to before the returned one.
__device__ __forceinline__ int lin_past(const LinArgs& p, const LinItem& x, int cv, int* t0) {
  const bool rev = p.pr[x.prob].rev != 0;
  const int c0 = rev ? p.NC - x.k1 : x.k0, c1 = rev ? p.NC - x.k0 : x.k1;
  *t0 = max(c0, cv) * p.chunk;
  return min(p.T, c1 * p.chunk);
}

// On at most `ctas` CTAs, one per SM.
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
