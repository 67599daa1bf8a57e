// Tensor-core (tcgen05 / TMEM / TMA) kernels of the linear attention with a decay per head
// (the scan of lindecay.cuh) for bf16 tensors with widths up to 128, multiples of 8.
//
// One persistent CTA per SM walks units of work (a head's 64 output columns over one
// segment of the sequence) and, inside a unit, 128-token chunks in scan order.  The state
// R (a x 64) stays in registers between chunks, so each chunk's X, Y and Z are read once
// and its output written once.  Widths are padded to 64 or 128 by TMA's zero fill; columns
// past a width are clipped by the TMA store.
//
// Per chunk and head, in fp32 tensor-memory accumulators:
//     S  = X Yᵀ                    128 x 128 x a
//     Ob = X (Rhi + Rlo)           128 x 64 x a     (R as two bf16 parts)
//     D  = Yᵀ (Zhi + Zlo)          a x 64 x 128     (w_j Z_j as two bf16 parts)
//     Oa = P Z                     128 x 64 x 128   (P = S g^|i-j|, masked, rounded to bf16)
// and out_i = Oa_i + g^(i'+sh) Ob_i, R <- g^nv R + D.  Where an output sums over a group with
// an even number of heads, a CTA takes two heads side by side: their items alternate, Oa
// adds up over both, each has its own Ob and R (for the gradients of 2 x 8192 tokens, 48
// heads of 128 and 64 in pairs, 408 us today, it took 560 -> 424 against one head after the
// other with fp32 sums in global memory; larger and odd groups still take their turns that way).
//
// Roundings: X, Y, Z enter exactly.  P enters as bf16: an output averages over its terms, or
// is one of them and then no less exact than its own rounding.  R enters Ob as two parts:
// one alone put the largest errors, where a row is mostly its state_in, at 0.053 RMS of the
// output, outside the package's bar of 0.05 (it costs 8 % at 4 x 8192 x 48 heads).  w_j Z_j
// takes two parts because the states are fp32 outputs, and an error made in one chunk stays in
// them: what is left of a term is below 2^-15 of it, 4e-6 in the mean square.  (Splitting in
// fp32 arithmetic leaves 2.4e-6 and takes 3 % longer; a third part 1.3e-7, and 7 to 14 % longer
// with a <= 64, 30 % with 128, where its place in shared memory makes more turns of it.)  R
// itself is carried in fp32.
//
// Bound: memory, where every SM holds a head's whole sequence (152 heads of 64 and 64, 8192
// tokens: 105 us, 89 % of the copy rate; of 128 and 64: 151 us, 93 %); elsewhere the way of a
// chunk through the roles, of which two are under way at a time: 2.1 to 2.3 us a chunk of a =
// 128, with the tensor cores active for 37 % of it and shared memory's banks for 30 (4 x 8192
// tokens, 48 heads in pairs: 187 us, 65 % of the copy rate).  Ob's and D's two parts lie side
// by side in one product of 128 columns where tensor memory has the room: each then reads its
// left operand once.
//
// Warp roles (640 threads, five warpgroups; each keeps to one part of the chain, so that the
// parts of consecutive chunks overlap):
//   warps 0-3   P: reads S, writes P over it in tensor memory (row t in lane t)
//   warps 4-7   state: R's update from D, R's bf16 parts for Ob
//   warps 8-11  output: Oa, Ob -> out, staged and stored by TMA (32-byte stores straight from
//               the registers: 15 % slower)
//   warps 12-15 w Z: the high and low parts, through two slots
//   warp 16     TMA loads, two or three chunks ahead
//   warp 17     the MMAs of S, a chunk ahead of warp 18
//   warp 18     the MMAs of D, Ob and Oa
// The launch gives 96 registers a thread; the groups pass on what they do not need.
//
// Every wait is bounded; one that runs out records LL_ERR_TIMEOUT, after which its role runs
// through its walk without waiting or working (those that meet at named barriers keep meeting
// there).  Roles that miss its part give up on their own 2 s later; each lets what it started
// end, and the CTA returns.  Nothing but its own waits makes a role give up: a word that all
// would look at first, to give up together, costs 4 % of the training gradients (409 -> 426 us
// for 2 x 8192 tokens, 48 heads; in shared memory 439), and the status word may hold what
// another launch has left there.
#include "launch_util.cuh"
#include "lindecay.cuh"
#include "tc_common.cuh"

namespace ll {

namespace {

constexpr int kThreads = 640;
constexpr int kC = kLinChunk;
constexpr int kZBytes = kC * kLinTile * 2;  // 16 KB: 128 tokens x 64 columns, bf16
constexpr int kMisc = 2048;     // barriers, P's tables

template <int KA>
struct Lay {
  static constexpr int kX = kC * KA * 2;
  static constexpr int kStages = KA == 64 ? 3 : 2;
  static constexpr int kRing = kStages * (2 * kX + kZBytes);
  static constexpr int kTok = KA == 64 ? 64 : 32;  // tokens of w Z in a slot, of two
  static constexpr int kSlot = kTok * 256;         // their high part, their low part
  static constexpr int kZt = kRing;
  static constexpr int kImg = kZt + 2 * kSlot;     // R's high part: KA rows x 128 bytes
  static constexpr int kImgLo = kImg + KA * 128;   // its low part
  static constexpr int kOut = kImgLo + KA * 128;   // out tile on its way out
  static constexpr int kMiscOff = kOut + kZBytes;
  static constexpr int kBytes = kMiscOff + kMisc + 1024;  // + alignment
};
static_assert(Lay<128>::kBytes <= 232448, "shared memory");
static_assert(3 * (2 * Lay<64>::kX + kZBytes) <= Lay<128>::kRing, "a narrow scan's three stages in a wide ring");

// The ring of stages, X then Y then Z in each: three stages of a scan with a <= 64, two of a
// wider one (KS = 64-wide blocks of a).  Where a CTA's items differ in width, the ring starts
// over with the other layout; every role follows it through the same sequence.
template <int KA>
struct Ring {
  uint32_t st = 0, bits = 0;  // stage, and the phase of each stage's barriers
  int ks = KA == 64 ? 1 : 0;
  __device__ __forceinline__ bool narrow() const { return KA == 64 || ks == 1; }
  __device__ __forceinline__ bool width(int k) {  // whether the layout changes
    if (KA == 64 || k == ks) return false;
    ks = k;
    st = 0;
    return true;
  }
  __device__ __forceinline__ uint32_t x() const { return st * (narrow() ? 49152u : 81920u); }
  __device__ __forceinline__ uint32_t y() const { return x() + (narrow() ? 16384u : 32768u); }
  __device__ __forceinline__ uint32_t z() const { return x() + (narrow() ? 32768u : 65536u); }
  __device__ __forceinline__ uint32_t phase() const { return (bits >> st) & 1u; }
  __device__ __forceinline__ void next() {
    bits ^= 1u << st;
    st = st + 1 == (narrow() ? 3u : 2u) ? 0u : st + 1;
  }
};

struct LinMaps {
  CUtensorMap m[kLinProbs][4];  // X, Y, Z (loads), out (stores)
};

// Tensor-memory columns.  S of even and odd items, 128 each, P over the first 64 of them.  One
// head at a time: Oa in the other 64, then Ob and D, high and low parts side by side.  Two
// heads: their Ob, Oa, D, the two parts of each added up in place.
template <bool kGrouped>
struct Cols {
  static constexpr uint32_t kS = 0, kOb = 256, kD = kGrouped ? 448 : 384;
  static __device__ __forceinline__ uint32_t oa(uint32_t bf) { return kGrouped ? 384 : kS + 128 * bf + 64; }
};

// The chunks a CTA works on, in runs of one head, or two at a time; every role walks the same
// sequence.  An item whose heads are summed, more than two or an odd number of them, is cut
// into blocks of p.sub chunks, the heads taking turns block by block; otherwise the item is one
// run.
struct Walk {
  const LinArgs& p;
  bool state_only, live_;
  int u;             // item: its number, or (wrapped) how manyth of this CTA
  LinItem x;
  int nh, hi;        // heads of the item, current one (first: h0)
  int h0, lanes;     // heads at a time: hi .. hi + lanes - 1
  int n;             // number of chunks with tokens
  int len;           // valid tokens of the batch row
  int k0, k, k1;     // the run's chunks in scan order: k0 .. k1 - 1, k the current one
  int c0, dc;        // chunk k is c0 + dc k in sequence order
  bool rev;
  __device__ __forceinline__ Walk(const LinArgs& a, bool s) : p(a), state_only(s) {
    u = !s && p.turn > 0 ? 0 : (int)blockIdx.x;
    enter();
  }
  __device__ __forceinline__ bool live() const { return live_; }
  __device__ __forceinline__ const LinProb& prob() const { return p.pr[x.prob]; }
  __device__ __forceinline__ int chunks_valid() const { return (len + kC - 1) / kC; }
  __device__ __forceinline__ void enter() {
    h0 = 0;
    if (!state_only && p.turn > 0) {
      // CTA numbers run against the line, so that a CTA waits for one of a lower number
      live_ = lin_wrapped_item(p, (int)(gridDim.x - 1 - blockIdx.x), u, x);
    } else {
      live_ = u < (state_only ? p.sitems : p.items);
      if (live_) x = state_only ? lin_state_item(p, u, &h0) : lin_item(p, u);
    }
    if (!live_) return;
    nh = state_only ? 1 : prob().nh;
    lanes = nh & 1 ? 1 : 2;
    hi = h0;
    len = lin_len(p, x.b);
    n = lin_visit(p, x, chunks_valid(), &c0, &dc);
    rev = dc < 0;
    block(0);
  }
  __device__ __forceinline__ void block(int first) {
    k0 = k = first;
    k1 = nh > lanes ? min(n, first + p.sub) : n;
  }
  __device__ __forceinline__ int head(int lane) const { return x.oh * prob().nh + hi + lane; }
  __device__ __forceinline__ int chunk() const { return c0 + dc * k; }
  __device__ __forceinline__ int valid() const { return min(kC, len - chunk() * kC); }
  __device__ __forceinline__ bool first_head() const { return hi == h0; }
  __device__ __forceinline__ bool last_head() const { return hi + lanes == h0 + nh; }
  __device__ __forceinline__ bool first_block() const { return k0 == 0; }
  __device__ __forceinline__ bool last_block() const { return k1 == n; }
  __device__ __forceinline__ void next_run() {
    if (!last_head()) {
      hi += lanes;
      k = k0;
    } else if (!last_block()) {
      hi = h0;
      block(k1);
    } else {
      u += !state_only && p.turn > 0 ? 1 : (int)gridDim.x;
      enter();
    }
  }
};

// Per-CTA barriers (in shared memory)
struct Bars {
  uint64_t xy_full[3], xy_empty[3], z_full[3], z_empty[3], s_full[2], p_ready[2], pv_done[2], z_ready[2], z_free[2],
      o_empty[2], o_full, r_ready, q_full, d_full, d_free, fin[2];
  uint32_t tmem;
};

// A bounded wait; %globaltimer is slow to read, so only waits that last come to it.
__device__ __forceinline__ bool lin_wait(uint64_t* bar, uint32_t parity, const LinArgs& p) {
#pragma unroll 1
  for (int i = 0; i < 1024; ++i)
    if (__builtin_expect(ptx::mbar_try_wait(bar, parity), 1)) return true;
  if (wait_bar(bar, parity)) return true;
  atomicExch(p.status, kStatusTimeout);
  return false;
}
// The same for a role of whole warps: every lane continues or none.
__device__ __forceinline__ bool lin_wait_warp(uint64_t* bar, uint32_t parity, const LinArgs& p) {
  return __all_sync(0xffffffffu, lin_wait(bar, parity, p));
}

// Waits (bounded: 4 s) until another CTA has raised a flag; reads behind it see what that
// CTA wrote before.
__device__ __forceinline__ bool lin_wait_flag(const unsigned* flag, const LinArgs& p) {
  const uint64_t t0 = ptx::globaltimer_ns();
  bool ok = true;
  while (ok && !__all_sync(0xffffffffu, ptx::ld_acquire_gpu(flag) != 0u))
    ok = !__any_sync(0xffffffffu, ptx::globaltimer_ns() - t0 > 2 * kWaitNs);
  if (!ok) atomicExch(p.status, kStatusTimeout);
  return ok;
}

// KA is the width that the stages are laid out for; with KA = 128 a scan of a <= 64 uses the
// first half of its X and Y places (KS = 64-wide blocks of a).
template <int KA>
__device__ __forceinline__ int lin_blocks(const LinProb& r) {
  return KA == 64 || r.a <= 64 ? 1 : 2;
}

template <int KA, bool kStateOnly, bool kGrouped>
__global__ void __launch_bounds__(kThreads, 1) lin_tc_kernel(const __grid_constant__ LinMaps maps,
                                                             const __grid_constant__ LinArgs p) {
  using S = Lay<KA>;
  using C = Cols<kGrouped>;
  constexpr int kH = kGrouped ? 2 : 1;  // heads at a time, at most
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + S::kMiscOff);
  float* s_pow = reinterpret_cast<float*>(smem + S::kMiscOff + 512) + 32;  // P's weights, 96 numbers a head
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler too
  const int row = tid & 127, quad = warp & 3;
  const uint32_t loff = (uint32_t)(quad * 32) << 16;  // tensor-memory lanes of this warp

  if (tid == 512) {
    for (int i = 0; i < 3; ++i) {
      ptx::mbar_init(&bars.xy_full[i], 1);
      ptx::mbar_init(&bars.xy_empty[i], kStateOnly ? 1 : 2);
      ptx::mbar_init(&bars.z_full[i], 1);
      ptx::mbar_init(&bars.z_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars.s_full[i], 1);
      ptx::mbar_init(&bars.p_ready[i], 128);
      ptx::mbar_init(&bars.pv_done[i], 1);
      ptx::mbar_init(&bars.o_empty[i], 128);
      ptx::mbar_init(&bars.z_ready[i], 128);
      ptx::mbar_init(&bars.z_free[i], 1);
    }
    ptx::mbar_init(&bars.o_full, 1);
    ptx::mbar_init(&bars.r_ready, 128);
    ptx::mbar_init(&bars.q_full, 1);
    ptx::mbar_init(&bars.d_full, 1);
    ptx::mbar_init(&bars.d_free, 128);
    ptx::mbar_init(&bars.fin[0], 1);
    ptx::mbar_init(&bars.fin[1], 1);
    ptx::fence_mbar_init();
  }
  if (warp == 18) {
    ptx::tmem_alloc(&bars.tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tb = bars.tmem;

  const int group = warp >> 2;
  if (group == 4) {
    ptx::regs_dec<kGrouped ? 56 : 72>();
    if (warp == 16) {
      // ---- loads ------------------------------------------------------------------------
      Ring<KA> rg;
      uint32_t used = 0;  // stages that have been filled
      bool ok = true;
      for (Walk w(p, kStateOnly); ok && w.live(); w.next_run()) {
        const LinProb& r = w.prob();
        const CUtensorMap* m = maps.m[w.x.prob];
        const int ks = lin_blocks<KA>(r);
        if (rg.width(ks))  // the whole ring has to be free of the other layout
          for (int i = 0; i < 3; ++i)
            if ((used >> i) & 1u) {
              const uint32_t par = ((rg.bits >> i) & 1u) ^ 1u;
              ok = ok && lin_wait_warp(&bars.xy_empty[i], par, p) && lin_wait_warp(&bars.z_empty[i], par, p);
            }
        for (; ok && w.k < w.k1; ++w.k) {
          const int t0 = w.chunk() * kC;
#pragma unroll 1
          for (int hs = 0; ok && hs < (kGrouped ? w.lanes : 1); ++hs) {
            const int h = w.head(hs), g = h / p.hpg;
            const int hx = r.xh == p.H ? h : g, hy = r.yh == p.H ? h : g, hz = r.zh == p.H ? h : g;
            const uint32_t s = rg.st, par = rg.phase() ^ 1u;
            const bool again = (used >> s) & 1u;
            ok = !again || lin_wait_warp(&bars.xy_empty[s], par, p);
            if (!ok) break;
            if (ptx::elect_one()) {
              ptx::mbar_arrive_expect_tx(&bars.xy_full[s], (kStateOnly ? 1 : 2) * ks * 16384);
#pragma unroll
              for (int c = 0; c < KA / 64; ++c) {
                if (c >= ks) break;
                ptx::tma_load_4d(smem + rg.y() + c * 16384, &m[1], &bars.xy_full[s], 64 * c, hy, t0, w.x.b);
                if (!kStateOnly)
                  ptx::tma_load_4d(smem + rg.x() + c * 16384, &m[0], &bars.xy_full[s], 64 * c, hx, t0, w.x.b);
              }
            }
            __syncwarp();
            ok = !again || lin_wait_warp(&bars.z_empty[s], par, p);
            if (!ok) {  // X and Y of this chunk are on their way
              wait_bar(&bars.xy_full[s], rg.phase());
              break;
            }
            if (ptx::elect_one()) {
              ptx::mbar_arrive_expect_tx(&bars.z_full[s], kZBytes);
              ptx::tma_load_4d(smem + rg.z(), &m[2], &bars.z_full[s], kLinTile * w.x.tile, hz, t0, w.x.b);
            }
            __syncwarp();
            used |= 1u << s;
            rg.next();
          }
        }
      }
      for (int i = 0; i < 3; ++i)  // let the copies in flight land before the CTA ends (bounded)
        if ((used >> i) & 1u) {
          const uint32_t par = ((rg.bits >> i) & 1u) ^ 1u;
          wait_bar(&bars.xy_full[i], par);
          wait_bar(&bars.z_full[i], par);
        }
    } else if (!kStateOnly && warp == 17) {
      // ---- MMAs of S: the whole warp walks, one lane issues --------------------------------
      // descriptors at the start of shared memory; their low 14 bits count 16-byte units, so
      // an offset is added there (addresses stay below 2^18)
      const uint64_t kmaj = ptx::smem_desc_sw128(ptx::smem_u32(smem), 16, 1024);
      uint32_t it = 0;
      Ring<KA> rg;
      bool ok = true;
      for (Walk w(p, false); ok && w.live(); w.next_run()) {
        const int ks = lin_blocks<KA>(w.prob());
        rg.width(ks);
        const int n = (w.k1 - w.k0) * (kGrouped ? w.lanes : 1);
        for (int i = 0; i < n; ++i, ++it, rg.next()) {
          const uint32_t bf = it & 1;
          // the product over P that lay in these columns two items ago (and was put there)
          ok = it < 2 || lin_wait_warp(kGrouped ? &bars.pv_done[bf] : &bars.o_empty[bf], ((it >> 1) & 1) ^ 1, p);
          ok = ok && lin_wait_warp(&bars.xy_full[rg.st], rg.phase(), p);
          if (!ok) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint32_t idesc = ptx::idesc_bf16_f32(128, 128, 0, 0);
            const uint64_t dx = kmaj + (rg.x() >> 4), dy = kmaj + (rg.y() >> 4);
#pragma unroll
            for (int kk = 0; kk < KA / 16; ++kk) {
              if (kk >= 4 * ks) break;
              const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
              ptx::umma_f16(tb + C::kS + 128 * bf, dx + off, dy + off, idesc, kk > 0);
            }
            ptx::umma_commit(&bars.s_full[bf]);
            ptx::umma_commit(&bars.xy_empty[rg.st]);
          }
          __syncwarp();
        }
      }
      // no MMA outlives the CTA, whatever its other roles came to (bounded)
      if (ptx::elect_one()) ptx::umma_commit(&bars.fin[0]);
      wait_bar(&bars.fin[0], 0);
    } else if (warp == 18) {
      // ---- MMAs of D, Ob, Oa --------------------------------------------------------------
      const uint32_t s0 = ptx::smem_u32(smem);
      const uint64_t kmaj = ptx::smem_desc_sw128(s0, 16, 1024);       // X of Ob
      const uint64_t zmaj = ptx::smem_desc_sw128(s0, 1024, 1024);     // operands of one 64-wide block
      const uint64_t amaj = ptx::smem_desc_sw128(s0, 16384, 1024);      // Yᵀ of D
      const uint64_t bmaj = ptx::smem_desc_sw128(s0, S::kSlot / 2, 1024);  // [Zhi | Zlo] of D
      const uint64_t rmaj = ptx::smem_desc_sw128(s0, KA * 128, 1024);   // [Rhi | Rlo] of Ob
      constexpr int kParts = kC / S::kTok;
      uint32_t it = 0, turn = 0;  // items, and output tiles before the current one
      Ring<KA> rg;
      bool ok = true;
      for (Walk w(p, kStateOnly); ok && w.live(); w.next_run()) {
        const int ks = lin_blocks<KA>(w.prob()), lanes = kGrouped ? w.lanes : 1;
        rg.width(ks);
        const int n = (w.k1 - w.k0) * lanes;
        int hs = 0;
        for (int i = 0; ok && i < n; ++i, ++it, rg.next()) {
          const uint32_t st = rg.st, bf = it & 1, par = it & 1;
          // D = Yᵀ Zhi, Yᵀ Zlo, a slot of tokens after the other: A is MN-major with M = 128 (with
          // a padded to 64 its second 64 rows read what lies 16 KB behind Y: lanes 64..127 of D
          // are never read); B is two 64-wide blocks, side by side or one after the other into
          // the same columns.
          ok = lin_wait_warp(&bars.xy_full[st], rg.phase(), p);
          if (it > 0) ok = ok && lin_wait_warp(&bars.d_free, par ^ 1, p);
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const int slot = part & 1;
            ok = ok && lin_wait_warp(&bars.z_ready[slot], kParts == 4 ? part >> 1 : par, p);
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t dy = amaj + (rg.y() >> 4) + part * (S::kTok * 8);
              const uint64_t dz = bmaj + ((S::kZt + slot * S::kSlot) >> 4);
              if (kGrouped) {
                const uint32_t idesc = ptx::idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                  for (int kk = 0; kk < S::kTok / 16; ++kk)
                    ptx::umma_f16(tb + C::kD, dy + kk * 128, dz + lo * (S::kSlot >> 5) + kk * 128, idesc, part + lo + kk > 0);
              } else {
                const uint32_t idesc = ptx::idesc_bf16_f32(128, 128, 1, 1);
#pragma unroll
                for (int kk = 0; kk < S::kTok / 16; ++kk)
                  ptx::umma_f16(tb + C::kD, dy + kk * 128, dz + kk * 128, idesc, part + kk > 0);
              }
              ptx::umma_commit(&bars.z_free[slot]);
              if (part == kParts - 1) {
                ptx::umma_commit(&bars.d_full);
                if (kStateOnly) {
                  ptx::umma_commit(&bars.xy_empty[st]);
                  ptx::umma_commit(&bars.z_empty[st]);
                }
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (!kStateOnly) {
            const uint32_t idesc = ptx::idesc_bf16_f32(128, 64, 0, 1);
            // the tile before has been read out of Ob (and Oa)
            if (kGrouped) {
              if (hs == 0 && turn > 0) ok = lin_wait_warp(&bars.o_empty[0], (turn & 1) ^ 1, p);
            } else {
              if (it > 0) ok = lin_wait_warp(&bars.o_empty[bf ^ 1], ((it - 1) >> 1) & 1, p);
            }
            ok = ok && lin_wait_warp(&bars.r_ready, par, p);
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t dx = kmaj + (rg.x() >> 4);
#pragma unroll
              for (int kk = 0; kk < KA / 16; ++kk) {
                if (kk >= 4 * ks) break;
                const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                if (kGrouped) {
                  ptx::umma_f16(tb + C::kOb + 64 * hs, dx + off, zmaj + (S::kImg >> 4) + kk * 128, idesc, kk > 0);
                  ptx::umma_f16(tb + C::kOb + 64 * hs, dx + off, zmaj + (S::kImgLo >> 4) + kk * 128, idesc, true);
                } else {
                  ptx::umma_f16(tb + C::kOb, dx + off, rmaj + (S::kImg >> 4) + kk * 128, ptx::idesc_bf16_f32(128, 128, 0, 1),
                                kk > 0);
                }
              }
              ptx::umma_commit(&bars.q_full);
              ptx::umma_commit(&bars.xy_empty[st]);
            }
            __syncwarp();
            ok = lin_wait_warp(&bars.p_ready[bf], (it >> 1) & 1, p);
            if (!ok) break;
            ptx::tc_fence_after();
            const bool last = !kGrouped || hs + 1 == lanes;
            if (ptx::elect_one()) {
              const uint32_t tp = tb + C::kS + 128 * bf;
              const uint64_t dz = zmaj + (rg.z() >> 4);
#pragma unroll
              for (int kk = 0; kk < kC / 16; ++kk)
                ptx::umma_f16_tmem_a(tb + C::oa(bf), tp + 8 * kk, dz + kk * 128, idesc, hs + kk > 0);
              if (kGrouped) ptx::umma_commit(&bars.pv_done[bf]);
              ptx::umma_commit(&bars.z_empty[st]);
              if (last) ptx::umma_commit(&bars.o_full);
            }
            __syncwarp();
            if (kGrouped) hs = last ? 0 : hs + 1;
            if (last) ++turn;
          }
        }
      }
      if (ptx::elect_one()) ptx::umma_commit(&bars.fin[1]);
      wait_bar(&bars.fin[1], 0);
    }
  } else if (group == 0) {
    if (kGrouped) ptx::regs_dec<88>();
    if (!kStateOnly) {
      // ---- P ----------------------------------------------------------------------------
      uint32_t it = 0;
      bool ok = true;
      for (Walk w(p, false); w.live(); w.next_run()) {
        if (w.k0 == w.k1) continue;
        const bool rev = w.rev;
        // Weights g^|i-j|, row i = 32 quad + lane against key j of group cg.  On the diagonal
        // (quad = cg) from a table over lane - j, 0 where the mask is: a warp's lanes read 32
        // entries in a row.  Off it the lag is a sum of three that are none of them negative, 32
        // per group between, the row's way to its group's edge and the key's to its own: a
        // factor per row and one per key, the same for every lane (no power overflows).
        ptx::named_bar_sync(1, 128);
        float rowf[kH], g32[kH];
#pragma unroll
        for (int hs = 0; hs < kH; ++hs) {
          const float l2 = lin_log2_decay(p.log_a, w.head(hs < w.lanes ? hs : 0));
          rowf[hs] = exp2f(l2 * (float)(rev ? 32 - lane : lane + 1));
          g32[hs] = exp2f(32.f * l2);
          const int d = row - 32;  // lag (of the other sign for a scan backwards)
          if (row < 64) s_pow[96 * hs + d] = (rev ? d > 0 : d < 0) ? 0.f : exp2f(l2 * fabsf((float)d));
          else if (row < 96) s_pow[96 * hs + d] = exp2f(l2 * (float)(rev ? row - 64 : 95 - row));
        }
        ptx::named_bar_sync(1, 128);
        for (; w.k < w.k1; ++w.k) {
          const int nv = w.valid();
#pragma unroll 1
          for (int hs = 0; hs < (kGrouped ? w.lanes : 1); ++hs, ++it) {
            const uint32_t bf = it & 1;
            ok = ok && lin_wait_warp(&bars.s_full[bf], (it >> 1) & 1, p);
            if (!ok) continue;
            ptx::tc_fence_after();
            const uint32_t ts = tb + C::kS + 128 * bf + loff;
#pragma unroll 1
            for (int cg = 0; cg < 4; ++cg) {
              uint32_t pk[16];
              const int back = rev ? cg - quad : quad - cg;  // 32-groups behind the row's own
              if (back >= 0) {
                float2 sv[16];
                ptx::tmem_ld32(ts + 32 * cg, reinterpret_cast<float*>(sv));
                if (back == 0) {
                  const float* t = s_pow + 96 * hs + lane;
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    const float2 wt = make_float2(t[-2 * j], t[-2 * j - 1]);
                    if (j == 0) ptx::tmem_ld_wait();
                    sv[j] = ptx::mul2(sv[j], wt);
                    pk[j] = pack_bf16(sv[j].x, sv[j].y);
                  }
                } else {
                  const float g = g32[hs && kH > 1], rw = rowf[hs && kH > 1] * (back == 1 ? 1.f : back == 2 ? g : g * g);
                  const float4* t = reinterpret_cast<const float4*>(s_pow + 96 * hs + 32);
                  ptx::tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float4 c = t[j];
                    const float2 a = ptx::mul2(ptx::mul2(sv[2 * j], make_float2(rw, rw)), make_float2(c.x, c.y));
                    const float2 b = ptx::mul2(ptx::mul2(sv[2 * j + 1], make_float2(rw, rw)), make_float2(c.z, c.w));
                    pk[2 * j] = pack_bf16(a.x, a.y);
                    pk[2 * j + 1] = pack_bf16(b.x, b.y);
                  }
                }
                if (nv < 32 * cg + 32) {  // keys past the row's length (warp-uniform): P = 0
                  const int keep = nv - 32 * cg;
#pragma unroll
                  for (int j = 0; j < 16; ++j) pk[j] &= 2 * j + 1 < keep ? ~0u : 2 * j < keep ? 0xffffu : 0u;
                }
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = 0u;
              }
              // keys 32 cg .. : columns of S that this warp has read by now
              ptx::tmem_st16(ts + 16 * cg, pk);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bars.p_ready[bf]);
          }
        }
      }
    }
  } else if (group == 1) {
    ptx::regs_inc<kGrouped ? 176 : 128>();
    // ---- state: thread `row` holds row `row` of R ----------------------------------------
    const uint32_t td = tb + C::kD + loff;
    const int rot = row & 7;
    uint8_t* img = smem + S::kImg + row * 128;
    bool holds = true;  // a row of R (warp-uniform)
    uint32_t it = 0;
    bool ok = true;
    float R[kH][kLinTile];
    // one item of the head whose state is in R
    auto item = [&](float(&R)[kLinTile], float dec) {
      if (!kStateOnly) {
        if (it > 0) ok = ok && lin_wait_warp(&bars.q_full, (it & 1) ^ 1, p);  // the image is free
        if (!ok) return;
        if (holds) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 x = make_float2(R[8 * c + 2 * e], R[8 * c + 2 * e + 1]);
              hi[e] = pack_bf16(x.x, x.y);
              const float2 f = make_float2(__uint_as_float(hi[e] << 16), __uint_as_float(hi[e] & 0xffff0000u));
              const float2 rest = ptx::fma2(f, make_float2(-1.f, -1.f), x);
              lo[e] = pack_bf16(rest.x, rest.y);
            }
            *reinterpret_cast<uint4*>(img + ((c ^ rot) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(img + KA * 128 + ((c ^ rot) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          ptx::fence_proxy_async_smem();
        }
        ptx::mbar_arrive(&bars.r_ready);
      }
      ok = ok && lin_wait_warp(&bars.d_full, it & 1, p);
      if (!ok) return;
      if (holds) {
        ptx::tc_fence_after();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float d[16], dl[16];
          ptx::tmem_ld16(td + 16 * q, d);
          if (!kGrouped) ptx::tmem_ld16(td + 64 + 16 * q, dl);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float2& x = *reinterpret_cast<float2*>(R + 16 * q + j);
            float2 y = make_float2(d[j], d[j + 1]);
            if (!kGrouped) y = ptx::add2(y, make_float2(dl[j], dl[j + 1]));
            x = ptx::fma2(make_float2(dec, dec), x, y);
          }
        }
        ptx::tc_fence_before();
      }
      ptx::mbar_arrive(&bars.d_free);
    };
    for (Walk w(p, kStateOnly); w.live(); w.next_run()) {
      const LinProb& r = w.prob();
      const int lanes = kGrouped ? w.lanes : 1;
      const int c0 = kLinTile * w.x.tile;
      const int nc = min(kLinTile, r.b - c0);  // columns of this tile, a multiple of 8
      // states of heads that wait for their turn, and of units that another CTA goes on with:
      // 16 float4s a row, consecutive rows side by side
      float4* keep = reinterpret_cast<float4*>(p.scratch) +
                     ((size_t)blockIdx.x * (p.sub + p.keep) + p.sub + w.hi) * (kC * kLinTile / 4) + row;
      float4* hand = reinterpret_cast<float4*>(p.hand) + ((size_t)w.x.slot * p.hpg + w.hi) * (kC * kLinTile / 4) + row;
      holds = row < 64 * lin_blocks<KA>(r);
      if (!kStateOnly && w.first_block() && w.first_head() && w.x.from == kLinHand)
        ok = ok && lin_wait_flag(p.flag + w.x.slot, p);
      float l2[kH];
#pragma unroll
      for (int hs = 0; hs < kH; ++hs) {
        l2[hs] = 0.f;
#pragma unroll
        for (int j = 0; j < kLinTile; ++j) R[hs][j] = 0.f;
        if (hs >= lanes) continue;
        l2[hs] = lin_log2_decay(p.log_a, w.head(hs));
        if (kStateOnly || row >= r.a) continue;
        const float4* from = nullptr;
        int step = kC;
        if (!w.first_block()) {
          from = keep + hs * (kC * kLinTile / 4);
        } else if (w.x.from == kLinHand) {
          from = hand + hs * (kC * kLinTile / 4);
        } else if (w.x.from == kLinSeg) {
          from = reinterpret_cast<const float4*>(lin_seg(p, w.x, w.hi + hs) + (size_t)row * kLinTile);
          step = 1;
        }
        if (from) {
#pragma unroll
          for (int j = 0; j < kLinTile / 4; ++j) {
            const float4 x = from[j * step];
            R[hs][4 * j] = x.x;
            R[hs][4 * j + 1] = x.y;
            R[hs][4 * j + 2] = x.z;
            R[hs][4 * j + 3] = x.w;
          }
        } else if (r.init) {
          const float* in = r.init + ((size_t)w.x.b * p.H + w.head(hs)) * r.a * r.b + (size_t)row * r.init_rs +
                            (size_t)c0 * r.init_cs;
#pragma unroll
          for (int j = 0; j < kLinTile; ++j)
            if (j < nc) R[hs][j] = in[(size_t)j * r.init_cs];
        }
      }
      for (; w.k < w.k1; ++w.k) {
        const float nv = (float)w.valid();
#pragma unroll
        for (int hs = 0; hs < kH; ++hs) {
          if (hs >= lanes) break;
          item(R[hs], exp2f(l2[hs] * nv));
          ++it;
        }
      }
#pragma unroll
      for (int hs = 0; hs < kH; ++hs) {
        if (!ok || hs >= lanes || row >= r.a) continue;
        if (kStateOnly) {
          float* seg = lin_seg(p, w.x, w.hi) + (size_t)row * kLinTile;
#pragma unroll
          for (int j = 0; j < kLinTile; j += 4)
            *reinterpret_cast<float4*>(seg + j) = make_float4(R[hs][j], R[hs][j + 1], R[hs][j + 2], R[hs][j + 3]);
        } else if (!w.last_block() || w.x.to == kLinHand) {
          float4* to = (w.last_block() ? hand : keep) + hs * (kC * kLinTile / 4);
#pragma unroll
          for (int j = 0; j < kLinTile / 4; ++j)
            to[j * kC] = make_float4(R[hs][4 * j], R[hs][4 * j + 1], R[hs][4 * j + 2], R[hs][4 * j + 3]);
        } else if (r.fin && w.x.to == kLinInit) {
          float* out = r.fin + (((size_t)w.x.b * p.H + w.head(hs)) * r.a + row) * r.b + c0;
#pragma unroll
          for (int j = 0; j < kLinTile; j += 4)
            if (j < nc)
              *reinterpret_cast<float4*>(out + j) = make_float4(R[hs][j], R[hs][j + 1], R[hs][j + 2], R[hs][j + 3]);
        }
      }
      if (!kStateOnly && w.x.to == kLinHand && w.last_block() && w.last_head()) {  // every head's state is out
        __threadfence();
        ptx::named_bar_sync(3, 128);
        if (ok && row == 0) ptx::st_release_gpu(p.flag + w.x.slot, 1u);
      }
    }
  } else if (group == 2) {
    if (!kGrouped) ptx::regs_inc<104>();  // 88 + 176 + 96 + 64 + 56, or 96 + 128 + 104 + 80 + 72: 5 x 96
    if (!kStateOnly) {
      // ---- output -----------------------------------------------------------------------
      const int rot = row & 7;
      uint8_t* stage = smem + S::kOut;
      float4* scr = reinterpret_cast<float4*>(p.scratch) +
                    (size_t)blockIdx.x * (p.sub + p.keep) * (kC * kLinTile / 4) + row;
      uint32_t turn = 0;
      bool ok = true;
      for (Walk w(p, false); w.live(); w.next_run()) {
        const LinProb& r = w.prob();
        const bool rev = w.rev;
        float l2[kH];
#pragma unroll
        for (int hs = 0; hs < kH; ++hs) l2[hs] = lin_log2_decay(p.log_a, w.head(hs < w.lanes ? hs : 0));
        const bool two = kGrouped && w.lanes == 2;
        const bool first = w.first_head(), last = w.last_head();
        const int c0 = kLinTile * w.x.tile;
        for (; w.k < w.k1; ++w.k, ++turn) {
          const int nv = w.valid(), ch = w.chunk();
          // sums over a group's heads: 16 float4 per row, consecutive rows side by side
          float4* sc = scr + (size_t)(w.k - w.k0) * (kC * kLinTile / 4);
          float wo[kH];
#pragma unroll
          for (int hs = 0; hs < kH; ++hs) wo[hs] = exp2f(l2[hs] * (float)(rev ? nv - 1 - row : row + 1));
          ok = ok && lin_wait_warp(&bars.o_full, turn & 1, p);
          ptx::tc_fence_after();
          if (!kGrouped || last) {
            if (row == 0) ptx::bulk_wait_read_all();  // the previous tile has left the staging area
            ptx::named_bar_sync(2, 128);
          }
          if (ok) {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              float2 acc[8], ob[8], ob2[8];
              float4 sum[4];
              ptx::tmem_ld16(tb + C::oa(turn & 1) + 16 * q + loff, reinterpret_cast<float*>(acc));
              ptx::tmem_ld16(tb + C::kOb + 16 * q + loff, reinterpret_cast<float*>(ob));
              if (!kGrouped || two) ptx::tmem_ld16(tb + C::kOb + 64 + 16 * q + loff, reinterpret_cast<float*>(ob2));
              if (kGrouped && !first)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = sc[(4 * q + j) * kC];
              ptx::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 8; ++j) acc[j] = ptx::fma2(make_float2(wo[0], wo[0]), ob[j], acc[j]);
              if (!kGrouped || two) {
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = ptx::fma2(make_float2(wo[kH - 1], wo[kH - 1]), ob2[j], acc[j]);
              }
              if (q == 3) {
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bars.o_empty[kGrouped ? 0 : turn & 1]);
              }
              if (row >= nv) {
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = make_float2(0.f, 0.f);
              }
              if (kGrouped && !first) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  acc[2 * j] = ptx::add2(acc[2 * j], make_float2(sum[j].x, sum[j].y));
                  acc[2 * j + 1] = ptx::add2(acc[2 * j + 1], make_float2(sum[j].z, sum[j].w));
                }
              }
              if (kGrouped && !last) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  sc[(4 * q + j) * kC] = make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
              } else {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  *reinterpret_cast<uint4*>(stage + row * 128 + (((2 * q + c) ^ rot) << 4)) =
                      make_uint4(pack_bf16(acc[4 * c].x, acc[4 * c].y), pack_bf16(acc[4 * c + 1].x, acc[4 * c + 1].y),
                                 pack_bf16(acc[4 * c + 2].x, acc[4 * c + 2].y),
                                 pack_bf16(acc[4 * c + 3].x, acc[4 * c + 3].y));
              }
            }
          }
          if (!kGrouped || last) {
            ptx::fence_proxy_async_smem();
            ptx::named_bar_sync(2, 128);
            if (ok && row == 0) {
              ptx::tma_store_4d(&maps.m[w.x.prob][3], stage, c0, w.x.oh, ch * kC, w.x.b);
              ptx::bulk_commit_group();
            }
          }
        }
        if (ok && last && w.last_block()) {  // chunks past the row's length: zeros
          int t0;
          const int t1 = lin_past(p, w.x, w.chunks_valid(), &t0);
          const int n8 = min(kLinTile, r.b - c0) / 8;
          for (int t = t0 + row; t < t1; t += kC) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(r.out) +
                                                (((size_t)w.x.b * p.T + t) * r.oh + w.x.oh) * r.b + c0);
            for (int c = 0; c < n8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      if (row == 0) ptx::bulk_wait_read_all();
    }
  } else if (group == 3) {
    ptx::regs_dec<kGrouped ? 64 : 80>();
    // ---- w Z: 32 tokens at a time, four threads a token and 16 columns each (in the narrow
    // kernel, whose slots have room, 64 tokens, two threads and 32 columns) -------------------
    constexpr int kTh = kC / S::kTok, kV = 8 / kTh;  // threads a token, 16-byte pieces of each
    const int part = (row & (kTh - 1)) * kV;
    uint32_t it = 0;
    Ring<KA> rg;
    bool ok = true;
    for (Walk w(p, kStateOnly); ok && w.live(); w.next_run()) {
      const bool rev = w.rev;
      float l2[kH];
#pragma unroll
      for (int hs = 0; hs < kH; ++hs) l2[hs] = lin_log2_decay(p.log_a, w.head(hs < w.lanes ? hs : 0));
      rg.width(lin_blocks<KA>(w.prob()));
      for (; ok && w.k < w.k1; ++w.k) {
        const int nv = w.valid();
#pragma unroll 1
        for (int hs = 0; ok && hs < (kGrouped ? w.lanes : 1); ++hs, ++it, rg.next()) {
          const float lg = hs == 0 ? l2[0] : l2[kH - 1];
          ok = lin_wait_warp(&bars.z_full[rg.st], rg.phase(), p);
          // rows of Y past the row's length are overwritten below: after their copy has landed
          if (ok && nv < kC) ok = lin_wait_warp(&bars.xy_full[rg.st], rg.phase(), p);
#pragma unroll 1
          for (int qt = 0; qt < kTh; ++qt) {
            const int slot = qt & 1, t = S::kTok * qt + row / kTh, rot = t & 7;
            uint8_t* z0 = smem + rg.z() + t * 128;
            uint8_t* zhi = smem + S::kZt + slot * S::kSlot + (row / kTh) * 128;
            uint4 x[kV];
#pragma unroll
            for (int c = 0; c < kV; ++c) x[c] = *reinterpret_cast<const uint4*>(z0 + (((part + c) ^ rot) << 4));
            const float wt = exp2f(lg * (float)(rev ? t + 1 : nv - 1 - t));
            const __nv_bfloat16 w1 = __float2bfloat16_rn(wt), w2 = __float2bfloat16_rn(wt - __bfloat162float(w1));
            const __nv_bfloat162 wh = __halves2bfloat162(w1, w1), wl = __halves2bfloat162(w2, w2);
            // the products over what the slot held before have read it
            if (ok && (qt > 1 || it > 0)) ok = lin_wait_warp(&bars.z_free[slot], (kTh == 4 ? qt >> 1 : it & 1) ^ 1, p);
            if (!ok) break;
            if (t < nv) {
#pragma unroll
              for (int c = 0; c < kV; ++c) {
                const int off = ((part + c) ^ rot) << 4;
                uint4 y;
                __nv_bfloat162* hx = reinterpret_cast<__nv_bfloat162*>(&x[c]);
                __nv_bfloat162* hy = reinterpret_cast<__nv_bfloat162*>(&y);
                // high part: bf16(wh z); low part: bf16(wl z + (wh z - high)), whose bracket
                // is exact in bf16 (a product of two 8-bit significands less its first 8 bits)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __nv_bfloat162 z = hx[e];
                  hx[e] = __hmul2(wh, z);
                  hy[e] = __hfma2(wl, z, __hfma2(wh, z, __hneg2(hx[e])));
                }
                *reinterpret_cast<uint4*>(zhi + off) = x[c];
                *reinterpret_cast<uint4*>(zhi + S::kSlot / 2 + off) = y;
              }
            } else {
              // past the row's length: whatever the padding holds must not reach a product
              const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
              uint8_t* y0 = smem + rg.y() + t * 128;
#pragma unroll 1
              for (int c = 0; c < kV; ++c) {
                const int off = (part + c) << 4;
                *reinterpret_cast<uint4*>(zhi + off) = zero;
                *reinterpret_cast<uint4*>(zhi + S::kSlot / 2 + off) = zero;
                *reinterpret_cast<uint4*>(z0 + off) = zero;
                for (int d = 0; d < rg.ks; ++d) *reinterpret_cast<uint4*>(y0 + d * 16384 + off) = zero;
              }
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&bars.z_ready[slot]);
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 18) ptx::tmem_dealloc(tb, 512);
}

template <int KA, bool kStateOnly, bool kGrouped>
cudaError_t launch_one(const LinArgs& p, const LinMaps& maps, int ctas, cudaStream_t st) {
  constexpr int smem = Lay<KA>::kBytes;
  static SmemLimit limit;
  cudaError_t e = limit.raise(lin_tc_kernel<KA, kStateOnly, kGrouped>, smem);
  if (e != cudaSuccess) return e;
  const bool wrapped = !kStateOnly && p.turn > 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(wrapped ? ctas : min(ctas, kStateOnly ? p.sitems : p.items));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (wrapped) {  // CTAs wait for one another: they have to run at the same time
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  if ((e = cudaLaunchKernelEx(&cfg, lin_tc_kernel<KA, kStateOnly, kGrouped>, maps, p)) == cudaSuccess) note_launch();
  return e;
}

template <int KA>
cudaError_t launch_ka(const LinArgs& p, const LinMaps& maps, int ctas, cudaStream_t st) {
  cudaError_t e;
  bool grouped = false;
  for (int i = 0; i < p.nprob; ++i) grouped = grouped || p.pr[i].nh > 1;
  if (p.turn > 0) {
    if ((e = cudaMemsetAsync(p.flag, 0, ctas * sizeof(unsigned), st)) != cudaSuccess) return e;
  } else if (p.nseg > 1) {
    if ((e = launch_one<KA, true, false>(p, maps, ctas, st)) != cudaSuccess) return e;
    if ((e = launch_lin_scan(p, st)) != cudaSuccess) return e;
  }
  return grouped ? launch_one<KA, false, true>(p, maps, ctas, st) : launch_one<KA, false, false>(p, maps, ctas, st);
}

}  // namespace

cudaError_t launch_lin_tc(LinArgs& p, int ctas, cudaStream_t st) {
  bool wide = false;
  LinMaps maps;
  for (int i = 0; i < p.nprob; ++i) {
    const LinProb& r = p.pr[i];
    wide = wide || r.a > 64;
    if (!make_map(&maps.m[i][0], r.X, r.a, r.xh, p.T, p.B) || !make_map(&maps.m[i][1], r.Y, r.a, r.yh, p.T, p.B) ||
        !make_map(&maps.m[i][2], r.Z, r.b, r.zh, p.T, p.B) || !make_map(&maps.m[i][3], r.out, r.b, r.oh, p.T, p.B))
      return cudaErrorInvalidValue;
  }
  for (int i = p.nprob; i < kLinProbs; ++i)
    for (int j = 0; j < 4; ++j) maps.m[i][j] = maps.m[0][j];
  return wide ? launch_ka<128>(p, maps, ctas, st) : launch_ka<64>(p, maps, ctas, st);
}

}  // namespace ll
