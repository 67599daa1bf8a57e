// Norm of every head of q and k, a weight, and the rotation by position, in one pass over both; the
// gradients.  Contracts are in include/loglinear.h.
//
// Bound by memory: a value is read once and written once (backward: two read).  A head lies in 1 to
// 32 lanes, each with eight values that hold the rotation's pairs whole, so no value changes lanes,
// and two pairs go through an instruction.  A warp takes a token and walks its heads, for which
// angles are made once, with the next heads' values on their way.
//
// 32768 tokens of 24 + 24 heads of 128 131 us (6.2 TB/s, 91 % of a copy's rate), gradients of 16396
// tokens of 32 + 8 heads, half of each turned, 94 us (5.4, 79 %; 128 registers leave 16 warps an SM).  On the way there: two
// values a lane and a product each, with a test for every head, 184 and 164 us; packed pairs 154 and
// 106; weights without bank conflicts and sums without a test a step 140 and 96; pointers that step from
// head to head instead of being made of the head's number 176; four heads on their way, more than
// registers hold, 170.
//
// Angles: position times frequency modulo a turn, as 64-bit integers (the frequency in 2^-64 turns),
// so a position of a million is as exact as one of ten: a unit of the frequency for each of up to 2^31 positions
// and the low half that is left out are 1.5 steps of 2^-32 turns, 2^-28.7 radians.  What is left of the nearest
// quarter turn is rounded to fp32 (2^-25.3 radians), and its sine and cosine are fp32's own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "headrope.cuh"
#include "launch_util.cuh"
#include "ptx.cuh"

namespace ll {
namespace {

// ---- values ------------------------------------------------------------------------------
using ptx::add2;
using ptx::fma2;
using ptx::mul2;
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A lane's eight values of a head, in the order of the rotation's pairs: values n and n + 4 are a
// pair, so v.p[0], v.p[1] turn with v.p[2], v.p[3], two pairs an instruction.
struct Eight {
  float2 p[4];
};

// Where they lie.  kVec (d and rot are multiples of 8): in the half layout two runs of four, rot/2
// apart (one after the other past the rotated part), interleaved one run of eight.  Otherwise each
// for itself, -1 for none.
template <bool kVec, bool kHalf>
struct Place {
  int at[kVec ? 2 : 8];
  __device__ __forceinline__ Place(int unit, int d, int rot) {
    if (kVec) {
      const bool turned = kHalf && 8 * unit < rot;
      at[0] = 8 * unit >= d ? -1 : turned ? 4 * unit : 8 * unit;
      at[1] = turned ? 4 * unit + (rot >> 1) : 8 * unit + 4;
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int pair = 4 * unit + n, a = kHalf && 2 * pair < rot ? pair : 2 * pair;
        const int b = kHalf && 2 * pair < rot ? pair + (rot >> 1) : 2 * pair + 1;
        at[n] = a < d ? a : -1;
        at[n + 4] = b < d ? b : -1;
      }
    }
  }
  __device__ __forceinline__ bool any() const { return at[0] >= 0; }
  // whether pair n turns.  kVec: a lane's pairs all do or none does.
  static __device__ __forceinline__ bool turns(int unit, int n, int rot) { return 8 * unit + (kVec ? 0 : 2 * n) < rot; }
  // where value e sits, -1 (kVec: with any() alone) for none
  __device__ __forceinline__ int of(int e) const {
    if constexpr (!kVec) return at[e];
    else if constexpr (kHalf) return at[e / 4] + e % 4;
    else return at[0] + 2 * (e % 4) + e / 4;
  }
};

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pair_bf(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ void put_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put_one(float* p, float v) { *p = v; }

// The eight as they lie in memory (32 bits of bf16 pairs or one fp32 each), their loads and stores.
template <typename T, bool kVec, bool kHalf>
struct Held {
  uint32_t w[sizeof(T) == 2 && kVec ? 4 : 8];
  __device__ __forceinline__ void load(const T* x, const Place<kVec, kHalf>& at) {
    if constexpr (!kVec) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = at.at[e] >= 0 ? __float_as_uint(one(x + at.at[e])) : 0u;
    } else if constexpr (sizeof(T) == 2 && !kHalf) {
      const uint4 r = __ldcs(reinterpret_cast<const uint4*>(x + at.at[0]));
      w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
    } else if constexpr (sizeof(T) == 2) {
      const uint2 r = __ldcs(reinterpret_cast<const uint2*>(x + at.at[0])), q = __ldcs(reinterpret_cast<const uint2*>(x + at.at[1]));
      w[0] = r.x, w[1] = r.y, w[2] = q.x, w[3] = q.y;
    } else {
      const uint4 r = __ldcs(reinterpret_cast<const uint4*>(x + at.at[0])), q = __ldcs(reinterpret_cast<const uint4*>(x + at.at[1]));
      w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w, w[4] = q.x, w[5] = q.y, w[6] = q.z, w[7] = q.w;
    }
  }
  __device__ __forceinline__ Eight get() const {
    Eight v;
    if constexpr (!kVec || (sizeof(T) == 4 && kHalf)) {
#pragma unroll
      for (int n = 0; n < 4; ++n) v.p[n] = make_float2(__uint_as_float(w[2 * n]), __uint_as_float(w[2 * n + 1]));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
        v.p[n] = make_float2(__uint_as_float(w[4 * (n % 2) + n / 2]), __uint_as_float(w[4 * (n % 2) + n / 2 + 2]));
    } else if constexpr (kHalf) {
#pragma unroll
      for (int n = 0; n < 4; ++n) v.p[n] = make_float2(low(w[n]), high(w[n]));
    } else {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        v.p[n] = make_float2(low(w[2 * n]), low(w[2 * n + 1]));
        v.p[n + 2] = make_float2(high(w[2 * n]), high(w[2 * n + 1]));
      }
    }
    return v;
  }
  static __device__ __forceinline__ void store(T* x, const Place<kVec, kHalf>& at, const Eight& v) {
    if constexpr (!kVec) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at.at[e] >= 0) put_one(x + at.at[e], e % 2 ? v.p[e / 2].y : v.p[e / 2].x);
    } else if constexpr (sizeof(T) == 2 && kHalf) {
      __stcs(reinterpret_cast<uint2*>(x + at.at[0]), make_uint2(pair_bf(v.p[0].x, v.p[0].y), pair_bf(v.p[1].x, v.p[1].y)));
      __stcs(reinterpret_cast<uint2*>(x + at.at[1]), make_uint2(pair_bf(v.p[2].x, v.p[2].y), pair_bf(v.p[3].x, v.p[3].y)));
    } else if constexpr (sizeof(T) == 2) {
      __stcs(reinterpret_cast<uint4*>(x + at.at[0]), make_uint4(pair_bf(v.p[0].x, v.p[2].x), pair_bf(v.p[0].y, v.p[2].y),
                                                                pair_bf(v.p[1].x, v.p[3].x), pair_bf(v.p[1].y, v.p[3].y)));
    } else if constexpr (kHalf) {
      __stcs(reinterpret_cast<float4*>(x + at.at[0]), make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y));
      __stcs(reinterpret_cast<float4*>(x + at.at[1]), make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y));
    } else {
      __stcs(reinterpret_cast<float4*>(x + at.at[0]), make_float4(v.p[0].x, v.p[2].x, v.p[0].y, v.p[2].y));
      __stcs(reinterpret_cast<float4*>(x + at.at[1]), make_float4(v.p[1].x, v.p[3].x, v.p[1].y, v.p[3].y));
    }
  }
};

// ---- angles ------------------------------------------------------------------------------
// inv_freq (radians a position) in 2^-64 turns a position, modulo a turn: its mantissa times
// floor(2^128 / (2 pi)), shifted by its exponent.  From 2^64 on that constant has too few digits.
__device__ __forceinline__ unsigned long long turns_of(float inv_freq) {
  const unsigned bits = __float_as_uint(inv_freq), field = (bits >> 23) & 255u;
  const unsigned long long m = field ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  constexpr unsigned long long kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;
  const unsigned long long p0 = m * kLow, carry = __umul64hi(m, kLow), low = m * kHigh;
  const unsigned long long p1 = low + carry, p2 = __umul64hi(m, kHigh) + (p1 < low ? 1ull : 0ull);
  // the product's 152 bits stand for turns of 2^(exponent - 128): of its bits from `shift` on, 64
  const int shift = 64 - ((int)(field ? field : 1u) - 150), in = shift & 63;
  const unsigned long long a = shift < 0 ? 0ull : shift < 64 ? p0 : shift < 128 ? p1 : shift < 192 ? p2 : 0ull;
  const unsigned long long b = shift < 0 ? 0ull : shift < 64 ? p1 : shift < 128 ? p2 : 0ull;
  const unsigned long long t = in ? (a >> in) | (b << (64 - in)) : a;
  return bits >> 31 ? 0ull - t : t;
}
__device__ __forceinline__ void angle_of(unsigned long long freq, int pos, float& c, float& s) {
  const unsigned hi = (unsigned)((freq * (unsigned long long)(long long)pos) >> 32);
  const unsigned quarter = (hi + 0x20000000u) >> 30;
  const int rest = (int)(hi - (quarter << 30));  // 2^-32 turns, at most an eighth
  float sn, cs;
  sincospif((float)rest * 4.656612873077393e-10f, &sn, &cs);  // in half turns
  const bool odd = quarter & 1u;
  s = odd ? cs : sn;
  c = odd ? sn : cs;
  if (quarter == 2u || quarter == 3u) s = -s;
  if (quarter == 1u || quarter == 2u) c = -c;
}
// The turn of the four pairs a lane holds, by c, s and to, as `minus`, -s.
struct Turn {
  float2 c[2], s[2], minus[2];
};
__device__ __forceinline__ void turned(Eight& v, const Turn& t) {
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float2 a = v.p[n], b = v.p[n + 2];
    v.p[n] = fma2(a, t.c[n], mul2(b, t.minus[n]));
    v.p[n + 2] = fma2(a, t.s[n], mul2(b, t.c[n]));
  }
}
// The same of one pair of pairs where `on`; as they are otherwise.
__device__ __forceinline__ void turned_if(bool on, float2& a, float2& b, float2 c, float2 s, float2 minus) {
  asm("{\n\t.reg .pred p;\n\t.reg .b64 a, b, c, s, m, x, y;\n\tsetp.ne.b32 p, %10, 0;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\tmov.b64 s, {%6, %7};\n\t"
      "mov.b64 m, {%8, %9};\n\tmul.rn.f32x2 x, b, m;\n\tmul.rn.f32x2 y, b, c;\n\t"
      "@p fma.rn.f32x2 b, a, s, y;\n\t@p fma.rn.f32x2 a, a, c, x;\n\t"
      "mov.b64 {%0, %1}, a;\n\tmov.b64 {%2, %3}, b;\n\t}"
      : "+f"(a.x), "+f"(a.y), "+f"(b.x), "+f"(b.y)
      : "f"(c.x), "f"(c.y), "f"(s.x), "f"(s.y), "f"(minus.x), "f"(minus.y), "r"((unsigned)on));
}
__device__ __forceinline__ float sum_of(const float2& x) { return x.x + x.y; }
// Sums over a head's lanes; for the usual sizes without a test for each step.
template <int S, int N>
__device__ __forceinline__ void lane_sums(float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], 1 << i);
}
template <int N>
__device__ __forceinline__ void head_sums(float (&x)[N], int tph_log) {
  if (tph_log == 4) {
    lane_sums<4>(x);
  } else if (tph_log == 3) {
    lane_sums<3>(x);
  } else {
    for (int i = 0; i < tph_log; ++i)
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], 1 << i);
  }
}
// Of what is at least the smallest normal number (with an epsilon of 0, rows below 1e-19 count as
// that small): the special functions' instruction itself.  NaN stays NaN.
__device__ __forceinline__ float inverse_norm(float ss, const HrArgs& p) {
  float x = fmaf(ss, p.norm == HR_RMS ? p.inv_d : 1.f, p.eps);
  asm("max.NaN.f32 %0, %0, 0f00800000;" : "+f"(x));
  asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}

// Frequencies, and the weights times the scale, of each lane's values in its order: all lanes' first
// four, then their second.
struct Shared {
  unsigned long long freq[kHrMaxDim / 2];
  float w[2][kHrMaxDim];
};

// What is known of a launch's heads: nothing; there is a norm, and part of a head turns; there is a norm, and
// all of it turns.  (32768 tokens of 48 heads with a test for the norm and the rotation 140 us, with one for the
// part that turns 137, without any 131.)
enum Heads { kAnyHeads, kPartHeads, kWholeHeads };

// What both kernels have: a warp's rows, a lane's place in them.  kFull: every lane has a head's
// values in every step.
template <typename T, bool kHalf, bool kVec>
struct Lane {
  const HrArgs& p;
  const Shared& sh;
  int slot, unit, hpw;  // a step's heads of a row; a lane's of them, and its place in the head
  bool turns[kVec ? 1 : 4];  // which of its pairs do
  Place<kVec, kHalf> at;
  unsigned long long freq[4];
  long long row;
  bool in;       // the row is there
  int from, to;  // of a row's steps

  __device__ __forceinline__ Lane(const HrArgs& p, const Shared& s)
      : p(p), sh(s), slot(((threadIdx.x & 31) >> p.tph_log) & ((32 >> p.tph_log >> p.rpw_log) - 1)),
        unit(threadIdx.x & ((1 << p.tph_log) - 1)), hpw(32 >> p.tph_log >> p.rpw_log), at(unit, p.d, p.rot) {
#pragma unroll
    for (int n = 0; n < (kVec ? 1 : 4); ++n) turns[n] = Place<kVec, kHalf>::turns(unit, n, p.rot);
  }
  // The pairs that turn by t.  The others stay: a product with the sine of 0 would hand a value that is not
  // finite on to its partner.  Forward by predicates (139.8 us for 32768 tokens of 48 half-turned heads, 141.9 as a
  // branch, 132.6 with those products), backward as a branch (94.0 for the gradients of 16396 of 40, 94.6, 92.6).
  template <Heads kHeads, bool kBranch>
  __device__ __forceinline__ void turn(Eight& v, const Turn& t) const {
    if constexpr (kHeads == kWholeHeads) {
      turned(v, t);
    } else if constexpr (kVec && kBranch) {
      if (turns[0]) turned(v, t);
    } else if constexpr (kVec) {
#pragma unroll
      for (int n = 0; n < 2; ++n) turned_if(turns[0], v.p[n], v.p[n + 2], t.c[n], t.s[n], t.minus[n]);
    } else {
      const Eight was = v;
      turned(v, t);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (turns[n]) continue;
        (n % 2 ? v.p[n / 2].y : v.p[n / 2].x) = n % 2 ? was.p[n / 2].y : was.p[n / 2].x;
        (n % 2 ? v.p[n / 2 + 2].y : v.p[n / 2 + 2].x) = n % 2 ? was.p[n / 2 + 2].y : was.p[n / 2 + 2].x;
      }
    }
  }
  // Fills the shared part, for all.
  __device__ __forceinline__ void prepare(Shared& s) {
    for (int j = threadIdx.x; j < p.rot / 2; j += blockDim.x) s.freq[j] = turns_of(p.inv_freq[j]);
    if (threadIdx.x < (1u << p.tph_log))  // the first lane of each place
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = at.any() ? at.of(e) : -1;
        s.w[0][kHrMaxDim / 2 * (e / 4) + 4 * unit + e % 4] = j < 0 ? 0.f : (p.w_q ? p.w_q[j] : 1.f) * p.scale_q;
        s.w[1][kHrMaxDim / 2 * (e / 4) + 4 * unit + e % 4] = j < 0 ? 0.f : (p.w_k ? p.w_k[j] : 1.f) * p.scale_k;
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 4; ++n) freq[n] = 4 * unit + n < p.rot / 2 ? s.freq[4 * unit + n] : 0ull;
  }
  __device__ __forceinline__ void take(long long item, int steps) {
    from = 0;
    to = steps;
    if (p.splits > 1) {
      row = item / p.splits;
      const int share = (int)(item - row * p.splits);
      from = (int)((unsigned)steps * (unsigned)share / (unsigned)p.splits);
      to = (int)((unsigned)steps * (unsigned)(share + 1) / (unsigned)p.splits);
    } else {
      row = (item << p.rpw_log) + (((threadIdx.x & 31) >> p.tph_log) / hpw);
    }
    in = row < p.rows;
    if (!in) row = p.rows - 1;
  }
  __device__ __forceinline__ Turn angles(bool back) const {
    Turn t;
    float c[4], s[4];
    const int pos = p.positions ? __ldg(p.positions + row) : (int)((unsigned)row % (unsigned)p.T);
#pragma unroll
    for (int n = 0; n < 4; ++n) angle_of(freq[n], pos, c[n], s[n]);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      t.c[n] = make_float2(c[2 * n], c[2 * n + 1]);
      t.s[n] = make_float2(s[2 * n], s[2 * n + 1]);
      t.minus[n] = mul2(t.s[n], both(-1.f));
      if (back) {
        const float2 x = t.s[n];
        t.s[n] = t.minus[n];
        t.minus[n] = x;
      }
    }
    return t;
  }
  __device__ __forceinline__ Eight weights(int side) const {
    Eight w;
    const float4 a = *reinterpret_cast<const float4*>(&sh.w[side][4 * unit]);
    const float4 b = *reinterpret_cast<const float4*>(&sh.w[side][kHrMaxDim / 2 + 4 * unit]);
    w.p[0] = make_float2(a.x, a.y), w.p[1] = make_float2(a.z, a.w), w.p[2] = make_float2(b.x, b.y), w.p[3] = make_float2(b.z, b.w);
    return w;
  }
};

template <typename T>
constexpr int kHrFwdAhead = sizeof(T) == 2 ? 3 : 2;  // heads a lane has on the way
template <typename T>
constexpr int kHrBwdAhead = sizeof(T) == 2 ? 4 : 2;
constexpr int kHrFwdCtas = 3;  // CTAs per SM, all of a launch's running at once
constexpr int kHrBwdCtas = 2;

// ---- forward -----------------------------------------------------------------------------
// Steps of a row: of q's heads, then of k's.
template <typename T, bool kHalf, bool kVec, bool kFull, Heads kHeads>
__global__ void __launch_bounds__(kHrWarps * 32, kHrFwdCtas) hr_fwd_kernel(HrArgs p) {
  __shared__ __align__(16) Shared sh;
  Lane<T, kHalf, kVec> l(p, sh);
  const int steps_q = (p.gq + l.hpw - 1) / l.hpw, steps = steps_q + (p.gk + l.hpw - 1) / l.hpw;
  const long long items = ((p.rows + (1 << p.rpw_log) - 1) >> p.rpw_log) * p.splits;
  bool ready = false;  // what the CTA shares is made behind the first loads
  for (long long it = (long long)blockIdx.x * kHrWarps + (threadIdx.x >> 5); it < items || !ready;
       it += (long long)gridDim.x * kHrWarps) {
    l.take(it < items ? it : 0, it < items ? steps : 0);
    // the place of step i's head, in q or in k
    auto side_of = [&](int i) { return i >= steps_q; };
    auto there = [&](int i) {
      if (kFull) return true;
      return l.in && l.at.any() && (side_of(i) ? (i - steps_q) * l.hpw + l.slot < p.gk : i * l.hpw + l.slot < p.gq);
    };
    const T *q = static_cast<const T*>(p.q) + (l.row * p.gq + l.slot) * p.d,
            *k = static_cast<const T*>(p.k) + (l.row * p.gk + l.slot - steps_q * l.hpw) * p.d;
    T *qo = static_cast<T*>(p.q_out) + (l.row * p.gq + l.slot) * p.d,
      *ko = static_cast<T*>(p.k_out) + (l.row * p.gk + l.slot - steps_q * l.hpw) * p.d;
    const int step = l.hpw * p.d;
    constexpr int N = kHrFwdAhead<T>;
    Held<T, kVec, kHalf> x[2][N];
    auto load = [&](int i0, Held<T, kVec, kHalf>* to) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i0 + i < l.to && there(i0 + i)) to[i].load((side_of(i0 + i) ? k : q) + (i0 + i) * step, l.at);
    };
    auto work = [&](int i0, const Held<T, kVec, kHalf>* from, const Turn& t) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i0 + i >= l.to) break;
        const bool has = there(i0 + i), in_k = side_of(i0 + i);
        Eight v{};
        if (has) v = from[i].get();
        float r = 1.f;
        if (kHeads != kAnyHeads || p.norm != HR_NONE) {
          float2 ss = mul2(v.p[0], v.p[0]);
#pragma unroll
          for (int n = 1; n < 4; ++n) ss = fma2(v.p[n], v.p[n], ss);
          float sum[1] = {sum_of(ss)};
          head_sums(sum, p.tph_log);
          r = inverse_norm(sum[0], p);
        }
        const Eight w = l.weights(in_k);
#pragma unroll
        for (int n = 0; n < 4; ++n) v.p[n] = mul2(v.p[n], mul2(w.p[n], both(r)));
        if (kHeads != kAnyHeads || p.rot) l.template turn<kHeads, false>(v, t);
        if (has) Held<T, kVec, kHalf>::store((in_k ? ko : qo) + (i0 + i) * step, l.at, v);
      }
    };
    load(l.from, x[0]);
    if (!ready) l.prepare(sh);
    ready = true;
    if (l.from >= l.to) continue;
    Turn t;
    if (kHeads != kAnyHeads || p.rot) t = l.angles(false);
    for (int i0 = l.from; i0 < l.to; i0 += 2 * N) {
      load(i0 + N, x[1]);
      work(i0, x[0], t);
      load(i0 + 2 * N, x[0]);
      work(i0 + N, x[1], t);
    }
  }
}

// ---- backward ----------------------------------------------------------------------------
// With u = R^-1 dy, g = u w scale and r the inverse norm: dw += u (scale r) x, and
// dx = r (g - x r (r mean(g x))), the sum in place of the mean for l2; both sums in one round.  r
// times its sum first: r^2 alone leaves fp32's range where x is far from 1.  A lane keeps its eight
// values' share of dw over all of its heads.
template <typename T, bool kHalf, bool kVec, bool kFull, Heads kHeads>
__global__ void __launch_bounds__(kHrWarps * 32, kHrBwdCtas) hr_bwd_kernel(HrArgs p) {
  __shared__ __align__(16) Shared sh;
  __shared__ float s_dw[kHrWarps][kHrMaxDim];
  Lane<T, kHalf, kVec> l(p, sh);
  const int steps_q = (p.gq + l.hpw - 1) / l.hpw, steps = steps_q + (p.gk + l.hpw - 1) / l.hpw;
  l.prepare(sh);
  ptx::griddep_launch_dependents();
  Eight dw[2]{};
  const float mean = p.norm == HR_RMS ? p.inv_d : 1.f;
  const long long items = ((p.rows + (1 << p.rpw_log) - 1) >> p.rpw_log) * p.splits;
  for (long long it = (long long)blockIdx.x * kHrWarps + (threadIdx.x >> 5); it < items;
       it += (long long)gridDim.x * kHrWarps) {
    l.take(it, steps);
    Turn t;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int lo = side ? max(l.from - steps_q, 0) : l.from, hi = side ? l.to - steps_q : min(l.to, steps_q);
      if (lo >= hi) continue;
      const int G = side ? p.gk : p.gq;
      const long long at = (l.row * G + l.slot) * p.d;
      const T* x0 = static_cast<const T*>(side ? p.k : p.q) + at;
      const T* y0 = static_cast<const T*>(side ? p.dk : p.dq) + at;
      T* o0 = static_cast<T*>(side ? p.k_out : p.q_out) + at;
      const int step = l.hpw * p.d;
      const float scale = side ? p.scale_k : p.scale_q;
      const Eight w = l.weights(side);
      for (int i0 = lo; i0 < hi; i0 += kHrBwdAhead<T>) {
        Held<T, kVec, kHalf> x[kHrBwdAhead<T>], y[kHrBwdAhead<T>];
#pragma unroll
        for (int i = 0; i < kHrBwdAhead<T>; ++i)
          if (i0 + i < hi && (kFull || (l.in && l.at.any() && (i0 + i) * l.hpw + l.slot < G))) {
            x[i].load(x0 + (i0 + i) * step, l.at);
            y[i].load(y0 + (i0 + i) * step, l.at);
          }
        if ((kHeads != kAnyHeads || p.rot) && (side ? max(l.from, steps_q) : l.from) == l.from && i0 == lo) t = l.angles(true);
#pragma unroll
        for (int i = 0; i < kHrBwdAhead<T>; ++i) {
          if (i0 + i >= hi) break;
          const bool has = kFull || (l.in && l.at.any() && (i0 + i) * l.hpw + l.slot < G);
          Eight v{}, u{};
          if (has) {
            v = x[i].get();
            u = y[i].get();
          }
          if (kHeads != kAnyHeads || p.rot) l.template turn<kHeads, true>(u, t);
          Eight g;
#pragma unroll
          for (int n = 0; n < 4; ++n) g.p[n] = mul2(u.p[n], w.p[n]);
          float r = 1.f;
          if (kHeads != kAnyHeads || p.norm != HR_NONE) {  // without a norm x has no part in dx, not even as 0 times an infinity
            float2 ss = mul2(v.p[0], v.p[0]), gx = mul2(g.p[0], v.p[0]);
#pragma unroll
            for (int n = 1; n < 4; ++n) {
              ss = fma2(v.p[n], v.p[n], ss);
              gx = fma2(g.p[n], v.p[n], gx);
            }
            float sums[2] = {sum_of(ss), sum_of(gx)};
            head_sums(sums, p.tph_log);
            r = inverse_norm(sums[0], p);
            const float k = -(r * (r * (sums[1] * mean)));
#pragma unroll
            for (int n = 0; n < 4; ++n) g.p[n] = mul2(fma2(v.p[n], both(k), g.p[n]), both(r));
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) dw[side].p[n] = fma2(mul2(u.p[n], both(scale * r)), v.p[n], dw[side].p[n]);
          if (has) Held<T, kVec, kHalf>::store(o0 + (i0 + i) * step, l.at, g);
        }
      }
    }
  }
  if (!p.part) return;
  // the heads of a warp add up over its slots, then the warps in order
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float sum = e % 2 ? dw[side].p[e / 2].y : dw[side].p[e / 2].x;
      for (int o = 1 << p.tph_log; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int j = l.at.any() ? l.at.of(e) : -1;
      if ((threadIdx.x & 31) == l.unit && j >= 0) s_dw[threadIdx.x >> 5][j] = sum;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < p.d; j += blockDim.x) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kHrWarps; ++w) sum += s_dw[w][j];
      p.part[((size_t)blockIdx.x * 2 + side) * p.d + j] = sum;
    }
  }
}

// dw_q and dw_k from the CTAs' partials, in a fixed order.  32 values by 32 threads each.
__global__ void __launch_bounds__(1024) hr_sum_kernel(const float* part, float* dw_q, float* dw_k, int ctas, int d) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = blockIdx.x * 32 + lane, side = blockIdx.y;
  float* out = side ? dw_k : dw_q;
  ptx::griddep_wait();
  if (!out) return;
  float acc = 0.f;
  if (j < d)
    for (int r = w; r < ctas; r += 32) acc += part[((size_t)r * 2 + side) * d + j];
  s[w][lane] = acc;
  __syncthreads();
  if (w == 0 && j < d) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) sum += s[k][lane];
    out[j] = sum;
  }
}

// ---- launches ----------------------------------------------------------------------------
// Lanes of a head, and how many warps share a row: as many as give every SM its 16 warps.  Where rows
// have so few heads that the lanes hold several rows of them, and rows are many, a warp takes several
// (115000 rows of 3 + 1 heads of 8, backward, 145 us -> 30).
int heads_at_once(int d) {
  int lanes = 1;
  while (lanes < (d + 7) / 8) lanes *= 2;
  return 32 / lanes;
}
void spread(HrArgs& p) {
  const int hpw = heads_at_once(p.d), most = p.gq > p.gk ? p.gq : p.gk;
  p.tph_log = 0;
  while (32 >> p.tph_log > hpw) ++p.tph_log;
  p.rpw_log = 0;
  while (hpw >> (p.rpw_log + 1) >= most && p.rows >> (p.rpw_log + 1) >= kHrSms * 16) ++p.rpw_log;
  const int at_once = hpw >> p.rpw_log, steps = (p.gq + at_once - 1) / at_once + (p.gk + at_once - 1) / at_once;
  const long long want = (kHrSms * 16 + p.rows - 1) / p.rows;
  p.splits = (int)(p.rpw_log || want < 1 ? 1 : want > steps ? steps : want);
}
int grid_of(const HrArgs& p, int most) {
  const long long items = ((p.rows + (1 << p.rpw_log) - 1) >> p.rpw_log) * p.splits;
  const long long ctas = (items + kHrWarps - 1) / kHrWarps;
  return (int)(ctas < most ? ctas : most);
}

template <template <typename, bool, bool, bool, Heads> class K>
cudaError_t choose(const HrArgs& p, int layout, bool bf16, int grid, cudaStream_t st) {
  const bool vec = p.d % 8 == 0 && p.rot % 8 == 0, half = layout == HR_HALF;
  const int hpw = 32 >> p.tph_log;
  const bool full = vec && p.rpw_log == 0 && p.d / 8 == 1 << p.tph_log && p.gq % hpw == 0 && p.gk % hpw == 0;
  const bool usual = p.norm != HR_NONE && p.rot > 0;
#define LL_HR(T, H)                                                               \
  return full && usual && p.rot == p.d ? K<T, H, true, true, kWholeHeads>::run(p, grid, st) \
         : full && usual               ? K<T, H, true, true, kPartHeads>::run(p, grid, st)  \
         : full                        ? K<T, H, true, true, kAnyHeads>::run(p, grid, st)   \
         : vec                         ? K<T, H, true, false, kAnyHeads>::run(p, grid, st)  \
                                       : K<T, H, false, false, kAnyHeads>::run(p, grid, st)
  if (bf16) {
    if (half) LL_HR(__nv_bfloat16, true);
    LL_HR(__nv_bfloat16, false);
  }
  if (half) LL_HR(float, true);
  LL_HR(float, false);
#undef LL_HR
}
template <typename T, bool kHalf, bool kVec, bool kFull, Heads kHeads>
struct Fwd {
  static cudaError_t run(const HrArgs& p, int grid, cudaStream_t st) {
    hr_fwd_kernel<T, kHalf, kVec, kFull, kHeads><<<grid, kHrWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
  }
};
template <typename T, bool kHalf, bool kVec, bool kFull, Heads kHeads>
struct Bwd {
  static cudaError_t run(const HrArgs& p, int grid, cudaStream_t st) {
    hr_bwd_kernel<T, kHalf, kVec, kFull, kHeads><<<grid, kHrWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_hr_fwd(HrArgs p, int layout, bool bf16, cudaStream_t st) {
  spread(p);
  const cudaError_t e = choose<Fwd>(p, layout, bf16, grid_of(p, kHrSms * kHrFwdCtas), st);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_hr_bwd(HrArgs p, int layout, bool bf16, cudaStream_t st) {
  spread(p);
  static_assert(kHrSms * kHrBwdCtas <= kHrMaxParts, "the workspace has a row of partials for each CTA");
  const int grid = grid_of(p, kHrSms * kHrBwdCtas);
  cudaError_t e = choose<Bwd>(p, layout, bf16, grid, st);
  if (e != cudaSuccess) return e;
  note_launch();
  if (!p.part) return cudaSuccess;
  e = launch_ahead(hr_sum_kernel, dim3((p.d + 31) / 32, 2), 1024, 0, st, p.part, p.dw_q, p.dw_k, grid, p.d);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ll
