// Entry points of the linear attention with a decay per head: argument checks, how a call
// is split into units of work, workspace layout.  Contracts are in include/loglinear.h.
#include <cuda_runtime.h>

#include <initializer_list>

#include "lindecay.cuh"

namespace {

using ll::LinArgs;
using ll::LinProb;

constexpr int kSms = 152;  // CTAs of a persistent launch: one per SM

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Whether the current device has an SM for each CTA of a cooperative launch (without a
// device, as if it had).
bool all_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return true;
  return n >= kSms;
}
size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

ll_status check_shape(const ll_shape* s) {
  if (!s) return LL_ERR_NULL;
  if (s->dtype != LL_F32 && s->dtype != LL_BF16) return LL_ERR_DTYPE;
  if (s->batch < 1 || s->heads < 1 || s->heads_per_group < 1 || s->heads % s->heads_per_group) return LL_ERR_SHAPE;
  if (s->d_k < 8 || s->d_k > 128 || s->d_k % 8 || s->d_v < 8 || s->d_v > 128 || s->d_v % 8) return LL_ERR_SHAPE;
  if ((long long)s->batch * s->heads > (1 << 20)) return LL_ERR_SHAPE;
  return LL_OK;
}
ll_status check_seq_shape(const ll_shape* s) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  return s->T < 1 || s->T > (1 << 30) ? LL_ERR_SHAPE : LL_OK;
}

struct Plan {
  LinArgs args;
  size_t off_seg[ll::kLinProbs], off_scratch, off_hand, off_flag;
  size_t bytes;  // workspace: for a wrapped plan also enough for the segmented one in its place
  double est;    // time, in chunks of a wide scan
};
// The wrapped sharing of the same units, where it is estimated to be shorter.
struct Wrap {
  long long turn, total;  // turn 0: it is not
  int abreast;
};

// Work items of a sharing (nwhole, nseg) of all units.
void share_items(LinArgs& p, int units) {
  p.items = p.nwhole + (units - p.nwhole) * p.nseg;
  p.sitems = 0;
  for (int i = 0; i < p.nprob; ++i) {
    LinProb& r = p.pr[i];
    const int w = p.nwhole - r.unit0;
    r.split0 = w < 0 ? 0 : w > r.nunits ? r.nunits : w;
    r.nsplit = r.nunits - r.split0;
    r.sunit0 = p.sitems;
    p.sitems += r.nsplit * r.nh * (p.nseg - 1);
  }
}

// How the units become work items, by estimated time in eighths of what a chunk of a wide
// scan (a > 64) takes on one SM (2 us in bf16; 8 us in fp32, where launches and starts weigh
// less: 2 x 400 tokens, 8 heads of 64 59 -> 19.5 us, 4 x 1000, 16 of 64 133 -> 95):
//  - wrapped: every SM gets an equal share of the line of units, or the longest unit's time
//    where that is more.  Tensor cores only.
//  - segmented: whole units in turn, the last incomplete turn's (all of them when there are
//    fewer units than SMs) cut into segments.  The cut costs a pass over Y and Z first
//    (kState of an output chunk's time per chunk), two more launches (kLaunch chunks), a
//    start per item (kItem) and the prefix over the segments (kSeg each).
// With many units the first needs no extra pass; with fewer than SMs only the second gives
// every SM work.
// Leaves the segmented sharing in p, and the wrapped one in *wrap if that is the shorter.  Returns
// the shorter one's estimate, in such chunks.
double cut_units(LinArgs& p, bool bf16, Wrap* wrap) {
  const double kState = bf16 ? 0.6 : 0.4, kLaunch = bf16 ? 4.0 : 1.0, kItem = bf16 ? 1.0 : 0.5, kSeg = bf16 ? 0.1 : 0.05;
  int units = 0, nh_tail = 1;
  long long line = 0, longest = 0;
  int abreast = 8;  // divides the 152 SMs
  for (int i = 0; i < p.nprob; ++i) {
    LinProb& r = p.pr[i];
    r.nunits = p.B * r.oh * r.tiles;
    r.unit0 = units;
    r.pos0 = line;
    r.cost = (bf16 && r.a <= 64 ? 7 : 8) * r.nh;
    units += r.nunits;
    // units that read the same X and Y: a head's tiles, and the heads of a group where X and
    // Y have one head for the group
    int same = r.tiles * (r.xh != p.H && r.yh != p.H && r.oh == p.H ? p.hpg : 1);
    while (same % abreast) abreast /= 2;
    line += r.cost * p.NC * r.nunits;
    longest = r.cost * p.NC > longest ? r.cost * p.NC : longest;
  }
  const int whole = units / kSms * kSms, rest = units - whole;
  for (int i = 0; i < p.nprob; ++i)
    if (p.pr[i].unit0 + p.pr[i].nunits > whole && p.pr[i].nh > nh_tail) nh_tail = p.pr[i].nh;
  p.nwhole = units;
  p.nseg = 1;
  p.L = p.NC;
  double tail = rest > 0 ? (double)p.NC * nh_tail : 0.0;
  for (int n = 2; rest > 0 && n <= 256 && n <= p.NC; ++n) {
    const int l = (p.NC + n - 1) / n, nseg = (p.NC + l - 1) / l;
    const long long items = (long long)rest * nseg, sitems = (long long)rest * nh_tail * (nseg - 1);
    const double c = (double)((items + kSms - 1) / kSms) * (l * nh_tail + kItem) +
                     (double)((sitems + kSms - 1) / kSms) * (l * kState + kItem) + kLaunch + kSeg * nseg;
    if (c < tail) {
      tail = c;
      p.nwhole = whole;
      p.nseg = nseg;
      p.L = l;
    }
  }
  double head = 0.0;  // the whole turns, each as long as its longest unit
  for (int u = 0; u < whole; u += kSms) {
    long long most = 0;
    for (int i = 0; i < p.nprob; ++i)
      if (p.pr[i].unit0 < u + kSms && p.pr[i].unit0 + p.pr[i].nunits > u && p.pr[i].cost > most) most = p.pr[i].cost;
    head += (double)most / 8.0 * p.NC;
  }
  p.turn = 0;
  share_items(p, units);
  // The wait for a part's state is bounded by 2 s: not for units whose parts may take that (a
  // chunk of every head that is summed takes up to 2.3 us; 2^17 of them 0.3 s).
  constexpr long long kLongest = 8LL << 17;
  const long long even = (line + kSms - 1) / kSms, turn = even > longest ? even : longest;
  *wrap = Wrap{};
  if (bf16 && units > kSms && units % kSms != 0 && longest <= kLongest && turn / 8.0 + 1.0 < head + tail) {
    *wrap = Wrap{turn, line / abreast, abreast};
    return turn / 8.0 + 1.0;
  }
  return head + tail;
}
// p, as cut_units left it, shared out by *w.
void wrap_units(LinArgs& p, const Wrap& w) {
  int units = 0;
  for (int i = 0; i < p.nprob; ++i) {
    p.pr[i].pos0 /= w.abreast;
    units += p.pr[i].nunits;
  }
  p.turn = w.turn;
  p.total = w.total;
  p.abreast = w.abreast;
  p.nwhole = units;
  p.nseg = 1;
  p.L = p.NC;
  share_items(p, units);
}

// Places in the workspace; returns its size.
size_t lay_out(Plan* pl, bool bf16, bool turns) {
  const LinArgs& p = pl->args;
  size_t off = 0;
  for (int i = 0; i < p.nprob; ++i) {
    const LinProb& r = p.pr[i];
    pl->off_seg[i] = off;
    off += a256((size_t)r.nsplit * r.nh * p.nseg * r.a * ll::kLinTile * 4);
  }
  pl->off_scratch = off;
  const int ctas = p.turn > 0 || p.items > kSms ? kSms : p.items;
  if (bf16 && turns) off += a256((size_t)ctas * (p.sub + p.keep) * ll::kLinChunk * ll::kLinTile * 4);
  pl->off_hand = off;
  if (p.turn > 0) off += a256((size_t)(kSms + 1) * p.hpg * ll::kLinChunk * ll::kLinTile * 4);
  pl->off_flag = off;
  if (p.turn > 0) off += a256(kSms * sizeof(unsigned));
  return off;
}

// Completes a plan whose scans' head counts, widths and directions are set; may_wrap false: for a
// stream that has only some of the SMs.  The size of the workspace goes by the shape alone, so
// that it does for either sharing.
void finish_plan(const ll_shape* s, Plan* pl, bool may_wrap) {
  // A group's heads take turns of 16 chunks, so that their fp32 sums (16 x 32 KB a CTA, 80
  // MB on 152 SMs) stay in the 126 MB L2.
  constexpr int kSub = 16;
  LinArgs& p = pl->args;
  const bool bf16 = s->dtype == LL_BF16;
  p.B = s->batch;
  p.T = s->T;
  p.H = s->heads;
  p.hpg = s->heads_per_group;
  p.chunk = bf16 ? ll::kLinChunk : ll::kLinChunk32;
  p.NC = (s->T + p.chunk - 1) / p.chunk;
  p.sub = kSub < p.NC ? kSub : p.NC;
  p.keep = p.NC > p.sub ? p.hpg : 0;
  bool turns = false;  // a pair of heads runs side by side, more of them or an odd number in turns
  for (int i = 0; i < p.nprob; ++i) {
    p.pr[i].tiles = (p.pr[i].b + ll::kLinTile - 1) / ll::kLinTile;
    p.pr[i].nh = p.pr[i].oh == p.H ? 1 : p.hpg;
    turns = turns || p.pr[i].nh > 2;
  }
  Wrap wrap;
  pl->est = cut_units(p, bf16, &wrap);
  pl->bytes = lay_out(pl, bf16, turns);
  if (wrap.turn == 0) return;
  Plan w = *pl;
  wrap_units(w.args, wrap);
  const size_t need = lay_out(&w, bf16, turns), both = need > pl->bytes ? need : pl->bytes;
  if (may_wrap && all_sms()) *pl = w;
  pl->bytes = both;
}

LinProb scan(const void* X, int xh, const void* Y, int yh, const void* Z, int zh, void* out, int oh, int a, int b,
             int rev) {
  LinProb r{};
  r.X = X;
  r.Y = Y;
  r.Z = Z;
  r.out = out;
  r.xh = xh;
  r.yh = yh;
  r.zh = zh;
  r.oh = oh;
  r.a = a;
  r.b = b;
  r.rev = rev;
  return r;
}

void plan_fwd(const ll_shape* s, const void* q, const void* k, const void* v, void* o, Plan* pl) {
  const int H = s->heads, G = H / s->heads_per_group;
  pl->args = LinArgs{};
  pl->args.nprob = 1;
  pl->args.pr[0] = scan(q, G, k, G, v, H, o, H, s->d_k, s->d_v, 0);
  finish_plan(s, pl, true);
}

// The gradients' three scans.  Where the tensor-core kernels pad d_k and d_v to different
// widths (dq and dk run over d_v, dv over d_k) either in one launch, whose stages are laid out
// for the wider (narrow chunks then take 15 % longer), or in two, each with its own remainder
// after the last whole turn of the SMs, whichever is estimated to be shorter.  For d_k = 128,
// d_v = 64, one and two launches: 13 and 25 us (2 x 500 tokens, 8 heads), 120 and 136 (8192, 16),
// 439 and 421 (2 x 8192, 48 in pairs).  Returns the number of launches; they run one after the
// other and share the workspace.
int plan_bwd(const ll_shape* s, const void* q, const void* k, const void* v, const void* dO, void* dq, void* dk,
             void* dv, Plan* pl) {
  constexpr double kMixed = 1.15, kLaunch = 2.0;
  const int H = s->heads, G = H / s->heads_per_group;
  const LinProb pq = scan(dO, H, v, H, k, G, dq, G, s->d_v, s->d_k, 0),
                pk = scan(v, H, dO, H, q, G, dk, G, s->d_v, s->d_k, 1),
                pv = scan(k, G, q, G, dO, H, dv, H, s->d_k, s->d_v, 1);
  auto plan = [&](Plan& x, std::initializer_list<LinProb> scans) {
    x.args = LinArgs{};
    for (const LinProb& r : scans) x.args.pr[x.args.nprob++] = r;
    finish_plan(s, &x, true);
  };
  plan(pl[0], {pq, pk, pv});
  if (s->dtype != LL_BF16 || (s->d_k > 64) == (s->d_v > 64)) return 1;
  Plan a, b;
  plan(a, {pq, pk});
  plan(b, {pv});
  if (pl[0].est * kMixed <= a.est + b.est + kLaunch) return 1;
  pl[0] = a;
  pl[1] = b;
  return 2;
}
size_t bwd_bytes(const Plan* pl, int n) { return n == 2 && pl[1].bytes > pl[0].bytes ? pl[1].bytes : pl[0].bytes; }

cudaError_t launch(const ll_shape* s, Plan* pl, const float* log_a, const int* lengths, void* workspace,
                   cudaStream_t st) {
  LinArgs& p = pl->args;
  p.log_a = log_a;
  p.lengths = lengths;
  char* ws = static_cast<char*>(workspace);
  for (int i = 0; i < p.nprob; ++i) p.pr[i].seg = reinterpret_cast<float*>(ws + pl->off_seg[i]);
  p.scratch = reinterpret_cast<float*>(ws + pl->off_scratch);
  p.hand = reinterpret_cast<float*>(ws + pl->off_hand);
  p.flag = reinterpret_cast<unsigned*>(ws + pl->off_flag);
  return s->dtype == LL_BF16 ? ll::launch_lin_tc(p, kSms, st) : ll::launch_lin_f32(p, st);
}
ll_status run(const ll_shape* s, Plan* pl, const float* log_a, const int* lengths, void* workspace, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  pl->args.status = ll::device_status_word();
  if (!pl->args.status) return LL_ERR_CUDA;
  cudaError_t e = launch(s, pl, log_a, lengths, workspace, st);
  if (e == cudaErrorCooperativeLaunchTooLarge) {
    // the stream or the context has only some of the SMs (a green context, an MPS share): the
    // segmented sharing, whose CTAs do not wait for one another
    cudaGetLastError();
    finish_plan(s, pl, false);
    e = launch(s, pl, log_a, lengths, workspace, st);
  }
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t lindecay_fwd_workspace_bytes(const ll_shape* s) {
  if (check_seq_shape(s) != LL_OK) return 0;
  Plan pl;
  plan_fwd(s, nullptr, nullptr, nullptr, nullptr, &pl);
  return pl.bytes > 0 ? pl.bytes : 16;
}

ll_status lindecay_fwd(const ll_shape* s, const void* q, const void* k, const void* v, const float* log_a,
                       const int* lengths, const float* state_in, void* o, float* state_out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const ll_status st = check_seq_shape(s);
  if (st != LL_OK) return st;
  if (!q || !k || !v || !log_a || !o) return LL_ERR_NULL;
  for (const void* x : {q, k, v, (const void*)o, (const void*)state_in, (const void*)state_out})
    if (!aligned16(x)) return LL_ERR_ALIGN;
  Plan pl;
  plan_fwd(s, q, k, v, o, &pl);
  if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes)) return LL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LL_ERR_ALIGN;
  // other heads and columns still read q and k when an output is written
  if (o == q || o == k) return LL_ERR_SHAPE;
  LinProb& r = pl.args.pr[0];
  r.init = state_in;
  r.init_rs = s->d_v;
  r.init_cs = 1;
  r.fin = state_out;
  return run(s, &pl, log_a, lengths, workspace, stream);
}

size_t lindecay_bwd_workspace_bytes(const ll_shape* s) {
  if (check_seq_shape(s) != LL_OK) return 0;
  Plan pl[2];
  const int n = plan_bwd(s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, pl);
  return bwd_bytes(pl, n) > 0 ? bwd_bytes(pl, n) : 16;
}

ll_status lindecay_bwd(const ll_shape* s, const void* q, const void* k, const void* v, const float* log_a,
                       const int* lengths, const float* state_in, const void* dO, const float* dstate_out, void* dq,
                       void* dk, void* dv, float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  ll_status st = check_seq_shape(s);
  if (st != LL_OK) return st;
  if (!q || !k || !v || !log_a || !dO || !dq || !dk || !dv) return LL_ERR_NULL;
  for (const void* x : {q, k, v, dO, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)state_in,
                        (const void*)dstate_out, (const void*)dstate_in})
    if (!aligned16(x)) return LL_ERR_ALIGN;
  // the scans run side by side: one may still read what another writes
  if (dstate_in && (dstate_in == state_in || dstate_in == dstate_out)) return LL_ERR_SHAPE;
  Plan pl[2];
  const int n = plan_bwd(s, q, k, v, dO, dq, dk, dv, pl);
  if (bwd_bytes(pl, n) > 0 && (!workspace || workspace_bytes < bwd_bytes(pl, n))) return LL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LL_ERR_ALIGN;
  for (const void* g : {dq, dk, dv})
    if (g == q || g == k || g == v || g == dO) return LL_ERR_SHAPE;
  if (dq == dk || dq == dv || dk == dv) return LL_ERR_SHAPE;
  LinProb &pq = pl[0].args.pr[0], &pk = pl[0].args.pr[1], &pv = n == 2 ? pl[1].args.pr[0] : pl[0].args.pr[2];
  pq.init = state_in;
  pk.init = pv.init = dstate_out;
  pq.init_rs = pk.init_rs = 1;  // dq and dk run over the transposed states
  pq.init_cs = pk.init_cs = s->d_v;
  pv.init_rs = s->d_v;
  pv.init_cs = 1;
  pv.fin = dstate_in;
  for (int i = 0; i < n; ++i)
    if ((st = run(s, &pl[i], log_a, lengths, workspace, stream)) != LL_OK) return st;
  return LL_OK;
}

ll_status lindecay_decode_step(const ll_shape* s, const void* q_t, const void* k_t, const void* v_t,
                               const float* log_a, void* o_t, float* states, void* stream) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  if (!q_t || !k_t || !v_t || !log_a || !o_t || !states) return LL_ERR_NULL;
  for (const void* x : {q_t, k_t, v_t, (const void*)o_t, (const void*)states})
    if (!aligned16(x)) return LL_ERR_ALIGN;
  const ll::LinStepArgs d{s->batch, s->heads, s->heads_per_group, s->d_k, s->d_v, q_t, k_t, v_t, log_a, o_t, states};
  const cudaError_t e = ll::launch_lin_step(d, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

}  // extern "C"
