// Entry points of the gated feed-forward block: argument checks, workspace layout and the lists of
// products.  Contracts are in include/loglinear.h.
#include <cuda_runtime.h>

#include <initializer_list>

#include "ffgate.cuh"

namespace {

using ll::FfArgs;
using ll::FfMaps;
using ll::FfProb;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t a256(size_t x) { return (x + 255) & ~size_t(255); }
int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

ll_status check_shape(const ffgate_shape* s) {
  if (!s) return LL_ERR_NULL;
  if (s->dtype != LL_F32 && s->dtype != LL_BF16) return LL_ERR_DTYPE;
  if (s->rows < 1 || s->rows > (1 << 24) || s->dim < 8 || s->dim > (1 << 20) || s->dim % 8) return LL_ERR_SHAPE;
  if (s->ff < 8 || s->ff > (1 << 20) || s->ff % 8) return LL_ERR_SHAPE;
  if (s->act != FF_IDENTITY && s->act != FF_SILU && s->act != FF_SIGMOID && s->act != FF_GELU) return LL_ERR_SHAPE;
  return LL_OK;
}

// Few rows of the forward go through the kernel that streams the weights.
bool streamed(const ffgate_shape* s) {
  return s->rows <= (s->dtype == LL_BF16 ? ll::kFfStreamRows : ll::kFfStreamRowsF32);
}

// Blocks of 64 summed values take a pair 0.27 us, in two parts 1.3 and in three 1.6, of a tile with 256
// columns; the
// launch that joins the sums of shared tiles costs some 4 us.  An item's way out counts for kWayOut blocks,
// and an item has kLeast at least where a tile is shared.
constexpr int kWayOut = 4, kLeast = 8;
constexpr double kJoinUs = 4.0;
double block_us(bool f32, bool bwd) { return !f32 ? 0.27 : bwd ? 1.6 : 1.3; }

// Columns of the forward's tiles: 128 keep the tensor cores fed best, but where there are few tiles the
// 76 pairs of CTAs may be done in fewer or shorter turns with narrower ones, or with shared ones.  Below
// 56 columns a block takes no less time (its loads' issue: 0.14 us with 16 columns, 0.24 with 96, 0.30
// with 128).
int gated_width(const ffgate_shape* s) {
  const int blocks = ceil_div(s->dim, 64);
  const double block = block_us(s->dtype == LL_F32, false) / 136;
  int best = 128;
  double least = 1e30;
  for (int width = 16; width <= 128; width += 16) {
    const long long tiles = (long long)ceil_div(s->rows, 256) * ceil_div(s->ff, width);
    const double columns = (width > 56 ? width : 56) + 8;
    for (int splits = 1; splits == 1 || (splits * tiles <= 152 && splits * kLeast <= blocks); splits += (splits + 3) / 4) {
      const double us = (double)((splits * tiles + 75) / 76) * (ceil_div(blocks, splits) + kWayOut) * columns * block +
                        (splits > 1 ? kJoinUs : 0);
      if (us < least) {
        best = width;
        least = us;
      }
    }
  }
  return best;
}

// Adds a problem of m rows and n columns of output, summed over `pairs` times k values.
FfProb& add_problem(FfArgs& p, long long m, long long n, long long k, int columns, int pairs) {
  FfProb& r = p.prob[p.probs++];
  r = FfProb{};
  r.rows = (int)m;
  r.cols = (int)n;
  r.tiles_m = ceil_div(m, 256);
  r.tiles_n = ceil_div(n, columns);
  r.kblocks = ceil_div(k, 64);
  r.width = columns;
  r.out_gate = r.out_up = -1;
  r.pairs = pairs;
  return r;
}
// Blocks of the pair of CTAs that has most of them, an item's way out among them: the items go round the 76
// pairs in their order, so each problem adds whole turns and a run of pairs with one item more, and the
// most lies where a run begins.
long long most_blocks(const FfArgs& p) {
  long long all = 0, most = 0;
  int first[ll::kFfProbs], more[ll::kFfProbs], next = 0;
  for (int i = 0; i < p.probs; ++i) {
    const FfProb& r = p.prob[i];
    const long long items = (long long)r.tiles_m * r.tiles_n * r.splits;
    all += items / 76 * (r.share + kWayOut);
    first[i] = next;
    more[i] = (int)(items % 76);
    next = (next + more[i]) % 76;
  }
  for (int j = 0; j < p.probs; ++j) {
    long long here = 0;
    for (int i = 0; i < p.probs; ++i)
      if ((first[j] - first[i] + 76) % 76 < more[i]) here += p.prob[i].share + kWayOut;
    most = here > most ? here : most;
  }
  return all + most;
}
void share(FfProb& r, int splits) {
  r.share = ceil_div(r.pairs * r.kblocks, splits);
  r.splits = ceil_div(r.pairs * r.kblocks, r.share);
}
// The most items that a tile may be shared by: 152 of the problem, with kLeast blocks at least.
int most_splits(const FfProb& r, double block) {
  const int tiles = r.tiles_m * r.tiles_n, blocks = r.pairs * r.kblocks;
  if (tiles > 76 || (blocks - kLeast) * block < kJoinUs) return 1;
  const int most = 152 / tiles < blocks / kLeast ? 152 / tiles : blocks / kLeast;
  return most < 1 ? 1 : most;
}
// The least items, so that no sum of bf16 products is longer than 131072 values: the tensor cores cut their sums off
// where fp32 would round, 8e-10 a value of a random sum towards 0, which is 1e-4 of it then (a bf16 result's own
// rounding is 1.7e-3 of it).  fp32 adds up short runs.
constexpr int kLongest = 2048;
int least_splits(const FfProb& r, bool f32) { return f32 ? 1 : ceil_div(r.pairs * r.kblocks, kLongest); }
// Numbers the items.  A tile's sum is shared by several where the launch would otherwise wait for it
// (a single tile of 30 rows over 2 x 10384 values 540 us): by as many as leave the least to the busiest pair,
// and where that saves more than joining the sums costs.  Found from two starts, a problem after the other: from
// whole sums, and from shares of one size, since both weights' gradients are alike and a launch that shares one of
// them still waits for the other (8192 x 64 x 64 41.8 -> 16.9 us, fp32 215 -> 33; 4096 x 256 x 512 27 -> 21 and 119 ->
// 42; 1003 x 1024 x 2816, with one more sum shared, 30.1 -> 31.0).  Returns the bytes of the sums.
size_t share_out(FfArgs& p, double block, bool f32) {
  int most[ll::kFfProbs], found[ll::kFfProbs], longest = 0;
  for (int i = 0; i < p.probs; ++i) {
    FfProb& r = p.prob[i];
    share(r, 1);
    most[i] = most_splits(r, block);
    found[i] = 1;
    if (most[i] > 1 && r.share > longest) longest = r.share;
  }
  const long long whole = most_blocks(p);
  long long least = whole;
  // from the splits that there are, of `now` blocks
  auto refine = [&](long long now) {
    for (int i = 0; i < p.probs; ++i) {
      FfProb& r = p.prob[i];
      int best = r.splits;
      for (int splits = 2; splits <= most[i]; splits += (splits + 3) / 4) {
        share(r, splits);
        const long long blocks = most_blocks(p);
        if (blocks < now) {
          now = blocks;
          best = splits;
        }
      }
      share(r, best);
    }
    if (now >= least) return;
    least = now;
    for (int i = 0; i < p.probs; ++i) found[i] = p.prob[i].splits;
  };
  if (longest) refine(whole);
  if (longest && p.probs > 1) {
    auto even = [&](int size) {
      for (int i = 0; i < p.probs; ++i) {
        const int splits = ceil_div(p.prob[i].pairs * p.prob[i].kblocks, size);
        share(p.prob[i], splits < most[i] ? splits : most[i]);
      }
      return most_blocks(p);
    };
    int best = longest;
    long long blocks = even(longest);
    for (int size = longest; size >= kLeast; size -= (size + 3) / 4) {
      const long long now = even(size);
      if (now < blocks) {
        blocks = now;
        best = size;
      }
    }
    refine(even(best));
  }
  const bool pays = (whole - least) * block >= kJoinUs;
  for (int i = 0; i < p.probs; ++i) {
    const int splits = pays ? found[i] : 1, floor = least_splits(p.prob[i], f32);
    share(p.prob[i], splits > floor ? splits : floor);
  }
  size_t bytes = 0;
  p.tiles = 0;
  for (int i = 0; i < p.probs; ++i) {
    FfProb& r = p.prob[i];
    r.tile0 = p.tiles;
    p.tiles += r.tiles_m * r.tiles_n * r.splits;
    if (r.splits > 1) bytes += a256((size_t)r.splits * (r.gated ? 2 : 1) * r.rows * r.cols * 4);
  }
  return bytes;
}

// The products of a call, in the order of their launch: forward one, backward up to three (the
// longest tiles first: sums over 2 ff and over the rows).  kDx and so on say which.
enum { kM, kDx, kDwGate, kDwUp };
struct Work {
  FfArgs args;
  int what[ll::kFfProbs];
  // workspace: operands that the call makes, bf16 (fp32 calls: in parts), and sums of split tiles
  size_t x, w_gate, w_up, scale, dgate, dup, part, bytes;
};
// plan: not for a bound on the bytes alone (backward).
Work work_of(const ffgate_shape* s, bool bwd, bool dx, bool dw_gate, bool dw_up, bool plan = true) {
  Work w{};
  FfArgs& p = w.args;
  if (!bwd) {
    w.what[p.probs] = kM;
    add_problem(p, s->rows, s->ff, s->dim, gated_width(s), 1).gated = 1;
  }
  auto add_dx = [&] {
    if (!dx) return;
    w.what[p.probs] = kDx;
    add_problem(p, s->rows, s->dim, s->ff, 256, 2).b_mn = 1;
  };
  auto add_dw = [&](int what) {
    w.what[p.probs] = what;
    FfProb& r = add_problem(p, s->ff, s->dim, s->rows, 256, 1);
    r.a_mn = r.b_mn = 1;
  };
  const bool dx_first = 2ll * s->ff >= s->rows;
  if (dx_first) add_dx();
  if (dw_gate) add_dw(kDwGate);
  if (dw_up) add_dw(kDwUp);
  if (!dx_first) add_dx();
  const bool f32 = s->dtype == LL_F32;
  const double block = block_us(f32, bwd);
  size_t parts = 0;
  if (plan) {
    parts = share_out(p, block, f32);
  } else {  // whatever the plan: room for the most items
    for (int i = 0; i < p.probs; ++i) {
      const int a = most_splits(p.prob[i], block), b = least_splits(p.prob[i], f32), most = a > b ? a : b;
      if (most > 1) parts += a256((size_t)most * p.prob[i].rows * p.prob[i].cols * 4);
    }
  }

  // Few rows of bf16: a stage has no more of them than there are, so that more of the weights is under way
  // (64 x 4096 x 11008 41 -> 37 us; with weights still in L2 and 512 values a row 6.3 -> 5.4, 2048 no less).
  // fp32 gains nothing by it (the runs' adding up bounds it).
  if (!bwd && !f32 && s->rows <= 128) {
    p.a_box = ((int)s->rows + 7) / 8 * 8;
    p.b_box = p.prob[0].width;
    const int stages = ll::kFfStageRoom / ((p.a_box + p.b_box) * 128);
    p.stages = stages < ll::kFfMaxStages ? stages : ll::kFfMaxStages;
  }
  auto take = [&](size_t n) {
    const size_t at = w.bytes;
    w.bytes += a256(n);
    return at;
  };
  if (f32) {
    const size_t bytes = bwd ? 6 : 4;
    w.x = take(bytes * s->rows * s->dim);
    w.w_gate = take(bytes * s->ff * s->dim);
    w.w_up = take(bytes * s->ff * s->dim);
    if (!bwd) w.scale = take(8 * (s->rows + 2 * (size_t)s->ff));
  }
  if (bwd) {
    w.dgate = take((size_t)(f32 ? 6 : 2) * s->rows * s->ff);
    w.dup = take((size_t)(f32 ? 6 : 2) * s->rows * s->ff);
  }
  w.part = take(parts);
  return w;
}
// Places the sums of split tiles, and lists what joins them.
void place_parts(Work& w, char* ws, void* const* outs, ll::FfJoin& j) {
  size_t at = w.part;
  j = ll::FfJoin{};
  for (int i = 0; i < w.args.probs; ++i) {
    FfProb& r = w.args.prob[i];
    if (r.splits < 2) continue;
    r.part = reinterpret_cast<float*>(ws + at);
    auto& q = j.prob[j.probs++];
    q.part = r.part;
    q.n = (long long)r.rows * r.cols;
    q.splits = r.splits;
    q.out = outs[w.what[i]];
    at += a256((size_t)r.splits * (r.gated ? 2 : 1) * q.n * 4);
  }
}
ll_status run(Work& w, const FfMaps& maps, const ll::FfJoin& j, ll::FfOperands kind, bool behind, cudaStream_t on) {
  const bool bf16 = kind == ll::FfOperands::kWhole;
  w.args.status = ll::device_status_word();
  if (!w.args.status) return LL_ERR_CUDA;
  if (ll::launch_ff_products(w.args, maps, kind, behind, on) != cudaSuccess) return LL_ERR_CUDA;
  return !j.probs || ll::launch_ff_join(j, bf16, on) == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}
// fp32: x and the weights as operands in parts, in the workspace.
bool split_operands(const ffgate_shape* s, Work& w, bool bwd, char* ws, const void*& x, const void*& w_gate,
                    const void*& w_up, cudaStream_t on) {
  if (s->dtype == LL_BF16) return true;
  if (!bwd) {
    float2* const scale = reinterpret_cast<float2*>(ws + w.scale);
    const ll::FfHalves c{{static_cast<const float*>(x), static_cast<const float*>(w_gate), static_cast<const float*>(w_up)},
                         {ws + w.x, ws + w.w_gate, ws + w.w_up},
                         {scale, scale + s->rows, scale + s->rows + s->ff},
                         {s->rows, s->ff, s->ff},
                         s->dim};
    x = ws + w.x;
    w_gate = ws + w.w_gate;
    w_up = ws + w.w_up;
    w.args.scale_x = c.scale[0];
    w.args.scale_gate = c.scale[1];
    w.args.scale_up = c.scale[2];
    return ll::launch_ff_halves(c, on) == cudaSuccess;
  }
  const long long rd = s->rows * s->dim, fd = (long long)s->ff * s->dim;
  const ll::FfSplit c{{static_cast<const float*>(x), static_cast<const float*>(w_gate), static_cast<const float*>(w_up)},
                      {ws + w.x, ws + w.w_gate, ws + w.w_up}, {rd, fd, fd}, 3};
  x = ws + w.x;
  w_gate = ws + w.w_gate;
  w_up = ws + w.w_up;
  return ll::launch_ff_split(c, on) == cudaSuccess;
}

}  // namespace

extern "C" {

size_t ffgate_fwd_workspace_bytes(const ffgate_shape* s) {
  if (check_shape(s) != LL_OK) return 0;
  const size_t n = streamed(s) ? 0 : work_of(s, false, false, false, false).bytes;
  return n < 16 ? 16 : n;
}

ll_status ffgate_fwd(const ffgate_shape* s, const void* x, const void* w_gate, const void* w_up, void* m, void* gate, void* up,
                     void* workspace, size_t workspace_bytes, void* stream) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  if (!x || !w_gate || !w_up || !m || (gate != nullptr) != (up != nullptr)) return LL_ERR_NULL;
  if (gate && (gate == up || gate == m || up == m)) return LL_ERR_SHAPE;
  for (const void* o : {(const void*)m, (const void*)gate, (const void*)up})
    if (o && (o == x || o == w_gate || o == w_up)) return LL_ERR_SHAPE;
  for (const void* q : {x, w_gate, w_up, (const void*)m, (const void*)gate, (const void*)up, (const void*)workspace})
    if (!aligned16(q)) return LL_ERR_ALIGN;
  const bool bf16 = s->dtype == LL_BF16;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  if (streamed(s)) {
    const ll::FfStream c{(int)s->rows, s->dim, s->ff, s->act, x, w_gate, w_up, m, gate, up};
    return ll::launch_ff_stream(c, bf16, on) == cudaSuccess ? LL_OK : LL_ERR_CUDA;
  }
  Work w = work_of(s, false, false, false, false);
  if (w.bytes && (!workspace || workspace_bytes < w.bytes)) return LL_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  if (!split_operands(s, w, false, ws, x, w_gate, w_up, on)) return LL_ERR_CUDA;
  const int parts = bf16 ? 1 : 2;
  FfMaps maps{};
  FfProb& r = w.args.prob[0];
  w.args.act = s->act;
  w.args.m = m;
  w.args.gate = gate;
  w.args.up = up;
  r.a[0] = 0;
  r.b[0] = 1;
  r.b[1] = 2;
  r.out = 3;
  bool ok = ll::ff_operand_map(&maps.m[0], x, s->dim, s->rows, parts, false, w.args.stages ? w.args.a_box : 128) &&
            ll::ff_operand_map(&maps.m[1], w_gate, s->dim, s->ff, parts, false, r.width) &&
            ll::ff_operand_map(&maps.m[2], w_up, s->dim, s->ff, parts, false, r.width) &&
            ll::ff_output_map(&maps.m[3], m, s->ff, s->rows, bf16);
  if (gate) {
    r.out_gate = 4;
    r.out_up = 5;
    ok = ok && ll::ff_output_map(&maps.m[4], gate, s->ff, s->rows, bf16) && ll::ff_output_map(&maps.m[5], up, s->ff, s->rows, bf16);
  }
  if (!ok) return LL_ERR_CUDA;
  void* const outs[] = {m};
  ll::FfJoin j;
  place_parts(w, ws, outs, j);
  j.gated = 1;
  j.act = s->act;
  j.gate = gate;
  j.up = up;
  return run(w, maps, j, bf16 ? ll::FfOperands::kWhole : ll::FfOperands::kHalves, !bf16, on);
}

size_t ffgate_bwd_workspace_bytes(const ffgate_shape* s) {
  if (check_shape(s) != LL_OK) return 0;
  // room for whichever gradients are asked for, and however their sums are shared
  return work_of(s, true, true, true, true, false).bytes;
}

ll_status ffgate_bwd(const ffgate_shape* s, const void* dm, const void* x, const void* w_gate, const void* w_up,
                     const void* gate, const void* up, void* dx, void* dw_gate, void* dw_up, void* workspace,
                     size_t workspace_bytes, void* stream) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  if (!dm || !x || !w_gate || !w_up || !gate || !up || (!dx && !dw_gate && !dw_up)) return LL_ERR_NULL;
  const void* given[] = {dx, dw_gate, dw_up};
  for (const void* o : given) {
    if (!o) continue;
    for (const void* q : {dm, x, w_gate, w_up, gate, up})
      if (o == q) return LL_ERR_SHAPE;
    int same = 0;
    for (const void* q : given) same += q == o;
    if (same > 1) return LL_ERR_SHAPE;
  }
  for (const void* q : {dm, x, w_gate, w_up, gate, up, (const void*)dx, (const void*)dw_gate, (const void*)dw_up,
                        (const void*)workspace})
    if (!aligned16(q)) return LL_ERR_ALIGN;
  const bool bf16 = s->dtype == LL_BF16;
  if (!workspace || workspace_bytes < ffgate_bwd_workspace_bytes(s)) return LL_ERR_WORKSPACE;
  Work w = work_of(s, true, dx != nullptr, dw_gate != nullptr, dw_up != nullptr);
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (!split_operands(s, w, true, ws, x, w_gate, w_up, on)) return LL_ERR_CUDA;
  void *dg = ws + w.dgate, *du = ws + w.dup;
  if (ll::launch_ff_act_bwd(dm, gate, up, dg, du, s->rows * s->ff, s->act, bf16, on) != cudaSuccess) return LL_ERR_CUDA;
  const int parts = bf16 ? 1 : 3;
  FfMaps maps{};
  int n = 0;
  bool ok = true;
  auto operand = [&](const void* base, long long inner, long long outer, bool mn) {
    ok = ok && ll::ff_operand_map(&maps.m[n], base, inner, outer, parts, mn);
    return n++;
  };
  auto output = [&](void* base, long long cols, long long rows) {
    ok = ok && ll::ff_output_map(&maps.m[n], base, cols, rows, bf16);
    return n++;
  };
  const int of_x = dw_gate || dw_up ? operand(x, s->dim, s->rows, true) : -1;
  for (int i = 0; i < w.args.probs; ++i) {
    FfProb& r = w.args.prob[i];
    if (w.what[i] == kDx) {
      r.a[0] = operand(dg, s->ff, s->rows, false);
      r.a[1] = operand(du, s->ff, s->rows, false);
      r.b[0] = operand(w_gate, s->dim, s->ff, true);
      r.b[1] = operand(w_up, s->dim, s->ff, true);
      r.out = output(dx, s->dim, s->rows);
    } else {
      const bool second = w.what[i] == kDwUp;
      r.a[0] = operand(second ? du : dg, s->ff, s->rows, true);
      r.b[0] = of_x;
      r.out = output(second ? dw_up : dw_gate, s->dim, s->ff);
    }
  }
  if (!ok) return LL_ERR_CUDA;
  void* const outs[] = {nullptr, dx, dw_gate, dw_up};
  ll::FfJoin j;
  place_parts(w, ws, outs, j);
  return run(w, maps, j, bf16 ? ll::FfOperands::kWhole : ll::FfOperands::kThirds, true, on);
}

}  // extern "C"
