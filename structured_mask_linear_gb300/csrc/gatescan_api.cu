// Entry points of the gated recurrence: argument checks.  Contracts are in
// include/loglinear.h.
#include <cuda_runtime.h>

#include <initializer_list>

#include "gatescan.cuh"

namespace {

using ll::GsArgs;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool among(const void* o, std::initializer_list<const void*> others) {
  for (const void* q : others)
    if (o && o == q) return true;
  return false;
}

ll_status check_shape(const gatescan_shape* s, bool seq) {
  if (!s) return LL_ERR_NULL;
  if (s->dtype != LL_F32 && s->dtype != LL_BF16) return LL_ERR_DTYPE;
  if (s->batch < 1 || s->batch > (1 << 20) || s->dim < 1 || s->dim > (1 << 20)) return LL_ERR_SHAPE;
  if (s->mix != GS_RMS && s->mix != GS_LERP && s->mix != GS_NONE) return LL_ERR_SHAPE;
  if (!seq) return LL_OK;
  if (s->T < 1 || s->T > (1 << 30)) return LL_ERR_SHAPE;
  // CTAs: units of 16 channels at least, up to kGsMaxCluster each
  const long long units = (long long)s->batch * ((s->dim + 15) / 16);
  return units > 0x7fffffff / ll::kGsMaxCluster ? LL_ERR_SHAPE : LL_OK;
}

GsArgs base_args(const gatescan_shape* s) {
  GsArgs p{};
  p.B = s->batch;
  p.T = s->T;
  p.D = s->dim;
  p.mix = s->mix;
  return p;
}

}  // namespace

extern "C" {

ll_status gatescan_fwd(const gatescan_shape* s, const void* x, const void* r, const void* i, const float* decay,
                       const int* lengths, const float* state_in, void* h, float* state_out, void* stream) {
  const ll_status st = check_shape(s, true);
  if (st != LL_OK) return st;
  if (!x || !r || !decay || !h) return LL_ERR_NULL;
  for (const void* q : {x, r, i, (const void*)decay, (const void*)lengths, (const void*)state_in, (const void*)h,
                        (const void*)state_out})
    if (!aligned16(q)) return LL_ERR_ALIGN;
  if (among(h, {decay, lengths, state_in, state_out}) || among(state_out, {x, r, i, decay, lengths})) return LL_ERR_SHAPE;
  GsArgs p = base_args(s);
  p.x = x;
  p.r = r;
  p.i = i;
  p.decay = decay;
  p.lengths = lengths;
  p.state_in = state_in;
  p.h = h;
  p.state_out = state_out;
  p.status = ll::device_status_word();
  if (!p.status) return LL_ERR_CUDA;
  const cudaError_t e = ll::launch_gs_fwd(p, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

size_t gatescan_bwd_workspace_bytes(const gatescan_shape* s) {
  return check_shape(s, true) == LL_OK ? (size_t)ll::kGsMaxCluster * s->batch * s->dim * 4 : 0;
}

ll_status gatescan_bwd(const gatescan_shape* s, const void* dh, const void* x, const void* r, const void* i,
                       const float* decay, const void* h, const int* lengths, const float* state_in,
                       const float* dstate_out, void* dx, void* dr, void* di, float* ddecay, float* dstate_in,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const ll_status st = check_shape(s, true);
  if (st != LL_OK) return st;
  if (!dh || !x || !r || !decay || !h || !dx || !dr || (i != nullptr) != (di != nullptr)) return LL_ERR_NULL;
  const void* outs[] = {dx, dr, di, ddecay, dstate_in};
  for (const void* q : {dh, x, r, i, (const void*)decay, h, (const void*)lengths, (const void*)state_in,
                        (const void*)dstate_out, (const void*)dx, (const void*)dr, (const void*)di,
                        (const void*)ddecay, (const void*)dstate_in, (const void*)workspace})
    if (!aligned16(q)) return LL_ERR_ALIGN;
  for (const void* o : outs) {
    if (!o) continue;
    for (const void* q : {dh, x, r, i, (const void*)decay, h, (const void*)lengths, (const void*)state_in,
                          (const void*)dstate_out})
      if (o == q) return LL_ERR_SHAPE;
    int same = 0;
    for (const void* q : outs) same += q == o;
    if (same > 1) return LL_ERR_SHAPE;
  }
  if (ddecay && (!workspace || workspace_bytes < gatescan_bwd_workspace_bytes(s))) return LL_ERR_WORKSPACE;
  GsArgs p = base_args(s);
  p.part = ddecay ? static_cast<float*>(workspace) : nullptr;
  p.dh = dh;
  p.x = x;
  p.r = r;
  p.i = i;
  p.decay = decay;
  p.h_in = h;
  p.lengths = lengths;
  p.state_in = state_in;
  p.dstate_out = dstate_out;
  p.dx = dx;
  p.dr = dr;
  p.di = di;
  p.ddecay = ddecay;
  p.dstate_in = dstate_in;
  p.status = ll::device_status_word();
  if (!p.status) return LL_ERR_CUDA;
  const cudaError_t e = ll::launch_gs_bwd(p, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

ll_status gatescan_decode_step(const gatescan_shape* s, const void* x_t, const void* r_t, const void* i_t,
                               const float* decay, float* states, void* h_t, void* stream) {
  const ll_status st = check_shape(s, false);
  if (st != LL_OK) return st;
  if (!x_t || !r_t || !decay || !states || !h_t) return LL_ERR_NULL;
  for (const void* q : {x_t, r_t, i_t, (const void*)decay, (const void*)states, (const void*)h_t})
    if (!aligned16(q)) return LL_ERR_ALIGN;
  if (among(states, {x_t, r_t, i_t, decay, h_t}) || among(h_t, {decay})) return LL_ERR_SHAPE;
  const ll::GsStepArgs p{(long long)s->batch * s->dim, s->dim, x_t, r_t, i_t, decay, states, h_t};
  const cudaError_t e = ll::launch_gs_step(p, s->mix, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

}  // extern "C"
