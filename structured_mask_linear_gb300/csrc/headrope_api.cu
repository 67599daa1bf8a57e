// Entry points of the head norms with rotation: argument checks and workspace size.  Contracts are
// in include/loglinear.h.
#include <cuda_runtime.h>

#include <initializer_list>

#include "headrope.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Whether an output takes the place of what all rows read.
bool over_shared(std::initializer_list<const void*> outs, std::initializer_list<const void*> shared) {
  for (const void* o : outs)
    for (const void* q : shared)
      if (o && o == q) return true;
  return false;
}

ll_status check_shape(const headrope_shape* s) {
  if (!s) return LL_ERR_NULL;
  if (s->dtype != LL_F32 && s->dtype != LL_BF16) return LL_ERR_DTYPE;
  if (s->rows < 1 || s->rows > 0x7fffffff || s->T < 1) return LL_ERR_SHAPE;
  if (s->q_heads < 1 || s->q_heads > 65536 || s->k_heads < 0 || s->k_heads > 65536) return LL_ERR_SHAPE;
  if (s->dim < 1 || s->dim > ll::kHrMaxDim || s->rot < 0 || s->rot > s->dim || s->rot % 2) return LL_ERR_SHAPE;
  if (s->layout != HR_HALF && s->layout != HR_INTERLEAVED) return LL_ERR_SHAPE;
  if (s->norm != HR_NONE && s->norm != HR_RMS && s->norm != HR_L2) return LL_ERR_SHAPE;
  if (!(s->eps >= 0.f) || s->eps > 1.f) return LL_ERR_SHAPE;
  return LL_OK;
}
ll::HrArgs base_args(const headrope_shape* s) {
  ll::HrArgs p{};
  p.rows = s->rows;
  p.T = s->T;
  p.gq = s->q_heads;
  p.gk = s->k_heads;
  p.d = s->dim;
  p.rot = s->rot;
  p.norm = s->norm;
  p.eps = s->eps;
  p.inv_d = 1.f / (float)s->dim;
  p.scale_q = s->scale_q;
  p.scale_k = s->scale_k;
  return p;
}

}  // namespace

extern "C" {

ll_status headrope_fwd(const headrope_shape* s, const void* q, const void* k, const float* w_q, const float* w_k,
                       const float* inv_freq, const int* positions, void* q_out, void* k_out, void* stream) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  if (!q || !q_out || (s->k_heads > 0) != (k != nullptr) || (k != nullptr) != (k_out != nullptr) || (w_k && !k) ||
      (s->rot > 0 && !inv_freq))
    return LL_ERR_NULL;
  if (k && (q_out == k_out || q_out == k || k_out == q)) return LL_ERR_SHAPE;
  for (const void* x : {q, k, (const void*)w_q, (const void*)w_k, (const void*)inv_freq, (const void*)positions,
                        (const void*)q_out, (const void*)k_out})
    if (!aligned16(x)) return LL_ERR_ALIGN;
  if (over_shared({q_out, k_out}, {w_q, w_k, inv_freq, positions})) return LL_ERR_SHAPE;
  ll::HrArgs p = base_args(s);
  p.q = q;
  p.k = k;
  p.w_q = w_q;
  p.w_k = w_k;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.q_out = q_out;
  p.k_out = k_out;
  const cudaError_t e = ll::launch_hr_fwd(p, s->layout, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

size_t headrope_bwd_workspace_bytes(const headrope_shape* s) {
  return check_shape(s) == LL_OK ? (size_t)ll::kHrMaxParts * 2 * s->dim * 4 : 0;
}

ll_status headrope_bwd(const headrope_shape* s, const void* dq_out, const void* dk_out, const void* q, const void* k,
                       const float* w_q, const float* w_k, const float* inv_freq, const int* positions, void* dq,
                       void* dk, float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes, void* stream) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  if (!dq_out || !q || !dq || (s->k_heads > 0) != (k != nullptr) || (k != nullptr) != (dk_out != nullptr) ||
      (k != nullptr) != (dk != nullptr) || (w_k && !k) || (dw_q && !w_q) || (dw_k && !w_k) || (s->rot > 0 && !inv_freq))
    return LL_ERR_NULL;
  if (k && (dq == dk || dq == k || dq == dk_out || dk == q || dk == dq_out)) return LL_ERR_SHAPE;
  for (const void* x : {dq_out, dk_out, q, k, (const void*)w_q, (const void*)w_k, (const void*)inv_freq,
                        (const void*)positions, (const void*)dq, (const void*)dk, (const void*)dw_q, (const void*)dw_k,
                        (const void*)workspace})
    if (!aligned16(x)) return LL_ERR_ALIGN;
  if (over_shared({dq, dk, dw_q, dw_k}, {w_q, w_k, inv_freq, positions}) || over_shared({dw_q, dw_k}, {dq, dk, dq_out, dk_out, q, k}) ||
      (dw_q && dw_q == dw_k))
    return LL_ERR_SHAPE;
  if ((dw_q || dw_k) && (!workspace || workspace_bytes < headrope_bwd_workspace_bytes(s))) return LL_ERR_WORKSPACE;
  ll::HrArgs p = base_args(s);
  p.q = q;
  p.k = k;
  p.w_q = w_q;
  p.w_k = w_k;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.dq = dq_out;
  p.dk = dk_out;
  p.q_out = dq;
  p.k_out = dk;
  p.dw_q = dw_q;
  p.dw_k = dw_k;
  p.part = dw_q || dw_k ? static_cast<float*>(workspace) : nullptr;
  const cudaError_t e = ll::launch_hr_bwd(p, s->layout, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

}  // extern "C"
