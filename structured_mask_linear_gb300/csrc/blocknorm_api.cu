// Entry points of the block norm: argument checks and workspace size.  Contracts are in
// include/loglinear.h.
#include <cuda_runtime.h>

#include "blocknorm.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ll_status check_shape(const blocknorm_shape* s) {
  if (!s) return LL_ERR_NULL;
  if (s->dtype != LL_F32 && s->dtype != LL_BF16) return LL_ERR_DTYPE;
  if (s->rows < 1 || s->rows > 0x7fffffff || s->dim < 1 || s->dim > ll::kBnMaxD) return LL_ERR_SHAPE;
  if (s->group < 1 || s->dim % s->group || s->dim / s->group > ll::kBnMaxGroups) return LL_ERR_SHAPE;
  if (s->act != BN_IDENTITY && s->act != BN_SILU && s->act != BN_SIGMOID) return LL_ERR_SHAPE;
  if (!(s->eps >= 0.f) || s->eps > 1.f) return LL_ERR_SHAPE;
  return LL_OK;
}

ll::BnArgs base_args(const blocknorm_shape* s) {
  ll::BnArgs p{};
  p.rows = s->rows;
  p.D = s->dim;
  p.group = s->group;
  p.act = s->act;
  p.eps = s->eps;
  p.inv_D = 1.f / (float)s->dim;
  p.inv_group = 1.f / (float)s->group;
  return p;
}

}  // namespace

extern "C" {

ll_status blocknorm_fwd(const blocknorm_shape* s, const void* x, const void* y, const void* gate,
                        const float* w_post, const float* scale, const float* w_pre, void* x_new, void* h,
                        void* stream) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  if (!x && !y) return LL_ERR_NULL;
  if (y ? !x_new : (!h || x_new || gate || w_post || scale)) return LL_ERR_NULL;
  if (!h && w_pre) return LL_ERR_NULL;
  if (h && h == x_new) return LL_ERR_SHAPE;
  for (const void* q : {x, y, gate, (const void*)w_post, (const void*)scale, (const void*)w_pre, (const void*)x_new,
                        (const void*)h})
    if (!aligned16(q)) return LL_ERR_ALIGN;
  ll::BnArgs p = base_args(s);
  p.x = x;
  p.y = y;
  p.gate = gate;
  p.w_post = w_post;
  p.scale = scale;
  p.w_pre = w_pre;
  p.x_new = x_new;
  p.h = h;
  const cudaError_t e = ll::launch_bn_fwd(p, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

size_t blocknorm_bwd_workspace_bytes(const blocknorm_shape* s) {
  if (check_shape(s) != LL_OK) return 0;
  return (size_t)ll::kBnMaxParts * 3 * s->dim * 4;
}

ll_status blocknorm_bwd(const blocknorm_shape* s, const void* dx_new, const void* dh, const void* x_new,
                        const void* y, const void* gate, const float* w_post, const float* scale,
                        const float* w_pre, void* dx, void* dy, void* dgate, float* dw_post, float* dscale,
                        float* dw_pre, void* workspace, size_t workspace_bytes, void* stream) {
  const ll_status st = check_shape(s);
  if (st != LL_OK) return st;
  if (!dx_new && !dh) return LL_ERR_NULL;
  if ((dh != nullptr) != (x_new != nullptr) || ((w_pre || dw_pre) && !dh)) return LL_ERR_NULL;
  if ((y != nullptr) != (dy != nullptr) || (gate != nullptr) != (dgate != nullptr)) return LL_ERR_NULL;
  if (y ? (dw_post && !w_post) || (dscale && !scale) : (!dx || gate || w_post || scale || dw_post || dscale))
    return LL_ERR_NULL;
  if (dw_pre && !w_pre) return LL_ERR_NULL;
  for (const void* q : {dx_new, dh, x_new, y, gate, (const void*)w_post, (const void*)scale, (const void*)w_pre,
                        (const void*)dx, (const void*)dy, (const void*)dgate, (const void*)dw_post,
                        (const void*)dscale, (const void*)dw_pre, (const void*)workspace})
    if (!aligned16(q)) return LL_ERR_ALIGN;
  if (!workspace || workspace_bytes < blocknorm_bwd_workspace_bytes(s)) return LL_ERR_WORKSPACE;
  ll::BnArgs p = base_args(s);
  p.x = x_new;
  p.y = y;
  p.gate = gate;
  p.w_post = w_post;
  p.scale = scale;
  p.w_pre = w_pre;
  p.dx_new = dx_new;
  p.dh = dh;
  p.dx = dx;
  p.dy = dy;
  p.dgate = dgate;
  p.dw_post = dw_post;
  p.dscale = dscale;
  p.dw_pre = dw_pre;
  p.part = static_cast<float*>(workspace);
  p.status = ll::device_status_word();
  if (!p.status) return LL_ERR_CUDA;
  const cudaError_t e = ll::launch_bn_bwd(p, s->dtype == LL_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

}  // extern "C"
