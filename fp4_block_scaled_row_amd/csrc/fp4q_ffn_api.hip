// fp4q_ffn_api.hip -- the C ABI of the linear layers over 4-bit weights and of
// the norm (see include/fp4q.h): host-side checks and dispatch.  Every check runs
// before anything is enqueued.
#include <limits.h>
#include <math.h>
#include <string.h>

#include "fp4q.h"
#include "fp4q_ffn.h"

using namespace fp4q;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
fp4q_status hip_status(hipError_t e) { return e == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }
bool float_type(int t) { return t == FP4Q_F32 || t == FP4Q_BF16; }
size_t size_of(int t) { return t == FP4Q_F32 ? 4 : 2; }

// Checks of a linear call.  With nothing to compute (no rows or no outputs) only
// the shapes are looked at.
fp4q_status check_linear(const fp4q_weight* w, const fp4q_linear_args* a, int kind, LinearLaunch* l) {
  if (!w || !a || kind < FP4Q_LINEAR || kind > FP4Q_LINEAR_BACKWARD) return FP4Q_ERR_INVALID_ARG;
  if (w->format != FP4Q_MXFP4 && w->format != FP4Q_NVFP4)
    return w->format == FP4Q_IF4 || w->format == FP4Q_MXFP8 ? FP4Q_ERR_UNSUPPORTED : FP4Q_ERR_INVALID_ARG;
  const int block = w->format == FP4Q_MXFP4 ? 32 : 16;
  if (w->n < 0 || w->k < 0 || w->k % block != 0) return FP4Q_ERR_INVALID_ARG;
  if (w->n > INT_MAX || w->k > INT_MAX || a->rows > INT_MAX) return FP4Q_ERR_UNSUPPORTED;
  if (a->rows < 0 || a->x_stride < 0 || !float_type(a->out_dtype)) return FP4Q_ERR_INVALID_ARG;
  if (!float_type(a->x_dtype) && a->x_dtype != FP4Q_E4M3) return FP4Q_ERR_INVALID_ARG;
  if (kind == FP4Q_GATED && w->n % 2 != 0) return FP4Q_ERR_INVALID_ARG;
  if (kind != FP4Q_LINEAR && a->bias) return FP4Q_ERR_UNSUPPORTED;
  if (kind != FP4Q_GATED && a->products) return FP4Q_ERR_UNSUPPORTED;
  if (a->products && !float_type(a->products_dtype)) return FP4Q_ERR_INVALID_ARG;
  const bool back = kind == FP4Q_LINEAR_BACKWARD;
  const int64_t len = back ? w->n : w->k, out = back ? w->k : kind == FP4Q_GATED ? w->n / 2 : w->n;
  if (a->x_dtype == FP4Q_E4M3) {
    if (back) return FP4Q_ERR_UNSUPPORTED;
    if (w->k % 32 != 0 || a->x_stride != w->k) return FP4Q_ERR_INVALID_ARG;
  }
  memset(l, 0, sizeof(*l));
  l->rows = a->rows;
  l->w.n = w->n;
  l->w.k = w->k;
  l->w.format = w->format == FP4Q_MXFP4 ? 0 : 1;
  l->gated = kind == FP4Q_GATED;
  l->transposed = back;
  l->x_type = a->x_dtype == FP4Q_F32 ? kXF32 : a->x_dtype == FP4Q_BF16 ? kXBF16 : kXE4M3;
  l->out_bf16 = a->out_dtype == FP4Q_BF16;
  l->products_bf16 = a->products_dtype == FP4Q_BF16;
  if (a->rows == 0 || out == 0) return FP4Q_OK;
  // (tiles, the smallest too, are counted in 31 bits)
  if ((a->rows + 63) / 64 * ((out + 63) / 64) > INT_MAX / 8) return FP4Q_ERR_UNSUPPORTED;
  if (!a->out || (w->format == FP4Q_NVFP4 && !w->global_scale)) return FP4Q_ERR_INVALID_ARG;
  if (len > 0) {
    if (!a->x || !w->codes || !w->scales || (a->x_dtype == FP4Q_E4M3 && !a->x_scales)) return FP4Q_ERR_INVALID_ARG;
  }
  const size_t os = size_of(a->out_dtype);
  if (!aligned(a->out, os) || !aligned(a->products, size_of(a->products_dtype)) || !aligned(a->bias, os) ||
      !aligned(w->global_scale, 4))
    return FP4Q_ERR_UNSUPPORTED;
  if (a->x_dtype != FP4Q_E4M3 && !aligned(a->x, size_of(a->x_dtype))) return FP4Q_ERR_UNSUPPORTED;
  l->w.codes = w->codes;
  l->w.scales = w->scales;
  l->w.g = w->global_scale;
  l->x = a->x;
  l->x_scales = a->x_scales;
  l->x_stride = a->x_stride;
  l->bias = a->bias;
  l->out = a->out;
  l->products = a->products;
  return linear_fits(*l) ? FP4Q_OK : FP4Q_ERR_UNSUPPORTED;
}

bool nothing(const LinearLaunch& l) { return l.out == nullptr; }

fp4q_status linear(const fp4q_weight* w, const fp4q_linear_args* a, int kind, void* workspace, size_t bytes, void* s) {
  LinearLaunch l;
  const fp4q_status st = check_linear(w, a, kind, &l);
  if (st != FP4Q_OK || nothing(l)) return st;
  const size_t need = linear_workspace(l);
  if (need > 0 && (!workspace || bytes < need || !aligned(workspace, 16))) return FP4Q_ERR_WORKSPACE;
  l.partials = static_cast<float*>(workspace);
  return hip_status(launch_linear(l, static_cast<hipStream_t>(s)));
}

fp4q_status check_norm_grad(const fp4q_rms_norm_grad_args* a) {
  if (!a) return FP4Q_ERR_INVALID_ARG;
  if (a->rows < 0 || a->d < 0 || a->dy_stride < 0 || a->s_stride < 0 || a->ds_stride < 0) return FP4Q_ERR_INVALID_ARG;
  if (!float_type(a->dtype) || !float_type(a->weight_dtype)) return FP4Q_ERR_INVALID_ARG;
  if (a->d > 32768 || a->rows > INT_MAX) return FP4Q_ERR_UNSUPPORTED;
  if (a->d == 0) return FP4Q_OK;
  if (!a->dw) return FP4Q_ERR_INVALID_ARG;
  if (a->rows > 0 && (!a->dy || !a->s || !a->weight || !a->rstd || !a->dx)) return FP4Q_ERR_INVALID_ARG;
  const size_t es = size_of(a->dtype), ws = size_of(a->weight_dtype);
  if (!aligned(a->dy, es) || !aligned(a->s, es) || !aligned(a->ds, es) || !aligned(a->dx, es) ||
      !aligned(a->weight, ws) || !aligned(a->dw, ws) || !aligned(a->rstd, 4))
    return FP4Q_ERR_UNSUPPORTED;
  return FP4Q_OK;
}

}  // namespace

extern "C" {

size_t fp4q_linear_workspace_bytes(const fp4q_weight* weight, const fp4q_linear_args* args, int32_t kind) {
  LinearLaunch l;
  if (check_linear(weight, args, kind, &l) != FP4Q_OK || nothing(l)) return 0;
  return linear_workspace(l);
}

fp4q_status fp4q_linear(const fp4q_weight* weight, const fp4q_linear_args* args, void* workspace,
                        size_t workspace_bytes, void* hip_stream) {
  return linear(weight, args, FP4Q_LINEAR, workspace, workspace_bytes, hip_stream);
}

fp4q_status fp4q_gated(const fp4q_weight* weight, const fp4q_linear_args* args, void* workspace,
                       size_t workspace_bytes, void* hip_stream) {
  return linear(weight, args, FP4Q_GATED, workspace, workspace_bytes, hip_stream);
}

fp4q_status fp4q_linear_backward(const fp4q_weight* weight, const fp4q_linear_args* args, void* workspace,
                                 size_t workspace_bytes, void* hip_stream) {
  return linear(weight, args, FP4Q_LINEAR_BACKWARD, workspace, workspace_bytes, hip_stream);
}

fp4q_status fp4q_gated_grad(const fp4q_gated_grad_args* a, void* hip_stream) {
  if (!a || a->rows < 0 || a->f < 0 || a->dh_stride < 0 || !float_type(a->dtype) ||
      !float_type(a->products_dtype))
    return FP4Q_ERR_INVALID_ARG;
  if (a->rows > INT_MAX || a->f > INT_MAX / 2) return FP4Q_ERR_UNSUPPORTED;
  if (a->rows == 0 || a->f == 0) return FP4Q_OK;
  if (a->rows * ((a->f + 7) / 8) / 256 >= INT_MAX) return FP4Q_ERR_UNSUPPORTED;
  if (!a->dh || !a->products || !a->dproducts) return FP4Q_ERR_INVALID_ARG;
  const size_t es = size_of(a->dtype);
  if (!aligned(a->dh, es) || !aligned(a->products, size_of(a->products_dtype)) || !aligned(a->dproducts, es))
    return FP4Q_ERR_UNSUPPORTED;
  // (a thread writes where it read only if both have the same type)
  if (a->dproducts == a->products && a->dtype != a->products_dtype) return FP4Q_ERR_INVALID_ARG;
  const GatedGradLaunch l = {a->dh, a->products, a->dproducts, a->rows, a->f, a->dh_stride, a->dtype == FP4Q_BF16,
                             a->products_dtype == FP4Q_BF16};
  return hip_status(launch_gated_grad(l, static_cast<hipStream_t>(hip_stream)));
}

fp4q_status fp4q_rms_norm(const fp4q_rms_norm_args* a, void* hip_stream) {
  if (!a) return FP4Q_ERR_INVALID_ARG;
  if (a->rows < 0 || a->d < 0 || a->x_stride < 0 || a->residual_stride < 0) return FP4Q_ERR_INVALID_ARG;
  if (!float_type(a->dtype) || !float_type(a->weight_dtype)) return FP4Q_ERR_INVALID_ARG;
  if (!(a->eps >= 0.0f) || !(a->eps < INFINITY)) return FP4Q_ERR_INVALID_ARG;
  if ((a->codes != nullptr) != (a->scales != nullptr)) return FP4Q_ERR_INVALID_ARG;
  if (a->codes && (a->y || a->d % 32 != 0)) return a->y ? FP4Q_ERR_UNSUPPORTED : FP4Q_ERR_INVALID_ARG;
  if (a->d > 32768 || a->rows > INT_MAX) return FP4Q_ERR_UNSUPPORTED;
  if (a->rows == 0 || a->d == 0) return FP4Q_OK;
  if (!a->x || !a->weight || (!a->y && !a->codes) || (a->residual != nullptr) != (a->summed != nullptr))
    return FP4Q_ERR_INVALID_ARG;
  const size_t es = size_of(a->dtype);
  if (!aligned(a->x, es) || !aligned(a->residual, es) || !aligned(a->summed, es) || !aligned(a->y, es) ||
      !aligned(a->weight, size_of(a->weight_dtype)) || !aligned(a->rstd, 4))
    return FP4Q_ERR_UNSUPPORTED;
  NormLaunch l;
  memset(&l, 0, sizeof(l));
  l.x = a->x;
  l.residual = a->residual;
  l.w = a->weight;
  l.y = a->y;
  l.summed = a->summed;
  l.rstd = a->rstd;
  l.codes = a->codes;
  l.scales = a->scales;
  l.rows = a->rows;
  l.d = a->d;
  l.x_stride = a->x_stride;
  l.residual_stride = a->residual_stride;
  l.bf16 = a->dtype == FP4Q_BF16;
  l.w_bf16 = a->weight_dtype == FP4Q_BF16;
  l.eps = a->eps;
  return hip_status(launch_rms_norm(l, static_cast<hipStream_t>(hip_stream)));
}

size_t fp4q_rms_norm_backward_workspace_bytes(const fp4q_rms_norm_grad_args* args) {
  if (check_norm_grad(args) != FP4Q_OK || args->d == 0) return 0;
  return rms_norm_grad_workspace(args->rows, args->d);
}

fp4q_status fp4q_rms_norm_backward(const fp4q_rms_norm_grad_args* a, void* workspace, size_t workspace_bytes,
                                   void* hip_stream) {
  const fp4q_status st = check_norm_grad(a);
  if (st != FP4Q_OK || a->d == 0) return st;
  const size_t need = rms_norm_grad_workspace(a->rows, a->d);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return FP4Q_ERR_WORKSPACE;
  NormGradLaunch l;
  memset(&l, 0, sizeof(l));
  l.dy = a->dy;
  l.s = a->s;
  l.w = a->weight;
  l.ds = a->ds;
  l.rstd = a->rstd;
  l.dx = a->dx;
  l.dw = a->dw;
  l.rows = a->rows;
  l.d = a->d;
  l.dy_stride = a->dy_stride;
  l.s_stride = a->s_stride;
  l.ds_stride = a->ds_stride;
  l.bf16 = a->dtype == FP4Q_BF16;
  l.w_bf16 = a->weight_dtype == FP4Q_BF16;
  l.partials = static_cast<float*>(workspace);
  return hip_status(launch_rms_norm_grad(l, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
