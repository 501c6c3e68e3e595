// C ABI of the dense half of a transformer block: argument validation and the
// sequence of launches of each call.  Declarations and the meaning of every
// argument are in include/moe.h.
#include <stdint.h>

#include "moe_internal.cuh"

namespace moe {

namespace {

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A workspace of at least `need` bytes, aligned to 256.
moe_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// A row stride in elements: 0 (dense) becomes `cols`; otherwise at least
// `cols` and a multiple of `mult`.
bool fix_stride(int64_t *stride, int64_t cols, int mult) {
  if (*stride == 0) *stride = cols;
  return *stride >= cols && *stride % mult == 0 && *stride < ((int64_t)1 << 36);
}

// A validated copy of the descriptor with its strides filled in.
moe_status_t norm_desc(const moe_norm_desc_t *in, moe_norm_desc_t *d) {
  if (in == nullptr) return MOE_ERR_INVALID_ARG;
  *d = *in;
  if (d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_FP16 && d->dtype != MOE_DTYPE_FP32)
    return MOE_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (d->T < 0 || d->T > kMaxT || d->H < 8 || d->H > 16384 || d->H % 8 != 0)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!fix_stride(&d->x_stride, d->H, 8) || !fix_stride(&d->residual_stride, d->H, 8) ||
      !fix_stride(&d->y_stride, d->H, 8))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_norm_workspace_size(const moe_norm_desc_t *in) {
  moe_norm_desc_t d;
  if (norm_desc(in, &d) != MOE_OK) return 0;
  return kStatusPad + norm_bwd_part_bytes(d);
}

moe_status_t moe_add_rms_norm(const moe_norm_desc_t *in, const void *x, const void *residual,
                              const void *weight, void *residual_out, void *y, void *y_q,
                              int8_t *scale_exp, moe_stream_t stream) {
  moe_norm_desc_t d;
  moe_status_t st = norm_desc(in, &d);
  if (st != MOE_OK) return st;
  if (d.T == 0) return MOE_OK;  // empty tensors may have no address
  if (!ok_ptr(x) || !ok_opt(residual) || !ok_ptr(weight) || !ok_opt(residual_out) || !ok_opt(y) ||
      !ok_opt(y_q))
    return MOE_ERR_INVALID_ARG;
  if ((y_q == nullptr) != (scale_exp == nullptr) || (y == nullptr && y_q == nullptr))
    return MOE_ERR_INVALID_ARG;
  // in place means row for row
  if (residual_out == x && d.residual_stride != d.x_stride) return MOE_ERR_INVALID_ARG;
  if (y == x && d.y_stride != d.x_stride) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  return cuda_status(launch_add_rms_norm(d, x, residual, weight, residual_out, y,
                                         static_cast<uint8_t *>(y_q), scale_exp,
                                         (cudaStream_t)stream));
}

moe_status_t moe_add_rms_norm_backward(const moe_norm_desc_t *in, const void *dy,
                                       const void *dresidual, const void *sum, const void *weight,
                                       void *dx, float *dweight, void *workspace, size_t ws_bytes,
                                       moe_stream_t stream) {
  moe_norm_desc_t d;
  moe_status_t st = norm_desc(in, &d);
  if (st != MOE_OK) return st;
  if ((st = check_ws(workspace, ws_bytes, kStatusPad + norm_bwd_part_bytes(d))) != MOE_OK) return st;
  float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kStatusPad);
  if (!ok_opt(dweight)) return MOE_ERR_INVALID_ARG;
  if (d.T == 0) {
    if (dweight == nullptr) return MOE_OK;
    if ((st = check_device()) != MOE_OK) return st;
    return cuda_status(launch_column_sum(part, 0, d.H, d.H, dweight, 0, (cudaStream_t)stream));
  }
  if (!ok_ptr(dy) || !ok_opt(dresidual) || !ok_ptr(sum) || !ok_ptr(weight) || !ok_ptr(dx))
    return MOE_ERR_INVALID_ARG;
  if (dx == dy && d.x_stride != d.y_stride) return MOE_ERR_INVALID_ARG;
  if (dx == dresidual && d.x_stride != d.residual_stride) return MOE_ERR_INVALID_ARG;
  if (dx == sum) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  return cuda_status(launch_add_rms_norm_backward(d, dy, dresidual, sum, weight, dx, dweight, part,
                                                  (cudaStream_t)stream));
}

}  // extern "C"
