// C ABI of the experts' ragged products: argument validation and the sequence of
// launches of each call.  Declarations and the meaning of every argument are in
// include/moe.h.
#include <stdint.h>

#include <algorithm>

#include "api_util.cuh"
#include "grouped.cuh"
#include "int4.cuh"

namespace moe {

namespace {

// A validated copy of the descriptor with its strides filled in.
moe_status_t grouped_desc(const moe_grouped_desc_t *in, moe_grouped_desc_t *d) {
  if (in == nullptr) return MOE_ERR_INVALID_ARG;
  *d = *in;
  if (d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_FP16) return MOE_ERR_INVALID_ARG;
  if (d->out_dtype != d->dtype && d->out_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  const int32_t most = 1 << 18;
  if (d->R < 0 || d->R > kMaxAssign || d->E < 1 || d->E > kMaxE || d->N < 8 || d->N > most ||
      d->N % 8 != 0 || d->K < 8 || d->K > most || d->K % 8 != 0)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!fix_stride(&d->x_stride, d->K, 8) || !fix_stride(&d->y_stride, d->N, 8))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// After the status block: the weight gradient's tensor maps, then partial sums, then the
// rows of the products with 4-bit weights.
struct GroupedWs {
  size_t maps, part, rows, total;
};
GroupedWs grouped_ws(const moe_grouped_desc_t &d) {
  GroupedWs w;
  w.maps = kStatusPad;
  w.part = w.maps + pad(grouped_map_bytes(d.E));
  w.rows = w.part + pad(std::max(grouped_part_bytes(d.R), int4_part_bytes(d.R)));
  w.total = w.rows + pad(int4_rows_bytes(d.R, d.K));
  return w;
}

GroupedGemm grouped_product(const moe_grouped_desc_t &d, const int32_t *offsets, const void *x,
                            const void *w, const void *dy, void *out, int out_dtype,
                            void *workspace) {
  const GroupedWs L = grouped_ws(d);
  GroupedGemm g = {};
  g.R = d.R;
  g.E = d.E;
  g.N = d.N;
  g.K = d.K;
  g.dtype = d.dtype;
  g.out_dtype = out_dtype;
  g.offsets = offsets;
  g.x = x;
  g.w = w;
  g.dy = dy;
  g.ldx = d.x_stride;
  g.ldy = d.y_stride;
  g.d = out;
  g.part = reinterpret_cast<float *>(at(workspace, L.part));
  g.maps = reinterpret_cast<CUtensorMap *>(at(workspace, L.maps));
  g.status = static_cast<uint32_t *>(workspace);
  return g;
}

bool ok_group(int32_t group) { return group == 32 || group == 64 || group == 128; }

// `rows`: int4_rows_bytes of the workspace.  Up to eight rows of one matrix by the kernel
// that multiplies where it unpacks (experts': int4_few), others by way of tcgen05: 14336 x 4096
// with 8 rows 13.5 and 16.9 us, 114688 x 4096 51 and 68; groups of 32 16.7 and 18.1, 81 and 75.
cudaError_t launch_int4(Int4Gemm g, void *rows, cudaStream_t s) {
  if (g.offsets != nullptr && int4_few(g)) return launch_int4_small(g, s);
  const bool small = g.offsets == nullptr && g.T <= kInt4SmallRows;
  if (small && int4_staged(g)) return launch_int4_small(g, s);
  float *factor = reinterpret_cast<float *>(at(rows, (size_t)std::min(g.T, kInt4Rows) * int4_pitch(g.K) * 2));
  g.xr = rows;
  g.factor = factor;
  g.part_bytes = int4_part_bytes(g.T);
  cudaError_t e = cudaSuccess;
  for (g.first = 0; g.first < g.T && e == cudaSuccess; g.first += kInt4Rows) {
    e = launch_int4_rows(static_cast<const uint16_t *>(g.x) + g.first * g.ldx, g.ldx, g.dtype,
                         std::min(kInt4Rows, g.T - g.first), g.K, rows, factor, s);
    if (e == cudaSuccess) e = small ? launch_int4_small(g, s) : launch_int4_tc(g, s);
  }
  return e;
}

bool ok_offsets(const int32_t *p) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_linear_workspace_size(const moe_grouped_desc_t *in) {
  moe_grouped_desc_t d;
  return grouped_desc(in, &d) == MOE_OK ? grouped_ws(d).total : 0;
}

moe_status_t moe_grouped_linear(const moe_grouped_desc_t *in, const void *x, const int32_t *offsets,
                                const void *w, void *y, void *workspace, size_t ws_bytes,
                                moe_stream_t stream) {
  moe_grouped_desc_t d;
  moe_status_t st = grouped_desc(in, &d);
  if (st != MOE_OK) return st;
  if ((st = check_ws(workspace, ws_bytes, grouped_ws(d).total)) != MOE_OK) return st;
  if (!ok_offsets(offsets)) return MOE_ERR_INVALID_ARG;
  if (d.R == 0) return MOE_OK;  // empty tensors may have no address
  if (!ok_ptr(x) || !ok_ptr(w) || !ok_ptr(y)) return MOE_ERR_INVALID_ARG;
  if (lies_on(y, {x, w, offsets})) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  const GroupedGemm g = grouped_product(d, offsets, x, w, nullptr, y, d.out_dtype, workspace);
  return cuda_status(launch_grouped_rows(g, false, (cudaStream_t)stream));
}

moe_status_t moe_grouped_linear_backward(const moe_grouped_desc_t *in, const void *dy,
                                         const void *x, const int32_t *offsets, const void *w,
                                         void *dx, void *dw, int32_t dw_dtype, int32_t accumulate,
                                         void *workspace, size_t ws_bytes, moe_stream_t stream) {
  moe_grouped_desc_t d;
  moe_status_t st = grouped_desc(in, &d);
  if (st != MOE_OK) return st;
  if (dw_dtype != d.dtype && dw_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, grouped_ws(d).total)) != MOE_OK) return st;
  if (!ok_offsets(offsets) || !ok_opt(dw)) return MOE_ERR_INVALID_ARG;
  if (d.R > 0) {
    if (!ok_ptr(dy) || !ok_opt(dx)) return MOE_ERR_INVALID_ARG;
    if ((dx != nullptr && !ok_ptr(w)) || (dw != nullptr && !ok_ptr(x))) return MOE_ERR_INVALID_ARG;
    const void *w_read = dx != nullptr ? w : nullptr, *x_read = dw != nullptr ? x : nullptr;
    if (lies_on(dx, {dy, x_read, w, offsets}) || lies_on(dw, {dy, x, w_read, dx, offsets}))
      return MOE_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != MOE_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (d.R == 0)
    return cuda_status(no_rows(dw, (int64_t)d.E * d.N * d.K, dw_dtype, accumulate, s));
  cudaError_t e = cudaSuccess;
  if (dx != nullptr)
    e = launch_grouped_rows(grouped_product(d, offsets, x, w, dy, dx, d.dtype, workspace), true, s);
  if (e == cudaSuccess && dw != nullptr) {
    GroupedGemm g = grouped_product(d, offsets, x, w, dy, dw, dw_dtype, workspace);
    g.accumulate = accumulate;
    e = launch_grouped_weight_grad(g, s);
  }
  return cuda_status(e);
}

moe_status_t moe_quantize_int4(const void *w, int32_t dtype, int64_t rows, int32_t K, int32_t group,
                               void *q, void *scale, void *values, moe_stream_t stream) {
  if ((dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) || !ok_group(group))
    return MOE_ERR_INVALID_ARG;
  if (rows < 0 || rows > ((int64_t)1 << 27) || K < 32 || K > 1 << 18 || K % 32 != 0)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;  // empty tensors may have no address
  if (!ok_ptr(w) || !ok_ptr(q) || !ok_ptr(scale) || !ok_opt(values)) return MOE_ERR_INVALID_ARG;
  // values may be w: a thread writes what it alone has read
  if (lies_on(q, {w, scale, values}) || lies_on(scale, {w, values})) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_device();
  if (st != MOE_OK) return st;
  return cuda_status(launch_quantize_int4(w, dtype, rows, K, group, static_cast<uint8_t *>(q), scale,
                                          values, (cudaStream_t)stream));
}

moe_status_t moe_linear_int4(const moe_linear_desc_t *in, int32_t group, const void *x,
                             const void *q, const void *scale, const void *bias,
                             const void *residual, void *y, void *workspace, size_t ws_bytes,
                             moe_stream_t stream) {
  moe_linear_desc_t d;
  moe_status_t st = check_linear_desc(in, &d);
  if (st != MOE_OK) return st;
  if (d.dtype == MOE_DTYPE_E4M3 || !ok_group(group)) return MOE_ERR_INVALID_ARG;
  if (d.K % 32 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_ws(workspace, ws_bytes, moe_linear_workspace_size(in))) != MOE_OK) return st;
  if (d.T == 0) return MOE_OK;  // empty tensors may have no address
  if (!ok_ptr(x) || !ok_ptr(q) || !ok_ptr(scale) || !ok_opt(bias) || !ok_opt(residual) ||
      !ok_ptr(y))
    return MOE_ERR_INVALID_ARG;
  if (residual == y && d.residual_stride != d.y_stride) return MOE_ERR_INVALID_ARG;
  if (lies_on(y, {x, q, scale, bias})) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  Int4Gemm g = {};
  g.T = d.T;
  g.E = 1;
  g.N = d.N;
  g.K = d.K;
  g.group = group;
  g.dtype = d.dtype;
  g.out_dtype = d.out_dtype;
  g.act = d.act;
  g.x = x;
  g.q = static_cast<const uint8_t *>(q);
  g.scale = scale;
  g.bias = bias;
  g.residual = residual;
  g.y = y;
  g.ldx = d.x_stride;
  g.ldr = d.residual_stride;
  g.ldy = d.y_stride;
  g.part = reinterpret_cast<float *>(at(workspace, kStatusPad));
  g.status = static_cast<uint32_t *>(workspace);
  void *rows = at(workspace, kStatusPad + pad(int4_part_bytes(d.T)));
  return cuda_status(launch_int4(g, rows, (cudaStream_t)stream));
}

moe_status_t moe_grouped_linear_int4(const moe_grouped_desc_t *in, int32_t group, const void *x,
                                     const int32_t *offsets, const void *q, const void *scale,
                                     void *y, void *workspace, size_t ws_bytes,
                                     moe_stream_t stream) {
  moe_grouped_desc_t d;
  moe_status_t st = grouped_desc(in, &d);
  if (st != MOE_OK) return st;
  if (!ok_group(group)) return MOE_ERR_INVALID_ARG;
  if (d.K % 32 != 0 || d.R > kMaxT) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_ws(workspace, ws_bytes, grouped_ws(d).total)) != MOE_OK) return st;
  if (!ok_offsets(offsets)) return MOE_ERR_INVALID_ARG;
  if (d.R == 0) return MOE_OK;  // empty tensors may have no address
  if (!ok_ptr(x) || !ok_ptr(q) || !ok_ptr(scale) || !ok_ptr(y)) return MOE_ERR_INVALID_ARG;
  if (lies_on(y, {x, q, scale, offsets})) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  Int4Gemm g = {};
  g.T = d.R;
  g.E = d.E;
  g.N = d.N;
  g.K = d.K;
  g.group = group;
  g.dtype = d.dtype;
  g.out_dtype = d.out_dtype;
  g.act = MOE_ACT_NONE;
  g.offsets = offsets;
  g.x = x;
  g.q = static_cast<const uint8_t *>(q);
  g.scale = scale;
  g.y = y;
  g.ldx = d.x_stride;
  g.ldy = d.y_stride;
  g.part = reinterpret_cast<float *>(at(workspace, grouped_ws(d).part));
  g.status = static_cast<uint32_t *>(workspace);
  return cuda_status(launch_int4(g, at(workspace, grouped_ws(d).rows), (cudaStream_t)stream));
}

}  // extern "C"
