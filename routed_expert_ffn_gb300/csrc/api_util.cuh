// What the C ABI's argument checks share (api_dense.cu, api_grouped.cu).
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "moe_internal.cuh"

namespace moe {

inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A workspace of at least `need` bytes, aligned to 256.
inline moe_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// Whether `out` is at the address of one of `others` that the call still reads, or
// writes too (null: no argument).
inline bool lies_on(const void *out, std::initializer_list<const void *> others) {
  for (const void *p : others)
    if (out != nullptr && out == p) return true;
  return false;
}

// A row stride in elements: 0 (dense) becomes `cols`; otherwise at least
// `cols` and a multiple of `mult`.
inline bool fix_stride(int64_t *stride, int64_t cols, int mult) {
  if (*stride == 0) *stride = cols;
  return *stride >= cols && *stride % mult == 0 && *stride < ((int64_t)1 << 36);
}

// A validated copy of the descriptor with its strides filled in (api_dense.cu).
moe_status_t check_linear_desc(const moe_linear_desc_t *in, moe_linear_desc_t *d);

inline size_t pad(size_t n) { return (n + 1023) / 1024 * 1024; }

inline uint8_t *at(void *ws, size_t off) { return static_cast<uint8_t *>(ws) + off; }

// The gradient of a weight over no rows: zeros, or what is accumulated.
inline cudaError_t no_rows(void *dw, int64_t n, int dw_dtype, int accumulate, cudaStream_t s) {
  if (dw == nullptr || accumulate) return cudaSuccess;
  return cudaMemsetAsync(dw, 0, (size_t)n * (dw_dtype == MOE_DTYPE_FP32 ? 4 : 2), s);
}

}  // namespace moe
