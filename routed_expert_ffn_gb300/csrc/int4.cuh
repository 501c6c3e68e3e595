// Shared by the products with 4-bit weights (int4_small.cu), the quantiser
// (quantize_int4.cu) and their C ABI (api_grouped.cu).
#pragma once

#include "dense.cuh"

namespace moe {

// y = act(x W^T + bias) + residual, or for each expert's rows y_p = W_e x_p, with W in 4
// bits: codes [E][N][K/2] (the even column's in a byte's low half) stand for code - 8,
// times scale [E][N][ceil(K/group)].
struct Int4Gemm {
  int T, E, N, K, group;
  int dtype;      // of x and the scales
  int out_dtype;  // of y, bias and residual
  int act;
  const int32_t *offsets;  // null: one matrix, rows [0, T)
  const void *x;
  const uint8_t *q;
  const void *scale;
  const void *bias, *residual;
  void *y;
  int64_t ldx, ldr, ldy;
  float *part;  // int4_part_bytes(T): partial sums of split tiles
  uint32_t *status;
};

cudaError_t launch_int4_small(const Int4Gemm &g, cudaStream_t s);
cudaError_t launch_int4_tc(const Int4Gemm &g, cudaStream_t s);
size_t int4_part_bytes(int T);

// codes, scales and (not null) the values that they stand for, of w [rows][K].
cudaError_t launch_quantize_int4(const void *w, int dtype, int64_t rows, int K, int group,
                                 uint8_t *q, void *scale, void *values, cudaStream_t s);

}  // namespace moe
