// Shared by the experts' ragged products (grouped_pair.cu) and their C ABI
// (api_grouped.cu).
#pragma once

#include "dense.cuh"

namespace moe {

// Rows [offsets[e], offsets[e+1]) of the row tensors belong to matrix e of w [E][N][K].
struct GroupedGemm {
  int R, E, N, K;
  int dtype;      // of every operand: MOE_DTYPE_BF16 or FP16
  int out_dtype;  // of the result
  const int32_t *offsets;
  const void *x, *w, *dy;     // x rows ldx apart, dy rows ldy apart
  int64_t ldx, ldy;
  void *d;                    // y (rows ldy apart), dx (rows ldx apart) or dw
  int accumulate;             // dw: added to what it holds
  float *part;                // partial sums of split tiles
  CUtensorMap *maps;          // dw: grouped_map_bytes(E)
  uint32_t *status;           // the workspace's status block
};

// Bytes of `part` for R rows.
size_t grouped_part_bytes(int R);
inline size_t grouped_map_bytes(int E) { return (size_t)E * 2 * sizeof(CUtensorMap); }

cudaError_t launch_grouped_rows(const GroupedGemm &g, bool grad, cudaStream_t s);
cudaError_t launch_grouped_weight_grad(const GroupedGemm &g, cudaStream_t s);

}  // namespace moe
