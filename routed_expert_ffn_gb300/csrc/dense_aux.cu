// The row-wise passes of the dense operators' gradients.
//
// act_grad: dz = dy act'(z), rounded once to the 16-bit type the gradient
// products take, with the column sums of the unrounded dz for the bias.
// Bound: HBM (dy and z read, dz written).  A CTA takes 256 columns (a thread
// 8 of them) and one slice of the rows; the slices' column sums are partials
// that column_sum adds in a fixed order.
#include <algorithm>

#include "dense.cuh"

namespace moe {

namespace {

constexpr int kCols = 256, kRowLanes = 8;  // 32 threads x 8 columns, 8 rows at a time

__global__ void __launch_bounds__(256)
    act_grad_kernel(const uint16_t *__restrict__ dy, int64_t ldy, const float *__restrict__ z,
                    int T, int N, int rows, int act, int dtype, uint16_t *__restrict__ dz,
                    float *__restrict__ part) {
  __shared__ float s[kRowLanes][kCols];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * kCols + tx * 8;
  const int r0 = blockIdx.y * rows, r1 = min(T, r0 + rows);
  pdl_wait();
  pdl_launch_dependents();
  float sum[8] = {};
  if (c < N) {
#pragma unroll 2
    for (int r = r0 + ty; r < r1; r += kRowLanes) {
      const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(dy + (int64_t)r * ldy + c));
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      float d[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack16(dtype, w[i]);
        d[2 * i] = v.x;
        d[2 * i + 1] = v.y;
      }
      if (z != nullptr) {
        const float4 *p = reinterpret_cast<const float4 *>(z + (int64_t)r * N + c);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        const float zz[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= activate_slope(act, zz[i]);
      }
      if (dz != nullptr)
        *reinterpret_cast<uint4 *>(dz + (int64_t)r * N + c) =
            make_uint4(pack16(dtype, d[0], d[1]), pack16(dtype, d[2], d[3]),
                       pack16(dtype, d[4], d[5]), pack16(dtype, d[6], d[7]));
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[ty][tx * 8 + i] = sum[i];
  __syncthreads();
  const int col = blockIdx.x * kCols + threadIdx.x;
  if (col < N) {
    float v = 0.f;
    for (int i = 0; i < kRowLanes; ++i) v += s[i][threadIdx.x];
    part[(int64_t)blockIdx.y * N + col] = v;
  }
}

}  // namespace

// Slices of the rows: about four CTAs for each of 152 SMs, each with at least
// 16 rows.
int act_grad_slices(int T, int N) {
  const int cols = (N + kCols - 1) / kCols;
  return std::max(1, std::min((608 + cols - 1) / cols, (T + 15) / 16));
}

cudaError_t launch_act_grad(const void *dy, int64_t ldy, const float *z, int T, int N, int act,
                            int dtype, void *dz, float *part, cudaStream_t s) {
  const int slices = act_grad_slices(T, N);
  const int rows = (T + slices - 1) / slices;
  return launch_pdl(act_grad_kernel, dim3((unsigned)((N + kCols - 1) / kCols), (unsigned)slices),
                    dim3(256), 0, s, static_cast<const uint16_t *>(dy), ldy, z, T, N, rows, act,
                    dtype, static_cast<uint16_t *>(dz), part);
}

}  // namespace moe
