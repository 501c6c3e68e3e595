// The row-wise pass of the dense operators' gradients.
//
// act_grad: dz = dy act'(z), rounded once to the 16-bit type the gradient
// products take (more bits would take each product twice; bf16 gradients end 0.0023
// off in the 2-norm, with their own rounding alone 0.0017), with the column sums of the unrounded dz for the bias.
// Bound: HBM (dy and z read, dz written), of which it draws 60%: a thread's next
// loads start when those before are used (2047 x 4096 with GELU by tanh 14 to 17 us,
// 67 MB).  A CTA takes 128 columns (a lane 4
// of them: 16 bytes of z, 8 of dy) and one slice of the rows, four rows a
// thread in flight.  A slice's column sums go to the workspace; the last CTA
// of the columns adds the slices in order, so the sums do not change from run
// to run (a kernel of its own for that cost 4 us of a gradient of 110).
#include <algorithm>

#include "dense.cuh"

namespace moe {

namespace {

constexpr int kCols = 128, kRowLanes = 8, kAhead = 4;
constexpr int kCtas = 4 * 152;

struct ActGradArgs {
  const uint16_t *dy;
  const float *z;
  uint16_t *dz;
  float *part, *dbias;
  uint32_t *counter;  // one for each 128 columns, zero before and after
  int64_t ldy;
  int T, N, rows, act, dtype, accumulate;
};

template <int kAct>
__device__ __forceinline__ void act_grad_rows(const ActGradArgs &a, int c, int r0, int r1,
                                              float (&sum)[4]) {
  for (int r = r0; r < r1; r += kRowLanes * kAhead) {
    uint2 dy[kAhead];
    float4 z[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int row = r + i * kRowLanes;
      if (row < r1) {
        dy[i] = __ldg(reinterpret_cast<const uint2 *>(a.dy + (int64_t)row * a.ldy + c));
        if (kAct != MOE_ACT_NONE)
          z[i] = __ldg(reinterpret_cast<const float4 *>(a.z + (int64_t)row * a.N + c));
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int row = r + i * kRowLanes;
      if (row >= r1) break;
      const float2 lo = unpack16(a.dtype, dy[i].x), hi = unpack16(a.dtype, dy[i].y);
      float d[4] = {lo.x, lo.y, hi.x, hi.y};
      if (kAct != MOE_ACT_NONE) {
        const float zz[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] *= activate_slope(kAct, zz[j]);
        if (a.dz != nullptr)
          *reinterpret_cast<uint2 *>(a.dz + (int64_t)row * a.N + c) =
              make_uint2(pack16(a.dtype, d[0], d[1]), pack16(a.dtype, d[2], d[3]));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += d[j];
    }
  }
}

__global__ void __launch_bounds__(256) act_grad_kernel(const ActGradArgs a) {
  __shared__ float s[kRowLanes][kCols];
  __shared__ bool last;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c0 = blockIdx.x * kCols, c = c0 + tx * 4;
  const int first = blockIdx.y * a.rows, r0 = first + ty, r1 = min(a.T, first + a.rows);
  pdl_wait();
  pdl_launch_dependents();
  float sum[4] = {};
  if (c < a.N) {
    switch (a.act) {
      case MOE_ACT_RELU: act_grad_rows<MOE_ACT_RELU>(a, c, r0, r1, sum); break;
      case MOE_ACT_GELU: act_grad_rows<MOE_ACT_GELU>(a, c, r0, r1, sum); break;
      case MOE_ACT_GELU_TANH: act_grad_rows<MOE_ACT_GELU_TANH>(a, c, r0, r1, sum); break;
      case MOE_ACT_SILU: act_grad_rows<MOE_ACT_SILU>(a, c, r0, r1, sum); break;
      default: act_grad_rows<MOE_ACT_NONE>(a, c, r0, r1, sum); break;
    }
  }
  if (a.dbias == nullptr) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) s[ty][tx * 4 + i] = sum[i];
  __syncthreads();
  const int j = threadIdx.x & (kCols - 1), col = c0 + j;
  if (threadIdx.x < kCols && col < a.N) {
    float v = 0.f;
    for (int i = 0; i < kRowLanes; ++i) v += s[i][j];
    a.part[(int64_t)blockIdx.y * a.N + col] = v;
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(a.counter + blockIdx.x, 1u) == gridDim.y - 1;
    if (last) a.counter[blockIdx.x] = 0;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  // two threads a column, half of the slices each
  const int half = threadIdx.x / kCols, mid = gridDim.y / 2;
  float v = 0.f;
  if (col < a.N) {
    const int from = half == 0 ? 0 : mid, to = half == 0 ? mid : (int)gridDim.y;
#pragma unroll 4
    for (int i = from; i < to; ++i) v += __ldcg(a.part + (int64_t)i * a.N + col);
  }
  __syncthreads();
  if (half == 1) s[0][j] = v;
  __syncthreads();
  if (half == 0 && col < a.N) {
    v += s[0][j];
    a.dbias[col] = a.accumulate ? a.dbias[col] + v : v;
  }
}

}  // namespace

// Slices of the rows: about four CTAs an SM, each with at least 32 rows.
int act_grad_slices(int T, int N) {
  const int cols = (N + kCols - 1) / kCols;
  return std::max(1, std::min((kCtas + cols - 1) / cols, (T + 31) / 32));
}

cudaError_t launch_act_grad(const void *dy, int64_t ldy, const float *z, int T, int N, int act,
                            int dtype, void *dz, float *part, uint32_t *counter, float *dbias,
                            int accumulate, cudaStream_t s) {
  const int slices = act_grad_slices(T, N);
  ActGradArgs a = {};
  a.dy = static_cast<const uint16_t *>(dy);
  a.z = z;
  a.dz = static_cast<uint16_t *>(dz);
  a.part = part;
  a.dbias = dbias;
  a.counter = counter;
  a.ldy = ldy;
  a.T = T;
  a.N = N;
  a.rows = (T + slices - 1) / slices;
  a.act = act;
  a.dtype = dtype;
  a.accumulate = accumulate;
  return launch_pdl(act_grad_kernel, dim3((unsigned)((N + kCols - 1) / kCols), (unsigned)slices),
                    dim3(256), 0, s, a);
}

}  // namespace moe
