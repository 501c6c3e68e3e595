// Rows of x as the products with 4-bit weights multiply them: fp16, each row times a power of
// two, and the eight columns of a word of codes in the order 0 4 1 5 2 6 3 7, in which
// the word is unpacked (int4.cuh).
//
// fp16 has three more significant bits than bf16, but not its range: a row's largest
// number is brought to 2^14 or more, so that all down to 2^-28 of it are exact and smaller
// ones off by 2^-39 of it at most, below what fp32 sums resolve.  Infinities and NaN stay
// what they are.  fp16 rows are only put in order.  Past K a row is zero.
#include "int4.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    int4_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, int dtype, int K, int pitch,
                     uint16_t *__restrict__ to, float *__restrict__ factor) {
  __shared__ float most[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const uint4 *row = reinterpret_cast<const uint4 *>(x + (int64_t)blockIdx.x * ldx);
  uint4 *out = reinterpret_cast<uint4 *>(to + (int64_t)blockIdx.x * pitch);
  float up = 1.f;
  if (dtype == MOE_DTYPE_BF16) {
    float m = 0.f;
    for (int c = threadIdx.x; c < K / 8; c += kThreads) m = fmaxf(m, finite_max_bf16(row[c]));
    // non-negative floats are in the order of their bits
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, most[i]);
    const RowFactor f = row_factor(m);
    up = f.up;
    if (threadIdx.x == 0) factor[blockIdx.x] = f.back;
  } else if (threadIdx.x == 0) {
    factor[blockIdx.x] = 1.f;
  }
  for (int c = threadIdx.x; c < pitch / 8; c += kThreads) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < K / 8) v = row[c];
    out[c] = row_piece(v, dtype, up);
  }
}

}  // namespace

cudaError_t launch_int4_rows(const void *x, int64_t ldx, int dtype, int rows, int K, void *to,
                             float *factor, cudaStream_t s) {
  return launch_pdl(int4_rows_kernel, dim3((unsigned)rows), dim3(kThreads), 0, s,
                    static_cast<const uint16_t *>(x), ldx, dtype, K, int4_pitch(K),
                    static_cast<uint16_t *>(to), factor);
}

}  // namespace moe
