// Matrices to 4-bit codes with one scale for each group of a row's columns:
//   scale = max |w| / 7 (rounded to the weights' type),  code = round(w / scale) + 8
// Bound: HBM (2 bytes read, 1/2 written for each weight, 2 more where the values
// that the codes stand for are asked for).  A lane takes 8 weights (16 bytes) at a
// time; the 4 to 16 lanes of a group share their maximum by shuffles.  A block's
// threads divide into rows of enough threads for one row's columns, so that narrow
// matrices fill a block too; each thread has the loads of kRows rows in flight.
#include <algorithm>

#include "int4.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;

// round(f / s) to even, in [-8, 7], by the reciprocal of s.  With f and s of 11 bits or
// fewer f / s is a half-integer exactly or away from it by more than 2^-14, far above
// the error of f * inv: only ties could go wrong, and their remainder is exact.
__device__ __forceinline__ float rounded_quotient(float f, float s, float inv) {
  const float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  const float t = fminf(fmaxf(f * inv, -8.f), 7.f);
  const float k = (t + kRound) - kRound;
  const float left = fmaf(-k, s, f);
  const bool odd = (__float_as_uint(t + kRound) & 1u) != 0;
  return odd && 2.f * fabsf(left) == s ? k + copysignf(1.f, left) : k;
}

template <int kGroup>
__global__ void __launch_bounds__(kThreads)
    quantize_int4_kernel(const uint16_t *__restrict__ w, int dtype, int64_t rows, int K, int per_row,
                         uint8_t *__restrict__ q, uint16_t *__restrict__ scale,
                         uint16_t *__restrict__ values) {
  constexpr int kLanes = kGroup / 8;
  pdl_wait();
  pdl_launch_dependents();
  const int groups = (K + kGroup - 1) / kGroup;
  const int chunks = groups * kLanes;  // of 8 columns, past K none
  const int in_block = kThreads / per_row;  // rows
  const int first = threadIdx.x % per_row;
  const int64_t step = (int64_t)gridDim.x * in_block;
  const int64_t r0 = (int64_t)blockIdx.x * in_block + threadIdx.x / per_row;
  // every thread of a warp takes as many turns
  const int64_t turns = (rows + step - 1) / step;
  for (int64_t turn = 0; turn < turns; turn += kRows) {
    for (int c0 = 0; c0 < chunks; c0 += per_row) {
      const int c = c0 + first;
      const bool in_row = c * 8 < K;
      uint4 v[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + (turn + i) * step;
        v[i] = in_row && r < rows ? __ldcs(reinterpret_cast<const uint4 *>(w + r * K) + c)
                                  : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + (turn + i) * step;
        const uint32_t word[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = unpack16(dtype, word[j]);
          f[2 * j] = u.x;
          f[2 * j + 1] = u.y;
        }
        float most = 0.f;  // NaN where one of them is
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmax_nan(most, fabsf(f[j]));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1)
          most = fmax_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
        const uint16_t s16 = (uint16_t)pack16(dtype, __fdiv_rn(most, 7.f), 0.f);
        const float s = unpack16(dtype, s16).x;
        uint32_t code = 0;
        float value[8];
        // reciprocals of the smallest numbers overflow
        const bool normal = s > 0x1p-100f && s < 0x1p100f;
        const float inv = normal ? __frcp_rn(s) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float k;
          if (normal) {
            k = rounded_quotient(f[j], s, inv);
          } else {
            // a scale of zero, or one that is no number: code 8 (zero)
            const float d = s > 0.f ? rintf(__fdiv_rn(f[j], s)) : 0.f;
            k = d == d ? fminf(fmaxf(d, -8.f), 7.f) : 0.f;
          }
          code |= (uint32_t)(__float_as_uint(k + 12582920.f) & 15u) << (4 * j);
          value[j] = k * s;
        }
        if (in_row && r < rows) {
          reinterpret_cast<uint32_t *>(q + r * (K / 2))[c] = code;
          if (values != nullptr)
            reinterpret_cast<uint4 *>(values + r * K)[c] =
                make_uint4(pack16(dtype, value[0], value[1]), pack16(dtype, value[2], value[3]),
                           pack16(dtype, value[4], value[5]), pack16(dtype, value[6], value[7]));
          if (c % kLanes == 0) scale[r * groups + c / kLanes] = s16;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_quantize_int4(const void *w, int dtype, int64_t rows, int K, int group,
                                 uint8_t *q, void *scale, void *values, cudaStream_t s) {
  const int lanes = group / 8, chunks = (K + group - 1) / group * lanes;
  int per_row = 32;  // a power of two: whole warps, or (never less than) a group's lanes
  while (per_row < kThreads && per_row < chunks) per_row *= 2;
  while (per_row > lanes && per_row / 2 >= chunks) per_row /= 2;
  const int in_block = kThreads / per_row;
  const int64_t blocks = (rows + in_block - 1) / in_block;
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms() * 8);
  auto kern = group == 32 ? quantize_int4_kernel<32>
                          : (group == 64 ? quantize_int4_kernel<64> : quantize_int4_kernel<128>);
  return launch_pdl(kern, dim3(grid), dim3(kThreads), 0, s, static_cast<const uint16_t *>(w), dtype,
                    rows, K, per_row, q, static_cast<uint16_t *>(scale),
                    static_cast<uint16_t *>(values));
}

}  // namespace moe
