// Matrices to 4-bit codes with one scale for each group of a row's columns:
//   scale = max |w| / 7 (rounded to the weights' type),  code = round(w / scale) + 8
// Bound: HBM (2 bytes read, 1/2 written for each weight, 2 more where the values that
// the codes stand for are asked for).  A lane takes 8 weights (16 bytes) at a time, and
// has kAhead loads in flight; the 4 to 16 lanes of a group share their maximum by
// shuffles.  A block takes a stretch of chunks of 8 columns whatever the rows' length: one
// 64-bit division finds its first row, a multiplication the others.  32768 x 4096 with
// values: 107.5 us, 5.6 TB/s (four loads in flight and blocks that stay 112).
#include <algorithm>

#include "int4.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;
constexpr int kBlock = kThreads * kAhead;  // chunks of a block's stretch

// round(f / s) + 8 as the low bits of a float's, for a quotient in [-7.5, 7.5].  With f
// and s of 11 bits or fewer f / s is a half-integer exactly or away from it by more than
// 2^-13: rounded to a multiple of 2^-16 first (by adding 192), which takes away the
// error of the reciprocal, a tie is one again and goes to even.
constexpr float kFine = 192.f, kWhole = 12582912.f + 8.f - 192.f;  // 1.5 * 2^7, 1.5 * 2^23

template <int kGroup, bool kValues>
__global__ void __launch_bounds__(kThreads)
    quantize_int4_kernel(const uint4 *w, int dtype, int64_t total, int per_row,
                         uint32_t magic, int in_row, uint32_t *__restrict__ q,
                         uint16_t *__restrict__ scale, uint4 *values) {  // (values may be w)
  constexpr int kLanes = kGroup / 8;
  pdl_wait();
  pdl_launch_dependents();
  const int groups = per_row / kLanes;
  // smaller scales are coarse (fp16 subnormals) or have no reciprocal
  const float least = dtype == MOE_DTYPE_FP16 ? 0x1p-14f : 0x1p-100f;
  for (int64_t from = (int64_t)blockIdx.x * kBlock; from < total;
       from += (int64_t)gridDim.x * kBlock) {
    const int64_t row0 = from / per_row;
    const int first = (int)(from - row0 * per_row);
    uint4 v[kAhead];
    int64_t at[kAhead];  // of the chunk in w, or -1
    int64_t group[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // per_row chunks to a row, of which those from in_row on are past its end
      const uint32_t c = (uint32_t)(first + i * kThreads + (int)threadIdx.x);
      const uint32_t r = __umulhi(c, magic);
      const int in = (int)(c - r * (uint32_t)per_row);
      const bool ok = from + i * kThreads + threadIdx.x < total && in < in_row;
      at[i] = ok ? (row0 + r) * in_row + in : -1;
      group[i] = (row0 + r) * groups + in / kLanes;
      v[i] = ok ? __ldcs(w + at[i]) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
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
      if (at[i] < 0) continue;
      uint32_t code = 0;
      float value[8];
      if (s >= least && s <= 0x1p100f) {
        const float inv = 1.f / s;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float k = fmaf(f[j], inv, kFine) + kWhole;  // 1.5 * 2^23 + 8 + code
          code += (__float_as_uint(k) - 0x4b400000u) << (4 * j);
          value[j] = (k - 12582920.f) * s;
        }
      } else {
        // a scale of zero, or one that is no number: code 8 (zero)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = s > 0.f ? rintf(__fdiv_rn(f[j], s)) : 0.f;
          const float k = d == d ? fminf(fmaxf(d, -8.f), 7.f) : 0.f;
          code |= (uint32_t)((int)k + 8) << (4 * j);
          value[j] = k * s;
        }
      }
      q[at[i]] = code;
      if (kValues)
        __stcs(values + at[i],
               make_uint4(pack16(dtype, value[0], value[1]), pack16(dtype, value[2], value[3]),
                          pack16(dtype, value[4], value[5]), pack16(dtype, value[6], value[7])));
      if (threadIdx.x % kLanes == 0) scale[group[i]] = s16;
    }
  }
}

template <int kGroup>
cudaError_t start(const void *w, int dtype, int64_t rows, int K, uint8_t *q, void *scale,
                  void *values, cudaStream_t s) {
  const int per_row = (K + kGroup - 1) / kGroup * (kGroup / 8);
  const int64_t total = rows * per_row;
  // c / per_row = c * magic >> 32 for c < 2^16, as per_row <= 2^15
  const uint32_t magic = (uint32_t)((((uint64_t)1 << 32) + per_row - 1) / per_row);
  const int64_t blocks = (total + kBlock - 1) / kBlock;
  auto kern = values != nullptr ? quantize_int4_kernel<kGroup, true> : quantize_int4_kernel<kGroup, false>;
  return launch_pdl(kern, dim3((unsigned)std::min<int64_t>(blocks, (int64_t)num_sms() * 64)),
                    dim3(kThreads), 0, s, static_cast<const uint4 *>(w), dtype, total, per_row, magic,
                    K / 8, reinterpret_cast<uint32_t *>(q), static_cast<uint16_t *>(scale),
                    static_cast<uint4 *>(values));
}

}  // namespace

cudaError_t launch_quantize_int4(const void *w, int dtype, int64_t rows, int K, int group,
                                 uint8_t *q, void *scale, void *values, cudaStream_t s) {
  if (group == 32) return start<32>(w, dtype, rows, K, q, scale, values, s);
  return group == 64 ? start<64>(w, dtype, rows, K, q, scale, values, s)
                     : start<128>(w, dtype, rows, K, q, scale, values, s);
}

}  // namespace moe
