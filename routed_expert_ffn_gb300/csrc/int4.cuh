// Shared by the products with 4-bit weights (int4_small.cu, int4_tc.cu), the rows that they
// take (int4_rows.cu), the quantiser (quantize_int4.cu) and their C ABI (api_grouped.cu).
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
  int first;          // kInt4Rows at a time: row p of x is row p - first of xr
  const void *xr;     // rows as launch_int4_rows made them, and their factors
  const float *factor;
  float *part;        // int4_part_bytes(T): partial sums of split tiles
  size_t part_bytes;
  uint32_t *status;
};

// A row's scales of kCols columns, as they lie: two to a word.
template <int kGroup, int kCols>
struct UnitScales {
  static constexpr int count = kCols / kGroup;  // 1 to 8
  uint32_t w[(count + 1) / 2];
  __device__ __forceinline__ void load(const uint16_t *row, int unit, int groups) {
    const int g = unit * count;
    const uint16_t *p = row + g;
    if (groups % count == 0) {  // whole units, as aligned as they are long
      if constexpr (count == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
      } else if constexpr (count == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
      } else if constexpr (count == 2) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
      } else {
        w[0] = __ldg(p);
      }
    } else {
#pragma unroll
      for (int i = 0; i < count; i += 2) {
        const uint32_t lo = g + i < groups ? __ldg(p + i) : 0u;
        const uint32_t hi = g + i + 1 < groups ? __ldg(p + i + 1) : 0u;
        w[i / 2] = lo | hi << 16;
      }
    }
  }
};

__device__ __forceinline__ float scale_half(int dtype, uint32_t two, int i) {
  return unpack16(dtype, i ? two >> 16 : two).x;
}

// A word of eight codes as code - 8 in fp16, exactly: nibbles j and j + 4 are the halves of
// number pair j.  Masked where they lie, in the low or the next four bits of a half, and
// given the exponent under which those count ones, they are 1024 + code and 64 + code.
// One shift, four LOP3 and four subtractions; bf16, with seven bits beside the exponent,
// needs two shifts more, and the logic unit is what limits the unpacking.
// The constants stay in registers (the compiler does not see what they are): as literals
// they took two LOP3 and moves, a third of all instructions more.
struct Unpack {
  uint32_t one_low, one_high, zero_low, zero_high;
  __device__ __forceinline__ Unpack() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(one_low));    // 1024, twice
    asm volatile("mov.b32 %0, 0x54005400;" : "=r"(one_high));   // 64
    asm volatile("mov.b32 %0, 0x64086408;" : "=r"(zero_low));   // 1032
    asm volatile("mov.b32 %0, 0x54805480;" : "=r"(zero_high));  // 72
  }
  __device__ __forceinline__ static uint32_t pair(uint32_t w, uint32_t mask, uint32_t one,
                                                  uint32_t zero) {
    uint32_t d;
    asm("{\n\t.reg .b32 t;\n\t"
        "lop3.b32 t, %1, %2, %3, 0xEA;\n\t"  // (w & mask) | one
        "sub.rn.f16x2 %0, t, %4;\n\t}"
        : "=r"(d)
        : "r"(w), "r"(mask), "r"(one), "r"(zero));
    return d;
  }
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t *to) const {
    const uint32_t high = w >> 8;
    to[0] = pair(w, 0x000f000fu, one_low, zero_low);
    to[1] = pair(w, 0x00f000f0u, one_high, zero_high);
    to[2] = pair(high, 0x000f000fu, one_low, zero_low);
    to[3] = pair(high, 0x00f000f0u, one_high, zero_high);
  }
};

// 16 rows of W by 16 of depth by 8 rows of x.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same, the sums before it zero.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Rows of x in the order and with the factors that the products take (int4_rows.cu): fp16
// [rows][int4_pitch(K)], and what the sums are to be multiplied by.
inline int int4_pitch(int K) { return (K + 255) / 256 * 256; }
cudaError_t launch_int4_rows(const void *x, int64_t ldx, int dtype, int rows, int K, void *to,
                             float *factor, cudaStream_t s);
// The largest finite magnitude of eight numbers.
__device__ __forceinline__ float finite_max_bf16(const uint4 &v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16(MOE_DTYPE_BF16, w[i]);
    const float a = fabsf(f.x), b = fabsf(f.y);
    if (a < INFINITY) m = fmaxf(m, a);  // (false for NaN)
    if (b < INFINITY) m = fmaxf(m, b);
  }
  return m;
}
// The powers of two that bring a row's largest magnitude m to [2^14, 2^15) and its sums back.
// Smaller ones than 2^-112 are multiplied by 2^126.
struct RowFactor {
  float up, back;
};
__device__ __forceinline__ RowFactor row_factor(float m) {
  if (m == 0.f) return {1.f, 1.f};
  const int e = max((int)(__float_as_uint(m) >> 23) - 127 - 14, -126);
  return {__uint_as_float((uint32_t)(127 - e) << 23), __uint_as_float((uint32_t)(127 + e) << 23)};
}
// Eight numbers as the products take them.
__device__ __forceinline__ uint4 row_piece(uint4 v, int dtype, float up) {
  if (dtype == MOE_DTYPE_BF16) {
    uint32_t *w[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16(MOE_DTYPE_BF16, *w[i]);
      *w[i] = pack_f16x2(f.x * up, f.y * up);
    }
  }
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                    __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}
// At most this many rows at a time: the workspace holds them.
constexpr int kInt4Rows = 1024;

// Up to eight rows of one matrix, or few rows of experts (int4_small.cu); others (int4_tc.cu).
constexpr int kInt4SmallRows = 8;
cudaError_t launch_int4_small(const Int4Gemm &g, cudaStream_t s);
bool int4_few(const Int4Gemm &g);     // whether launch_int4_small is to take the experts' rows
bool int4_staged(const Int4Gemm &g);  // whether launch_int4_small makes the rows itself
cudaError_t launch_int4_tc(const Int4Gemm &g, cudaStream_t s);
// Bytes of `part`, and of rows and their factors.
size_t int4_part_bytes(int T);
inline size_t int4_rows_bytes(int T, int K) {
  const int rows = T < kInt4Rows ? T : kInt4Rows;
  return (size_t)rows * int4_pitch(K) * 2 + (size_t)rows * 4;
}

// codes, scales and (not null) the values that they stand for, of w [rows][K].
cudaError_t launch_quantize_int4(const void *w, int dtype, int64_t rows, int K, int group,
                                 uint8_t *q, void *scale, void *values, cudaStream_t s);

}  // namespace moe
