// Shared by the dense operators' GEMMs (dense_pair.cu, dense_small.cu): the
// description of a launch, activations, and the packing of output elements.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// What is done with the accumulator before it is stored.
//   kEpiLinear  D = act(acc + bias) + residual; acc + bias to `preact` if asked
//   kEpiGated   the accumulators g and u of a gate and an up column: h = silu(g) u;
//               g and u to `saved` if asked
//   kEpiGatedGrad  acc = dh with g and u from `saved`: dg, du and h
enum { kEpiLinear = 0, kEpiGated = 1, kEpiGatedGrad = 2 };

// One product D[M,N] = sum over k of A(m,k) B(n,k), row-major D.
// An operand is K-major (rows of K elements, `ld` apart) or MN-major (its K
// index runs over the rows, `ld` apart): gradients read the same tensors as
// the forward product, without a transposed copy.
struct DenseGemm {
  int M, N, K;      // kEpiGated: N = columns of h (I)
  int epi;
  int dtype;        // A and B: MOE_DTYPE_BF16, FP16 or E4M3
  int out_dtype;    // D (kEpiLinear): BF16, FP16 or FP32
  int act;          // kEpiLinear
  bool a_mn, b_mn;  // MN-major operands
  const void *a, *b;
  int64_t lda, ldb;
  const void *bias, *residual;  // out_dtype; residual rows ldr apart; may be null
  void *d;                      // rows ldd apart; kEpiGatedGrad: null
  int64_t ldr, ldd;
  float *preact;  // kEpiLinear: [M][N] fp32 or null
  float *saved;   // [M][2N] fp32: g then u.  kEpiGated: out or null; kEpiGatedGrad: in
  void *dgu, *h;  // kEpiGatedGrad: [M][2N] and [M][N] out
  const int8_t *a_scale, *b_scale;  // E4M3: exponents [M][ceil(K/128)], [ceil(N/128)][ceil(K/128)]
  uint32_t *status;
};

// Prefill and training sizes: 256-row tiles on CTA pairs (dense_pair.cu).
cudaError_t launch_dense_pair(const DenseGemm &g, cudaStream_t s);
// Two or three products with MN-major B and nothing but a residual in their
// epilogues, in one launch: g[1] and g[2] of equal depth, g[0] of any.
cudaError_t launch_dense_multi(const DenseGemm *g, int n, cudaStream_t s);
// Few rows: weight rows as the MMA's M, rows of A as its N, K split over a
// cluster (dense_small.cu).  A K-major, B either (MN-major: 16 bits, not gated), no
// preact or saved, at most kSmallRows rows.
constexpr int kSmallRows = 1024;
cudaError_t launch_dense_small(const DenseGemm &g, cudaStream_t s);
// Tiles of rows x cols, K split in `split`, and what that is estimated to take, in us
// (0 if it cannot be told).
struct DensePlan {
  int rows, cols, split;
  float us;
};
DensePlan dense_pair_plan(const DenseGemm &g);
DensePlan dense_small_plan(const DenseGemm &g);
inline float dense_pair_us(const DenseGemm &g) { return dense_pair_plan(g).us; }
inline float dense_small_us(const DenseGemm &g) { return dense_small_plan(g).us; }
float dense_multi_us(const DenseGemm *g, int n);

// dz = dy act'(z) in 16 bits (act none: not written) and the column sums of the
// unrounded dz to dbias (null: none), by way of part [slices][N] and one zero
// counter for each 128 columns.
int act_grad_slices(int T, int N);
cudaError_t launch_act_grad(const void *dy, int64_t ldy, const float *z, int T, int N, int act,
                            int dtype, void *dz, float *part, uint32_t *counter, float *dbias,
                            int accumulate, cudaStream_t s);

// ------------------------------------------------------------ element types --

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Two fp32 values to a word of the 16-bit output type (round to nearest even).
__device__ __forceinline__ uint32_t pack16(int dtype, float lo, float hi) {
  return dtype == MOE_DTYPE_FP16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
__device__ __forceinline__ float2 unpack16(int dtype, uint32_t w) {
  if (dtype == MOE_DTYPE_FP16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// -------------------------------------------------------------- activations --

constexpr float kGeluC0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;

// The approximate division: 2 ulp, and 0 where 1 + e^-z overflows.  Unless kExact, the
// approximate exponential too, whose error grows with |z| (2^-22 of the result at 0,
// 2^-19 at 16): enough for results that are rounded to 16 bits next.
template <bool kExact = false>
__device__ __forceinline__ float sigmoid(float z) {
  return __fdividef(1.0f, 1.0f + (kExact ? expf(-z) : __expf(-z)));
}

// kExact: to a few fp32 steps for any z, for fp32 results.  2048 x 8192 x 1024 with
// SiLU takes 36.4 us so and 28.0 without, with GELU 78.7 and 44.8.
template <bool kExact>
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    // comparisons that let a NaN through
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;
    case MOE_ACT_GELU:
      // 1 + erf v = erfc(-v), where nothing cancels far below zero
      return 0.5f * z *
             (kExact ? erfcf(z * -0.7071067811865476f) : 1.0f + erff(z * 0.7071067811865476f));
    case MOE_ACT_GELU_TANH: {
      // 1/2 (1 + tanh v) = sigmoid(2 v)
      return z * sigmoid<kExact>(2.0f * kGeluC0 * (z + kGeluC1 * z * z * z));
    }
    case MOE_ACT_SILU: return z * sigmoid<kExact>(z);
    default: return z;
  }
}

// All of an array, the choice made once.
template <bool kExact, int kAct, int kN>
__device__ __forceinline__ void activate_as(float (&f)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) f[i] = activate<kExact>(kAct, f[i]);
}
template <bool kExact, int kN>
__device__ __forceinline__ void activate_all(int act, float (&f)[kN]) {
  switch (act) {
    case MOE_ACT_RELU: return activate_as<kExact, MOE_ACT_RELU>(f);
    case MOE_ACT_GELU: return activate_as<kExact, MOE_ACT_GELU>(f);
    case MOE_ACT_GELU_TANH: return activate_as<kExact, MOE_ACT_GELU_TANH>(f);
    case MOE_ACT_SILU: return activate_as<kExact, MOE_ACT_SILU>(f);
    default: return;
  }
}

// The activation's slope at z.
__device__ __forceinline__ float activate_slope(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
    case MOE_ACT_GELU:
      return 0.5f * (1.0f + erff(z * 0.7071067811865476f)) +
             z * __expf(-0.5f * z * z) * 0.3989422804014327f;  // 1 / sqrt(2 pi)
    case MOE_ACT_GELU_TANH: {
      // with p = sigmoid(2v): p + 2 z p (1 - p) dv/dz; beyond |z| = 30 the
      // second term is zero, and z^2 does not overflow
      const float p = sigmoid(2.0f * kGeluC0 * (z + kGeluC1 * z * z * z));
      const float c = fminf(fmaxf(z, -30.f), 30.f);
      return p + 2.0f * c * p * (1.0f - p) * kGeluC0 * (1.0f + 3.0f * kGeluC1 * c * c);
    }
    case MOE_ACT_SILU: {
      const float p = sigmoid(z);
      return p * (1.0f + z * (1.0f - p));
    }
    default: return 1.f;
  }
}

// ------------------------------------------------------------ MMA operands --

// Instruction descriptor of kind::f16 with fp32 accumulators for either 16-bit
// type and majorness (bits 7-9 and 10-12: 0 fp16, 1 bf16; bits 15, 16: MN-major).
__host__ __device__ constexpr uint32_t idesc_16(int dtype, bool a_mn, bool b_mn, int M, int N) {
  const uint32_t f = dtype == MOE_DTYPE_BF16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Words of the shared-memory descriptors of operands in 128-byte swizzled
// boxes, without the address (bits 0-13 of the low word, in 16-byte units).
// Low word, from bit 16: leading offset; high word: stride offset, version 1
// (bit 14), swizzle mode 2 (bits 29-31).
//   K-major:  rows of 128 bytes, groups of 8 rows 1024 bytes apart (stride)
//   MN-major: boxes of 64 MN elements by 64 K rows (8 KB): groups of 8 K rows
//             1024 bytes apart (stride), boxes 8192 bytes apart (leading)
constexpr uint32_t kDescLoK = 1u << 16, kDescLoMn = (8192u >> 4) << 16;
constexpr uint32_t kDescHiK = (1024u >> 4) | (1u << 14) | (2u << 29), kDescHiMn = kDescHiK;
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  return (uint64_t)kDescHiMn << 32 | kDescLoMn | (saddr & 0x3FFFFu) >> 4;
}

// 32 lanes x 32 consecutive 32-bit columns; thread i gets lane (base + i).
// The wait is part of the same statement: no use can move in front of it.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&f)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float (&f)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}

// ------------------------------------------------ block-scaled E4M3 products --

// Instruction descriptor of kind::mxf8f6f4: E4M3 operands (types 0), both
// K-major, scale factors UE8M0 (bit 23), scale-factor bytes 0 of both, N >> 3
// in bits 17-22, M >> 7 in bits 27-28.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N) {
  return ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}

// Which of a scale-factor word's bytes the MMA takes, for both operands.
__host__ __device__ constexpr uint32_t idesc_sf_byte(uint32_t b) { return (b << 4) | (b << 29); }

// Scale-factor columns: 4 for 128 rows of A, 8 for 256 rows of B.
constexpr uint32_t kSfCols = 12;

// A block exponent as four equal UE8M0 bytes (2^(byte - 127)).
__device__ __forceinline__ uint32_t e8m0x4(int8_t e) {
  return (uint32_t)((int)e + 127) * 0x01010101u;
}

// Four successive block exponents as UE8M0 bytes; of those past `left` (which
// no product takes) none is read.
__device__ __forceinline__ uint32_t e8m0_4(const int8_t *e, int left) {
  uint32_t w = 0x7f7f7f7fu;
  if (left >= 4 && (reinterpret_cast<uintptr_t>(e) & 3u) == 0)
    return __vadd4(__ldg(reinterpret_cast<const uint32_t *>(e)), w);
  w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) w |= (uint32_t)((int)__ldg(e + i) + 127) << (8 * i);
  return w;
}

// D (+)= (A * 2^sfa) (B * 2^sfb)^T, 32 of K, one CTA.
__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
          "r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// This warp's 32 lanes x 4 columns.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------- tensor maps --

inline CUtensorMapDataType map_type(int dtype) {
  switch (dtype) {
    case MOE_DTYPE_BF16: return CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    case MOE_DTYPE_FP16: return CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    case MOE_DTYPE_FP32: return CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    default: return CU_TENSOR_MAP_DATA_TYPE_UINT8;
  }
}
inline int type_bytes(int dtype) {
  return dtype == MOE_DTYPE_FP32 ? 4 : (dtype == MOE_DTYPE_E4M3 ? 1 : 2);
}
// What HBM needs for B (a gated product's: both halves), in us.
inline float weight_us(const DenseGemm &g) {
  return (float)g.N * (float)g.K * (g.epi == kEpiGated ? 2.f : 1.f) *
         (float)type_bytes(g.dtype) / 6.6e6f;
}

// [rows][cols] with rows `ld` elements apart, boxes of box_rows x box_cols.
inline bool map_2d(CUtensorMap *m, int dtype, CUtensorMapSwizzle sw, const void *p, int64_t rows,
                   int64_t cols, int64_t ld, int box_rows, int box_cols) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * type_bytes(dtype)};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  return encode_map(m, map_type(dtype), sw, p, 2, dims, strides, box);
}
// Two matrices [rows][cols], `ld` between rows and `plane` between the two;
// a box holds box_planes of them.
inline bool map_two(CUtensorMap *m, int dtype, CUtensorMapSwizzle sw, const void *p, int64_t rows,
                    int64_t cols, int64_t ld, int64_t plane, int box_rows, int box_cols,
                    int box_planes) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 2};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * type_bytes(dtype),
                                 (cuuint64_t)plane * type_bytes(dtype)};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, (cuuint32_t)box_planes};
  return encode_map(m, map_type(dtype), sw, p, 3, dims, strides, box);
}

}  // namespace moe
