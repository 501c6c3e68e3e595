// What the matrix kernels on CTA pairs share: the 16-bit MMA, tensor copies, and the
// way of 32 x 32 blocks of results through shared memory (dense_pair.cu,
// grouped_pair.cu).
#pragma once

#include "dense.cuh"
#include "pair_ptx.cuh"

namespace moe {

constexpr uint32_t kSlotBytes = 2048;  // 32 x 32 16-bit values

// D (+)= A B^T over the pair, 16 of K; operand descriptors as low and high words.
__device__ __forceinline__ void umma_16_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                             uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *m, uint32_t bar,
                                                 int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int c0,
                                             int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::
                   "l"(m),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, const void *src, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}

// An arrival that hands over TMEM alone: tcgen05.fence orders the reads before
// it, and no memory is released (a release at cluster scope takes 0.85 us, which
// a tile of few K stages waits for).
__device__ __forceinline__ void arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A warp's output buffer: kCount slots of 32 x 32 16-bit values, of which two
// hold one of fp32.
template <int kCount>
struct Slots {
  uint8_t *base;
  uint32_t next;
  bool wide;  // the last store was fp32
  // Each waits for the stores that still read what it hands out.
  __device__ __forceinline__ uint8_t *take16(int lane) {
    if (lane == 0) {
      if (wide)
        bulk_wait_read<0>();
      else
        bulk_wait_read<kCount - 1>();
    }
    wide = false;
    __syncwarp();
    uint8_t *p = base + next * kSlotBytes;
    next = next + 1 == kCount ? 0 : next + 1;
    return p;
  }
  __device__ __forceinline__ uint8_t *take32(int lane) {
    if (lane == 0) bulk_wait_read<0>();
    wide = true;
    __syncwarp();
    return base;
  }
};

// 32 rows (lanes) of 32 values to a slot in the layout of the TMA store's
// swizzle: 16-bit rows of 64 bytes, 16-byte chunk c at c ^ ((row >> 1) & 3);
// fp32 rows of 128 bytes, chunk c at c ^ (row & 7).
__device__ __forceinline__ void put16(uint8_t *slot, int lane, int dtype, const float (&f)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 w = make_uint4(pack16(dtype, f[8 * c], f[8 * c + 1]),
                               pack16(dtype, f[8 * c + 2], f[8 * c + 3]),
                               pack16(dtype, f[8 * c + 4], f[8 * c + 5]),
                               pack16(dtype, f[8 * c + 6], f[8 * c + 7]));
    *reinterpret_cast<uint4 *>(slot + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = w;
  }
}
__device__ __forceinline__ void put16(uint8_t *slot, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4 *>(slot + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
__device__ __forceinline__ void put32(uint8_t *slot, int lane, const float (&f)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4 *>(slot + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_float4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]);
}
// Adds what put32 left.
__device__ __forceinline__ void add32(float (&f)[32], const uint8_t *slot, int lane) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float4 v = *reinterpret_cast<const float4 *>(slot + lane * 128 + ((c ^ (lane & 7)) << 4));
    f[4 * c] += v.x;
    f[4 * c + 1] += v.y;
    f[4 * c + 2] += v.z;
    f[4 * c + 3] += v.w;
  }
}
__device__ __forceinline__ void send_2d(const CUtensorMap *m, uint8_t *slot, int lane, int c0,
                                        int c1) {
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(m, slot, c0, c1);
    bulk_commit();
  }
}
__device__ __forceinline__ void send_3d(const CUtensorMap *m, uint8_t *slot, int lane, int c0,
                                        int c1, int c2) {
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(m, slot, c0, c1, c2);
    bulk_commit();
  }
}

// 32 rows of 32 values of the output type: loaded four lanes (16 bits) or eight
// (fp32) to a row, so that a request takes whole sectors of few lines -- a lane
// to a row made the epilogue of 4096 x 4096 with a residual 14 us longer -- and
// turned by way of the output slot so that lane r has row r.  Rows and columns
// past the ends are zero.
struct Rows32 {
  uint4 v[8];
  __device__ __forceinline__ void load(const void *p, int64_t ld, int rows, int cols, int dtype,
                                       int lane) {
    const bool wide = dtype == MOE_DTYPE_FP32;
    const int r = wide ? lane >> 3 : lane >> 2, c = wide ? (lane & 7) * 4 : (lane & 3) * 8;
    const int step = wide ? 4 : 8;
    const char *q = static_cast<const char *>(p) + ((int64_t)r * ld + c) * (wide ? 4 : 2);
    const int64_t stride = ld * step * (wide ? 4 : 2);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < 4 || wide)
        v[i] = step * i + r < rows && c < cols ? *reinterpret_cast<const uint4 *>(q + i * stride)
                                               : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void add_to(float (&f)[32], uint8_t *slot, int dtype, int lane) const {
    if (dtype == MOE_DTYPE_FP32) {
      const int r = lane >> 3, c = lane & 7;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4 *>(slot + (4 * i + r) * 128 + ((c ^ ((4 * i + r) & 7)) << 4)) = v[i];
      __syncwarp();
      add32(f, slot, lane);
    } else {
      const int r = lane >> 2, c = lane & 3;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(slot + (8 * i + r) * 64 + ((c ^ ((r >> 1) & 3)) << 4)) = v[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 o =
            *reinterpret_cast<const uint4 *>(slot + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4));
        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = unpack16(dtype, w[j]);
          f[8 * i + 2 * j] += u.x;
          f[8 * i + 2 * j + 1] += u.y;
        }
      }
    }
    __syncwarp();
  }
};

}  // namespace moe
