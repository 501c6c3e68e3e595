// Matrix products of the dense operators for few rows (decoding, short
// chunks): D[t, n] = epilogue( sum over k of X(t, k) W(n, k) ).
//
// Bound: the bytes of W from HBM.  W's rows are the MMA's M (128 a tile), the
// rows of X its N (16 to 256), so a tile of W flows through the tensor core
// once for all rows of X.  There are too few tiles of W to draw the whole
// bandwidth, so K is split over the CTAs of a cluster: each streams its own
// part of K through a ring of TMA stages into its TMEM accumulator, and the
// partial tiles are added in rank order through distributed shared memory --
// one kernel, no partials in HBM, and the same bits every time.
//
// Gated tiles hold 64 gate and the same 64 up rows of W.  E4M3 operands are
// multiplied as they are (kind::mxf8f6f4, block-scaled): the exponent of each
// 128 x 128 block of W and of each row of X and 128 columns goes to TMEM as
// the MMA's scale factors.
//
// CTA = 6 warps: 0-3 write the scale factors (E4M3), then move the accumulator
// to shared memory; 4 TMA producer; 5 TMEM and MMA.  All warps add, apply the
// epilogue and store.  Every wait is bounded.
#include <algorithm>

#include "dense.cuh"
#include "pair_ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 192;
constexpr int kMaxStages = 6;
constexpr uint32_t kWBytes = 128 * 128;  // 128 rows of 128 bytes of K
constexpr int kMaxSplit = 8;             // portable cluster size

struct SmallMaps {
  CUtensorMap w, x;
};

struct SmallArgs {
  int T, N, K;      // rows of X, output columns, depth
  int n;            // rows of X a tile (a multiple of 16)
  int split, stages;
  int dtype, out_dtype, act;
  const void *bias, *residual;
  void *d;
  int64_t ldr, ldd;
  const int8_t *w_scale, *x_scale;
  uint32_t tmem_cols, sf_col;  // allocated; first scale-factor column
  uint32_t *status;
};

// 8 consecutive values of type `dtype`, as fp32
__device__ __forceinline__ void load8(float (&f)[8], const void *p, int64_t off, int dtype) {
  if (dtype == MOE_DTYPE_FP32) {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + off);
    const float4 a = q[0], b = q[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + off);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = unpack16(dtype, w[i]);
      f[2 * i] = u.x;
      f[2 * i + 1] = u.y;
    }
  }
}
__device__ __forceinline__ void store8(const float (&f)[8], void *p, int64_t off, int dtype) {
  if (dtype == MOE_DTYPE_FP32) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + off);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + off) =
        make_uint4(pack16(dtype, f[0], f[1]), pack16(dtype, f[2], f[3]),
                   pack16(dtype, f[4], f[5]), pack16(dtype, f[6], f[7]));
  }
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// f[i] = sum over the cluster's ranks, in rank order, of 8 floats at `p`
__device__ __forceinline__ void cluster_add8(float (&f)[8], const float *p, int split) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.f;
#pragma unroll 4
  for (int r = 0; r < split; ++r) {
    const uint32_t a = cluster_addr(p, (uint32_t)r);
    const float4 lo = ld_cluster4(a), hi = ld_cluster4(a + 16);
    f[0] += lo.x, f[1] += lo.y, f[2] += lo.z, f[3] += lo.w;
    f[4] += hi.x, f[5] += hi.y, f[6] += hi.z, f[7] += hi.w;
  }
}

template <bool kGated, bool kE4m3>
__global__ void __launch_bounds__(kThreads)
    dense_small_kernel(const __grid_constant__ SmallMaps maps, const SmallArgs a) {
  constexpr uint32_t kCode = kStatusTimeoutDense;
  constexpr int kCols = kGated ? 64 : 128;  // output columns of a tile
  constexpr int kKb = kE4m3 ? 128 : 64;     // K elements of a stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sf_full[kMaxStages], tfull;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t stage_bytes = kWBytes + (uint32_t)a.n * 128u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_full[s], 4);
    }
    mbar_init(&tfull, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&tmem_slot, a.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;
  const int tile = blockIdx.x / a.split;
  const int c0 = tile * kCols;              // first output column
  const int t0 = blockIdx.y * a.n;          // first row of X
  const int rows = min(a.n, a.T - t0);
  const int nkb = (a.K + kKb - 1) / kKb;
  const int k0 = (int)((int64_t)nkb * rank / a.split);
  const int k1 = (int)((int64_t)nkb * (rank + 1) / a.split);
  float *part = reinterpret_cast<float *>(ring);  // [n][128] once the ring is done

  if (warp == 4) {
    if (lane == 0) {
      uint32_t st = 0, ph = 0, issued = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(&empty[st], ph ^ 1u, &abort_flag, a.status, kCode)) break;
        mbar_arrive_expect_tx(&full[st], stage_bytes);
        uint8_t *dst = ring + st * stage_bytes;
        if (kGated)
          tma_load_3d(dst, &maps.w, &full[st], kb * kKb, c0, 0);
        else
          tma_load_2d(dst, &maps.w, &full[st], kb * kKb, c0);
        tma_load_2d(dst + kWBytes, &maps.x, &full[st], kb * kKb, t0);
        ++issued;
        if (++st == (uint32_t)a.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
      // every copy lands before the ring is used for the partial sums
      const uint32_t n = issued < (uint32_t)a.stages ? issued : (uint32_t)a.stages;
      for (uint32_t i = 0; i < n; ++i) {
        st = st == 0 ? a.stages - 1 : st - 1;
        if (st == (uint32_t)a.stages - 1) ph ^= 1u;
        mbar_wait_drain(&full[st], ph);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      const uint32_t idesc = kE4m3 ? idesc_mxf8(128, a.n) : idesc_16(a.dtype, false, false, 128, a.n);
      const uint64_t w0 = sdesc_k_sw128(smem_u32(ring));
      uint32_t st = 0, ph = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(&full[st], ph, &abort_flag, a.status, kCode)) break;
        if (kE4m3 && !mbar_wait(&sf_full[st], ph, &abort_flag, a.status, kCode)) break;
        tc_fence_after();
        const uint64_t wd = w0 + st * (stage_bytes >> 4), xd = wd + (kWBytes >> 4);
        const uint32_t sf = tmem + a.sf_col + st * kSmallSfCols;
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
          const uint32_t acc = (kb != k0 || q != 0) ? 1u : 0u;
          if (kE4m3)
            umma_mxf8(tmem, wd + 2 * q, xd + 2 * q, idesc, sf, sf + 4, acc);
          else
            umma_bf16(tmem, wd + 2 * q, xd + 2 * q, idesc, acc);
        }
        umma_commit(&empty[st]);
        if (++st == (uint32_t)a.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
      umma_commit(&tfull);
    }
    __syncwarp();
  } else {
    bool ok = true;
    if (kE4m3) {
      // Scale factors of stage kb, the same in each warp's 32 lanes: column j
      // of the first 4 holds W rows 32 j + lane, of the next 8 X rows 32 j +
      // lane; the word's four bytes are the four 32-deep parts of the 128.
      const int nb = nkb;
      const int8_t *ws = a.w_scale + (int64_t)(c0 / 128) * nb;
      uint32_t st = 0, ph = 0;
      for (int kb = k0; kb < k1 && ok; ++kb) {
        const uint32_t w = e8m0x4(ws[kb]);
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = 32 * j + lane;
          x[j] = t < rows ? e8m0x4(a.x_scale[(int64_t)(t0 + t) * nb + kb]) : 0x7f7f7f7fu;
        }
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&empty[st], ph ^ 1u, &abort_flag, a.status, kCode));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + a.sf_col + st * kSmallSfCols;
        const uint32_t w4[4] = {w, w, w, w};
        tmem_st4(at, w4);
        tmem_st8(at + 4, x);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[st]);
        if (++st == (uint32_t)a.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    ok = mbar_wait(&tfull, 0, &abort_flag, a.status, kCode) && ok;
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(warp * 32) << 16);
      float *p = part + warp * 32 + lane;
      for (int q = 0; q < a.n; q += 16) {
        float v[16];
        tmem_ld16f(tb + q, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) p[(q + i) * 128] = v[i];
      }
    }
    tc_fence_before();
  }
  cluster_sync_all();  // partial tiles of every rank in place
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, a.tmem_cols);

  if (!abort_flag) {
    constexpr int kGroups = kCols / 8;
    const int units = rows * kGroups;
    for (int u = (int)threadIdx.x * a.split + (int)rank; u < units; u += kThreads * a.split) {
      const int t = u / kGroups, g = u - t * kGroups, c = c0 + g * 8;
      if (c >= a.N) continue;
      const int64_t row = t0 + t;
      float f[8], r[8], b[8];
      if (!kGated && a.bias != nullptr) load8(b, a.bias, c, a.out_dtype);
      if (a.residual != nullptr) load8(r, a.residual, row * a.ldr + c, a.out_dtype);
      cluster_add8(f, part + t * 128 + g * 8, a.split);
      if (kGated) {
        float up[8];
        cluster_add8(up, part + t * 128 + 64 + g * 8, a.split);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * sigmoid(f[i]) * up[i];
      } else {
        if (a.bias != nullptr)
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += b[i];
        activate_all(a.act, f);
      }
      if (a.residual != nullptr)
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += r[i];
      store8(f, a.d, row * a.ldd + c, a.out_dtype);
    }
  }
  cluster_sync_all();  // no CTA's shared memory goes while a peer reads it
}

template <bool kGated, bool kE4m3>
cudaError_t launch(const DenseGemm &g, cudaStream_t s) {
  auto kern = dense_small_kernel<kGated, kE4m3>;
  constexpr int kCols = kGated ? 64 : 128, kKb = kE4m3 ? 128 : 64;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;

  SmallArgs a = {};
  a.T = g.M;
  a.N = g.N;
  a.K = g.K;
  const int chunks = (g.M + kSmallRows - 1) / kSmallRows;
  a.n = ((g.M + chunks - 1) / chunks + 15) / 16 * 16;
  const uint32_t stage = kWBytes + (uint32_t)a.n * 128u;
  // Two CTAs share an SM while a ring of at least four stages fits in half of
  // its shared memory (n <= 64): one streams while the other adds and stores.
  const int per_sm = a.n <= 64 ? 2 : 1;
  const uint32_t room = per_sm == 2 ? 110u * 1024u : 220u * 1024u;
  a.stages = std::min<int>(kMaxStages, (int)(room / stage));
  const size_t smem = 1024 + (size_t)a.stages * stage;
  uint32_t cols = (uint32_t)a.n;
  a.sf_col = cols;
  if (kE4m3) cols += (uint32_t)a.stages * kSmallSfCols;
  a.tmem_cols = 32;
  while (a.tmem_cols < cols) a.tmem_cols *= 2;

  // As many parts of K as keep every CTA resident at once.
  const int tiles = (g.N + kCols - 1) / kCols * chunks;
  const int nkb = (g.K + kKb - 1) / kKb;
  a.split = 1;
  while (a.split < kMaxSplit && tiles * a.split * 2 <= num_sms() * per_sm && a.split * 2 <= nkb)
    a.split *= 2;

  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.act = g.act;
  a.bias = g.bias;
  a.residual = g.residual;
  a.d = g.d;
  a.ldr = g.ldr;
  a.ldd = g.ldd;
  a.w_scale = g.b_scale;
  a.x_scale = g.a_scale;
  a.status = g.status;

  SmallMaps maps;
  const bool ok =
      (kGated ? map_two(&maps.w, g.dtype, CU_TENSOR_MAP_SWIZZLE_128B, g.b, g.N, g.K, g.ldb,
                        g.ldb * g.N, 64, kKb, 2)
              : map_2d(&maps.w, g.dtype, CU_TENSOR_MAP_SWIZZLE_128B, g.b, g.N, g.K, g.ldb, 128, kKb)) &&
      map_2d(&maps.x, g.dtype, CU_TENSOR_MAP_SWIZZLE_128B, g.a, g.M, g.K, g.lda, a.n, kKb);
  if (!ok) return cudaErrorInvalidValue;

  static size_t configured[64] = {};
  if (smem > configured[dev]) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    configured[dev] = smem;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(tiles / chunks * a.split), (unsigned)chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

}  // namespace

cudaError_t launch_dense_small(const DenseGemm &g, cudaStream_t s) {
  if (g.dtype == MOE_DTYPE_E4M3) return launch<false, true>(g, s);
  return g.epi == kEpiGated ? launch<true, false>(g, s) : launch<false, false>(g, s);
}

}  // namespace moe
