// Matrix products of the dense operators for prefill and training batches, on
// CTA pairs (tcgen05.mma.cta_group::2, sm_103a):
//
//   D[m, n] = epilogue( sum over k of A(m, k) B(n, k) )
//
// Bound: the tensor cores.  A cluster of two CTAs on two SMs computes a tile
// of 256 rows by up to 256 columns: each CTA's shared memory holds 128 rows of
// A and half of the columns' B, one thread of the even CTA issues the MMAs for
// both (M = 256), and each CTA's TMEM receives its own 128 rows of the fp32
// accumulator for all columns: 32 KB of operands per SM for 128 x 256 x 64
// multiply-adds.  Two accumulators of 256 columns let the epilogue of a tile
// run under the next tile's products.
//
// Operands are K-major or MN-major, as they lie in memory: the gradient
// products dX = dY W and dW = dY^T X read the forward tensors without a
// transposed copy.  Tails of M, N and K are zeros filled in by TMA on the way
// in and clipped by TMA on the way out.
//
// CTA = 10 warps, in both CTAs of the pair:
//   warps 0-7  epilogue: 32 accumulator rows by 32 columns at a time, from
//              TMEM through registers to a swizzled slot in shared memory and
//              out by a TMA store of the warp's own (no barrier between warps);
//   warp 8     TMA producer of its CTA's operands (completion counted on the
//              even CTA's `full` barrier);
//   warp 9     TMEM allocation; in the even CTA one thread issues the MMAs.
// Every wait is bounded; on expiry the CTA latches the status bit and leaves
// its loops, and both CTAs meet at a cluster barrier before TMEM is freed.
#include <algorithm>

#include "dense.cuh"
#include "pair_ptx.cuh"

namespace moe {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kStages = 6;
constexpr int kTileM = 256;
constexpr int kTileN = 256;                      // the most columns of a tile
constexpr uint32_t kABytes = kBM * kBK * 2;      // 16 KB
constexpr uint32_t kBBytes = kTileN / 2 * kBK * 2;  // <= 16 KB
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr uint32_t kSlotBytes = 4096;            // an epilogue warp's: 32 x 32 fp32, or two of 16 bits
constexpr uint32_t kTmemCols = 512;
constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * kSlotBytes +
                         (2 * kStages + 5) * 8 + 16;
static_assert(kSmem <= 232448, "shared memory per CTA");
// Row tiles of a raster group: tiles that run together share the A rows of 8
// row tiles and the B rows of ~10 column tiles, ~20 MB at K = 4096: in L2.
constexpr int kGroupM = 8;

struct PairMaps {
  CUtensorMap a, b, d, extra;  // extra: preact, saved or dgu
};

struct PairArgs {
  int M, N, K;
  int bn, cols;  // accumulator columns of a tile; output columns of a tile
  int mt, nt;
  int dtype, out_dtype, act;
  const void *bias, *residual;
  int64_t ldr;
  const float *saved;
  int extra;  // kEpiLinear: store preact; kEpiGated: store saved
  uint32_t *status;
};

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

struct Tile {
  int m0, j;  // first row, column tile
};
__device__ __forceinline__ Tile tile_at(int tile, const PairArgs &a) {
  const int per = kGroupM * a.nt;
  const int g = tile / per, r = tile - g * per;
  const int gm = min(kGroupM, a.mt - g * kGroupM);
  Tile t;
  t.j = r / gm;
  t.m0 = (g * kGroupM + r - t.j * gm) * kTileM;
  return t;
}

// A warp's output buffer: two slots of 32 x 32 16-bit values, or one of fp32.
struct Slots {
  uint8_t *base;
  uint32_t n;
  bool wide;  // the last store was fp32
  // Each waits for the stores that still read what it hands out.
  __device__ __forceinline__ uint8_t *take16(int lane) {
    if (lane == 0) {
      if (wide)
        bulk_wait_read<0>();
      else
        bulk_wait_read<1>();
    }
    wide = false;
    __syncwarp();
    return base + (n++ & 1u) * (kSlotBytes / 2);
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
__device__ __forceinline__ void put32(uint8_t *slot, int lane, const float (&f)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4 *>(slot + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_float4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]);
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

// 32 consecutive values of the output type at `p` + off, of which `left` exist
// (a multiple of 8; the rest zero): loaded early, added later.
struct Values32 {
  uint4 v[8];
  __device__ __forceinline__ void load(const void *p, int64_t off, int left, int dtype) {
    if (dtype == MOE_DTYPE_FP32) {
      const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + off);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = 4 * c < left ? q[c] : make_uint4(0, 0, 0, 0);
    } else {
      const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + off);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = 8 * c < left ? q[c] : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void add_to(float (&f)[32], int dtype) const {
    if (dtype == MOE_DTYPE_FP32) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        f[4 * c] += __uint_as_float(v[c].x);
        f[4 * c + 1] += __uint_as_float(v[c].y);
        f[4 * c + 2] += __uint_as_float(v[c].z);
        f[4 * c + 3] += __uint_as_float(v[c].w);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = unpack16(dtype, w[i]);
          f[8 * c + 2 * i] += u.x;
          f[8 * c + 2 * i + 1] += u.y;
        }
      }
    }
  }
};

// 32 consecutive fp32 values; those past `left` are zero.
__device__ __forceinline__ void read32(float (&f)[32], const float *p, int left) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float4 v = 4 * c < left ? __ldg(reinterpret_cast<const float4 *>(p) + c)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
    f[4 * c] = v.x;
    f[4 * c + 1] = v.y;
    f[4 * c + 2] = v.z;
    f[4 * c + 3] = v.w;
  }
}

template <int kEpi, bool kAMn, bool kBMn>
__global__ void __launch_bounds__(kThreads, 1)
    dense_pair_kernel(const __grid_constant__ PairMaps maps, const PairArgs a) {
  constexpr uint32_t kCode = kStatusTimeoutDense;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *ring = smem;
  uint8_t *slots = ring + kStages * kStageBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(slots + kEpiWarps * kSlotBytes);
  uint64_t *empty = full + kStages;
  uint64_t *tfull = empty + kStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *fin = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);  // of both CTAs
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    tma_prefetch_desc(&maps.d);
  }
  pdl_wait();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = a.mt * a.nt;
  const int nkb = (a.K + kBK - 1) / kBK;
  const int half = a.bn >> 1;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      const int b_boxes = (half + 63) >> 6;
      const uint32_t bytes =
          kABytes + (kBMn ? (uint32_t)b_boxes * 8192u : (uint32_t)half * (kBK * 2));
      uint32_t st = 0, ph = 0, issued = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        const Tile t = tile_at(tile, a);
        const int m = t.m0 + (int)rank * kBM;
        const int n = kEpi == kEpiGated ? t.j * a.cols : t.j * a.cols + (int)rank * half;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[st], ph ^ 1u, abort_flag, a.status, kCode)) {
            ok = false;
            break;
          }
          const uint32_t bar = cluster_addr(&full[st], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * bytes);
          uint8_t *da = ring + st * kStageBytes, *db = da + kABytes;
          const int k = kb * kBK;
          if (kAMn) {
            tma_load_2d_pair(da, &maps.a, bar, m, k);
            tma_load_2d_pair(da + 8192, &maps.a, bar, m + 64, k);
          } else {
            tma_load_2d_pair(da, &maps.a, bar, k, m);
          }
          if (kEpi == kEpiGated) {
            // the even CTA holds the gate columns' rows, the odd CTA the up columns'
            tma_load_3d_pair(db, &maps.b, bar, k, n, (int)rank);
          } else if (kBMn) {
            for (int i = 0; i < b_boxes; ++i)
              tma_load_2d_pair(db + i * 8192, &maps.b, bar, n + 64 * i, k);
          } else {
            tma_load_2d_pair(db, &maps.b, bar, k, n);
          }
          ++issued;
          if (++st == kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      if (rank == 0) {
        // every copy of both CTAs completes on these barriers
        const uint32_t n = issued < kStages ? issued : kStages;
        for (uint32_t i = 0; i < n; ++i) {
          st = st == 0 ? kStages - 1 : st - 1;
          if (st == kStages - 1) ph ^= 1u;
          mbar_wait_drain(&full[st], ph);
        }
      } else if (!ok) {
        // the odd CTA's copies complete on the even CTA's barriers: after an
        // abort give copies in flight time to land before leaving
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------- MMA issuer --
    if (rank == 0 && lane == 0) {
      constexpr uint32_t kAStep = kAMn ? 128 : 2, kBStep = kBMn ? 128 : 2;  // 16 K, in 16 bytes
      const uint32_t idesc = idesc_16(a.dtype, kAMn, kBMn, 2 * kBM, a.bn);
      const uint64_t a0 = kAMn ? sdesc_mn_sw128(smem_u32(ring)) : sdesc_k_sw128(smem_u32(ring));
      const uint64_t b0 = kBMn ? sdesc_mn_sw128(smem_u32(ring + kABytes))
                               : sdesc_k_sw128(smem_u32(ring + kABytes));
      uint32_t st = 0, ph = 0, tl = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl, ++tl) {
        const uint32_t buf = tl & 1u, use = tl >> 1;
        if (!mbar_wait(&tempty[buf], (use & 1u) ^ 1u, abort_flag, a.status, kCode)) break;
        tc_fence_after();
        const uint32_t d0 = tmem_base + buf * (kTmemCols / 2);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&full[st], ph, abort_flag, a.status, kCode)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = a0 + st * (kStageBytes >> 4), bd = b0 + st * (kStageBytes >> 4);
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q)
            umma_bf16_pair(d0, ad + q * kAStep, bd + q * kBStep, idesc, (kb | q) != 0 ? 1u : 0u);
          umma_commit_pair(&empty[st], 3);
          if (++st == kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(&tfull[buf], 3);
      }
      umma_commit_pair(fin, 1);
      mbar_wait_drain(fin, 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue --
    // warps w and w + 4 share 32 TMEM lanes and take every other 32 columns
    Slots slot = {slots + warp * kSlotBytes, 0, false};
    const int quad = warp & 3, turn = (warp >> 2) * 32;
    uint32_t tl = 0;
    for (int tile = cid; tile < total; tile += ncl, ++tl) {
      const Tile t = tile_at(tile, a);
      const uint32_t buf = tl & 1u, use = tl >> 1;
      const bool waited = mbar_wait(&tfull[buf], use & 1u, abort_flag, a.status, kCode);
      if (!__all_sync(0xffffffffu, waited)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(quad * 32) << 16) + buf * (kTmemCols / 2);
      const int row0 = t.m0 + (int)rank * kBM + quad * 32, row = row0 + lane;
      const int c0 = t.j * a.cols;
      const int cend = row0 < a.M ? min(a.N, c0 + a.cols) : c0;
      for (int c = c0 + turn; c < cend; c += 64) {
        const int left = row < a.M ? a.N - c : 0;  // this row's columns from c on
        float v[32];
        if (kEpi == kEpiLinear) {
          Values32 bias, res;
          if (a.bias != nullptr) bias.load(a.bias, c, a.N - c, a.out_dtype);
          if (a.residual != nullptr)
            res.load(a.residual, (int64_t)row * a.ldr + c, left, a.out_dtype);
          tmem_ld32(tb + (c - c0), v);
          if (a.bias != nullptr) bias.add_to(v, a.out_dtype);
          if (a.extra) {
            uint8_t *p = slot.take32(lane);
            put32(p, lane, v);
            send_2d(&maps.extra, p, lane, c, row0);
          }
          activate_all(a.act, v);
          if (a.residual != nullptr) res.add_to(v, a.out_dtype);
          uint8_t *p;
          if (a.out_dtype == MOE_DTYPE_FP32) {
            p = slot.take32(lane);
            put32(p, lane, v);
          } else {
            p = slot.take16(lane);
            put16(p, lane, a.out_dtype, v);
          }
          send_2d(&maps.d, p, lane, c, row0);
        } else if (kEpi == kEpiGated) {
          float u[32];
          tmem_ld32(tb + (c - c0), v);
          tmem_ld32(tb + half + (c - c0), u);
          if (a.extra) {
            uint8_t *p = slot.take32(lane);
            put32(p, lane, v);
            send_3d(&maps.extra, p, lane, c, row0, 0);
            p = slot.take32(lane);
            put32(p, lane, u);
            send_3d(&maps.extra, p, lane, c, row0, 1);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
          uint8_t *p = slot.take16(lane);
          put16(p, lane, a.dtype, v);
          send_2d(&maps.d, p, lane, c, row0);
        } else {
          // dh = acc;  p = sigmoid(g):  h = g p u, dg = dh u p (1 + g (1 - p)), du = dh g p
          float g[32], u[32];
          const float *sv = a.saved + (int64_t)row * 2 * a.N + c;
          read32(g, sv, left);
          read32(u, sv + a.N, left);
          tmem_ld32(tb + (c - c0), v);
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float p = sigmoid(g[i]), gp = g[i] * p;
            o[i] = gp * u[i];
            u[i] = v[i] * u[i] * p * (1.0f + g[i] * (1.0f - p));
            v[i] = v[i] * gp;
          }
          uint8_t *p = slot.take16(lane);
          put16(p, lane, a.dtype, o);
          send_2d(&maps.d, p, lane, c, row0);
          p = slot.take16(lane);
          put16(p, lane, a.dtype, u);
          send_3d(&maps.extra, p, lane, c, row0, 0);
          p = slot.take16(lane);
          put16(p, lane, a.dtype, v);
          send_3d(&maps.extra, p, lane, c, row0, 1);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[buf], 0));
    }
    // the slots outlive the copies that read them
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still signal it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

CUtensorMapSwizzle out_swizzle(int dtype) {
  return dtype == MOE_DTYPE_FP32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
}

template <int kEpi, bool kAMn, bool kBMn>
cudaError_t launch(const DenseGemm &g, cudaStream_t s) {
  auto kern = dense_pair_kernel<kEpi, kAMn, kBMn>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static int clusters[64] = {};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  if (clusters[dev] == 0) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(num_sms() / 2 * 2));
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    clusters[dev] = std::min(n, num_sms() / 2);
  }

  PairArgs a = {};
  a.M = g.M;
  a.N = g.N;
  a.K = g.K;
  a.mt = (g.M + kTileM - 1) / kTileM;
  // Tile width: the one with the least whole rounds x columns over the
  // clusters.
  const int step = kEpi == kEpiGated ? 64 : 32;
  int64_t best = 0;
  for (int bn = kTileN; bn >= 64; bn -= step) {
    const int cols = kEpi == kEpiGated ? bn / 2 : bn;
    const int nt = (g.N + cols - 1) / cols;
    const int64_t rounds = ((int64_t)a.mt * nt + clusters[dev] - 1) / clusters[dev];
    const int64_t cost = rounds * (std::max(bn, 112) + 8);
    if (best == 0 || cost < best) {
      best = cost;
      a.bn = bn;
      a.cols = cols;
      a.nt = nt;
    }
  }
  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.act = g.act;
  a.bias = g.bias;
  a.residual = g.residual;
  a.ldr = g.ldr;
  a.saved = g.saved;
  a.status = g.status;
  const int half = a.bn / 2;

  PairMaps maps;
  const CUtensorMapSwizzle in = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = kAMn ? map_2d(&maps.a, g.dtype, in, g.a, g.K, g.M, g.lda, kBK, 64)
                 : map_2d(&maps.a, g.dtype, in, g.a, g.M, g.K, g.lda, kBM, kBK);
  if (kEpi == kEpiGated)
    ok = ok && map_two(&maps.b, g.dtype, in, g.b, g.N, g.K, g.ldb, g.ldb * g.N, half, kBK, 1);
  else
    ok = ok && (kBMn ? map_2d(&maps.b, g.dtype, in, g.b, g.K, g.N, g.ldb, kBK, 64)
                     : map_2d(&maps.b, g.dtype, in, g.b, g.N, g.K, g.ldb, half, kBK));
  if (kEpi == kEpiLinear) {
    ok = ok && map_2d(&maps.d, g.out_dtype, out_swizzle(g.out_dtype), g.d, g.M, g.N, g.ldd, 32, 32);
    a.extra = g.preact != nullptr;
    maps.extra = maps.d;
    if (a.extra)
      ok = ok && map_2d(&maps.extra, MOE_DTYPE_FP32, out_swizzle(MOE_DTYPE_FP32), g.preact, g.M,
                        g.N, g.N, 32, 32);
  } else if (kEpi == kEpiGated) {
    ok = ok && map_2d(&maps.d, g.dtype, out_swizzle(g.dtype), g.d, g.M, g.N, g.ldd, 32, 32);
    a.extra = g.saved != nullptr;
    maps.extra = maps.d;
    if (a.extra)
      ok = ok && map_two(&maps.extra, MOE_DTYPE_FP32, out_swizzle(MOE_DTYPE_FP32), g.saved, g.M,
                         g.N, 2 * (int64_t)g.N, g.N, 32, 32, 1);
  } else {
    ok = ok && map_2d(&maps.d, g.dtype, out_swizzle(g.dtype), g.h, g.M, g.N, g.N, 32, 32) &&
         map_two(&maps.extra, g.dtype, out_swizzle(g.dtype), g.dgu, g.M, g.N, 2 * (int64_t)g.N,
                 g.N, 32, 32, 1);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int ncl = (int)std::min<int64_t>(clusters[dev], (int64_t)a.mt * a.nt);
  cfg.gridDim = dim3((unsigned)(2 * ncl));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

}  // namespace

cudaError_t launch_dense_pair(const DenseGemm &g, cudaStream_t s) {
  switch (g.epi) {
    case kEpiGated: return launch<kEpiGated, false, false>(g, s);
    case kEpiGatedGrad: return launch<kEpiGatedGrad, false, true>(g, s);
    default:
      if (g.a_mn) return launch<kEpiLinear, true, true>(g, s);
      if (g.b_mn) return launch<kEpiLinear, false, true>(g, s);
      return launch<kEpiLinear, false, false>(g, s);
  }
}

}  // namespace moe
