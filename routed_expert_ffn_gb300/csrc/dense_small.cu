// Matrix products of the dense operators for few rows (decoding, short
// chunks): D[t, n] = epilogue( sum over k of X(t, k) W(n, k) ).
//
// Bound: the bytes of W from HBM.  W's rows are the MMA's M (128 a tile), the
// rows of X its N (16 to 64), so a tile of W flows through the tensor core
// once for up to 64 rows of X; each further 64 read it again, from L2 (the caller's
// estimates send batches of up to 1024 rows here where few columns leave the other
// kernel's tiles too few).  There are too few tiles of W to draw the whole
// bandwidth, so K is split over the CTAs of a cluster: each streams its own
// part of K through a ring of TMA stages into its TMEM accumulator, and the
// partial tiles are sent through distributed shared memory to the CTA that adds
// them (each takes some of the rows of X), in rank order -- one kernel, no
// partials in HBM, and the same bits every time.
//
// Gated tiles hold 64 gate and the same 64 up rows of W.  A gradient's W (dX =
// dY W) is read as it lies, MN-major.  E4M3 operands are
// multiplied as they are (kind::mxf8f6f4, block-scaled): the exponent of each
// 128 x 128 block of W and of each row of X and 128 columns goes to TMEM as
// the MMA's scale factors.
//
// CTA = 6 warps: 0-3 write the scale factors (E4M3), then send the accumulator's
// rows; 4 TMA producer; 5 TMEM and MMA.  All warps add, apply the
// epilogue and store.  Every wait is bounded.
#include <algorithm>

#include "dense.cuh"
#include "pair_ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 192;
constexpr int kTmaWarp = 4, kMmaWarp = 5;
constexpr int kMaxStages = 6;
constexpr uint32_t kSmallSfCols = 8;     // scale-factor columns of a stage
constexpr uint32_t kWBytes = 128 * 128;  // 128 rows of 128 bytes of K
constexpr int kChunk = 64;               // the most rows of X a tile
constexpr int kMaxSplit = 8;             // portable cluster size
constexpr uint32_t kRingRoom = 102u * 1024u;  // of a CTA: two to an SM
// and behind the ring up to 16 rows' partial tiles (more rows' fit in its place)
constexpr size_t kMostSmem = 1024 + kRingRoom + 16 * 512;
static_assert(2 * kChunk * 512 <= kRingRoom, "partial tiles in the ring's place");

struct SmallMaps {
  CUtensorMap w, x;
};

struct SmallArgs {
  int T, N, K;      // rows of X, output columns, depth
  int n;            // rows of X a tile (a multiple of 16)
  int split, stages;
  int own;          // rows of X whose sums a CTA of the cluster adds
  int bulk;         // how partial tiles travel: 0 single stores, 1 bulk copies
  uint32_t part_off;  // where they arrive in shared memory
  int dtype, out_dtype, act;
  const void *bias, *residual;
  void *d;
  int64_t ldr, ldd;
  const int8_t *w_scale, *x_scale;
  uint32_t tmem_cols, sf_col;  // allocated; first scale-factor column
  uint32_t *status;
};

// 8 consecutive values of type `dtype`, loaded early and converted late
struct Values8 {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void *p, int64_t off, int dtype) {
    if (dtype == MOE_DTYPE_FP32) {
      const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + off);
      lo = q[0];
      hi = q[1];
    } else {
      lo = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + off);
    }
  }
  __device__ __forceinline__ void add_to(float (&f)[8], int dtype) const {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (dtype == MOE_DTYPE_FP32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = unpack16(dtype, w[i]);
        f[2 * i] += u.x;
        f[2 * i + 1] += u.y;
      }
    }
  }
};
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
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// f[i] = sum over the ranks, in rank order, of 8 floats of their partial tiles
__device__ __forceinline__ void add_parts(float (&f)[8], const float *p, int split, int stride) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.f;
  for (int r = 0; r < split; ++r, p += stride) {
    const float4 lo = reinterpret_cast<const float4 *>(p)[0];
    const float4 hi = reinterpret_cast<const float4 *>(p)[1];
    f[0] += lo.x, f[1] += lo.y, f[2] += lo.z, f[3] += lo.w;
    f[4] += hi.x, f[5] += hi.y, f[6] += hi.z, f[7] += hi.w;
  }
}

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *m, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(m), "r"(c0),
               "r"(c1)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *m, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(m),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// W's tile of a stage: kGated 64 gate and 64 up rows; kMn 128 columns of the
// MN-major W (a gradient's) in two boxes of 64.
template <bool kGated, bool kMn>
__device__ __forceinline__ void load_w(void *dst, const CUtensorMap *m, uint64_t *bar, int k, int c0) {
  if (kGated) {
    tma_load_3d(dst, m, bar, k, c0, 0);
  } else if (kMn) {
    tma_load_2d(dst, m, bar, c0, k);
    tma_load_2d(static_cast<uint8_t *>(dst) + kWBytes / 2, m, bar, c0 + 64, k);
  } else {
    tma_load_2d(dst, m, bar, k, c0);
  }
}

template <bool kGated, bool kE4m3, bool kMn>
__global__ void __launch_bounds__(kThreads)
    dense_small_kernel(const __grid_constant__ SmallMaps maps, const SmallArgs a) {
  constexpr int kCols = kGated ? 64 : 128;  // output columns of a tile
  constexpr int kKb = kE4m3 ? 128 : 64;     // K elements of a stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sf_full[kMaxStages], tfull, recv;
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
    mbar_init(&recv, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, a.tmem_cols);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x);
  }
  const int tile = blockIdx.x / a.split;
  const int c0 = tile * kCols;              // first output column
  const int t0 = blockIdx.y * a.n;          // first row of X
  const int rows = min(a.n, a.T - t0);
  const int nkb = (a.K + kKb - 1) / kKb;
  const int k0 = (int)((int64_t)nkb * rank / a.split);
  const int k1 = (int)((int64_t)nkb * (rank + 1) / a.split);
  // [rank][own][128]: every rank's partial tile of this CTA's rows
  float *part = reinterpret_cast<float *>(ring + a.part_off);
  // Until the kernel before this one is done nothing may be read, but W's first
  // stages may come to L2: whatever is still written to them goes there too.
  // (One ring of them: 4096 x 4096 at one row 9.0 -> 8.3 us; all of W measured
  // slower, 14336 x 4096 21 -> 26 us.)
  if (warp == kTmaWarp && lane == 0)
    for (int kb = k0; kb < min(k1, k0 + a.stages); ++kb) {
      if (kGated) {
        tma_prefetch_3d(&maps.w, kb * kKb, c0, 0);
      } else if (kMn) {
        tma_prefetch_2d(&maps.w, c0, kb * kKb);
        tma_prefetch_2d(&maps.w, c0 + 64, kb * kKb);
      } else {
        tma_prefetch_2d(&maps.w, kb * kKb, c0);
      }
    }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;
  // this CTA runs, so its shared memory may be written (nothing to release yet)
  if (!a.bulk) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // This CTA's rows of X, 8 columns a thread.
  constexpr int kGroups = kCols / 8;
  const int first = (int)rank * a.own;
  const int units = max(0, min(a.own, rows - first)) * kGroups;
  const int stride = a.own * 128;
  const bool alone = a.split == 1;
  if (a.bulk && !alone && threadIdx.x == 0)
    mbar_arrive_expect_tx(&recv, (uint32_t)(a.split * (units / kGroups)) * 512u);
  Values8 r = {}, b = {};
  auto fetch = [&](int u) {
    const int t = u / kGroups, c = c0 + (u - t * kGroups) * 8;
    if (u >= units || c >= a.N) return;
    if (!kGated && a.bias != nullptr) b.load(a.bias, c, a.out_dtype);
    if (a.residual != nullptr)
      r.load(a.residual, (int64_t)(t0 + first + t) * a.ldr + c, a.out_dtype);
  };
  fetch(threadIdx.x);  // the first long before it is needed

  if (warp == kTmaWarp) {
    {
      uint32_t st = 0, ph = 0, issued = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait_warp(&empty[st], ph ^ 1u, &abort_flag, a.status, kStatusTimeoutDense)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[st], stage_bytes);
          uint8_t *dst = ring + st * stage_bytes;
          load_w<kGated, kMn>(dst, &maps.w, &full[st], kb * kKb, c0);
          tma_load_2d(dst + kWBytes, &maps.x, &full[st], kb * kKb, t0);
        }
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
  } else if (warp == kMmaWarp) {
    {
      const uint32_t idesc = kE4m3 ? idesc_mxf8(128, a.n) : idesc_16(a.dtype, kMn, false, 128, a.n);
      const uint64_t x0 = sdesc_k_sw128(smem_u32(ring + kWBytes));
      const uint64_t w0 = kMn ? sdesc_mn_sw128(smem_u32(ring)) : sdesc_k_sw128(smem_u32(ring));
      constexpr uint32_t kWStep = kMn ? 128 : 2;  // 16 of K, in 16 bytes
      uint32_t st = 0, ph = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait_warp(&full[st], ph, &abort_flag, a.status, kStatusTimeoutDense)) break;
        if (kE4m3 &&
            !mbar_wait_warp(&sf_full[st], ph, &abort_flag, a.status, kStatusTimeoutDense))
          break;
        tc_fence_after();
        const uint64_t wd = w0 + st * (stage_bytes >> 4), xd = x0 + st * (stage_bytes >> 4);
        const uint32_t sf = tmem + a.sf_col + st * kSmallSfCols;
        if (elect_one()) {
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) {
            const uint32_t acc = (kb != k0 || q != 0) ? 1u : 0u;
            if (kE4m3)
              umma_mxf8(tmem, wd + 2 * q, xd + 2 * q, idesc, sf, sf + 4, acc);
            else
              umma_bf16(tmem, wd + kWStep * q, xd + 2 * q, idesc, acc);
          }
          umma_commit(&empty[st]);
        }
        if (++st == (uint32_t)a.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (elect_one()) umma_commit(&tfull);
    }
    __syncwarp();
  } else {
    bool ok = true;
    if (kE4m3) {
      // Scale factors of stage kb, the same in each warp's 32 lanes: column j
      // of the first 4 holds W rows 32 j + lane, of the next 4 X rows 32 j +
      // lane; the word's four bytes are the four 32-deep parts of the 128.
      const int nb = nkb;
      const int8_t *ws = a.w_scale + (int64_t)(c0 / 128) * nb;
      uint32_t st = 0, ph = 0;
      for (int kb = k0; kb < k1 && ok; ++kb) {
        const uint32_t w = e8m0x4(ws[kb]);
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 32 * j + lane;
          x[j] = t < rows ? e8m0x4(a.x_scale[(int64_t)(t0 + t) * nb + kb]) : 0x7f7f7f7fu;
        }
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&empty[st], ph ^ 1u, &abort_flag, a.status, kStatusTimeoutDense));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + a.sf_col + st * kSmallSfCols;
        const uint32_t w4[4] = {w, w, w, w};
        tmem_st4(at, w4);
        tmem_st4(at + 4, x);
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
    ok = mbar_wait(&tfull, 0, &abort_flag, a.status, kStatusTimeoutDense) && ok;
    ok = __all_sync(0xffffffffu, ok);
    const uint32_t tb = tmem + ((uint32_t)(warp * 32) << 16);
    if (a.bulk) {
      // the ring's place: this CTA's partial tile [row of X][row of W], then
      // what it receives
      cluster_arrive();  // this CTA's ring is done
      if (ok) {
        tc_fence_after();
        float *p = reinterpret_cast<float *>(ring) + warp * 32 + lane;
        for (int q = 0; q < rows; q += 16) {
          float v[16];
          tmem_ld16f(tb + q, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) p[(q + i) * 128] = v[i];
        }
      }
      fence_proxy_async_shared();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      cluster_wait();  // every ring is done
      const int to = (int)threadIdx.x;
      if (ok && !alone && to < a.split) {
        const int n = min(a.own, rows - to * a.own);
        if (n > 0)
          bulk_send(cluster_addr(part + (int)rank * stride, (uint32_t)to),
                    ring + (uint32_t)(to * a.own) * 512u, (uint32_t)n * 512u,
                    cluster_addr(&recv, (uint32_t)to));
      }
    } else {
      cluster_wait();  // every CTA runs
      if (ok) {
        // each row of X goes to the CTA that adds it: 128 bytes a warp and row
        tc_fence_after();
        const float *p = part + (int)rank * stride + warp * 32 + lane;
        float v[16];
        tmem_ld16f(tb, v);
        int to = 0, t = 0;  // rank, its row
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i < rows) st_cluster(cluster_addr(p + t * 128, (uint32_t)to), v[i]);
          if (++t == a.own) {
            t = 0;
            ++to;
          }
        }
      }
    }
    tc_fence_before();
    __syncwarp();
  }
  if (warp >= kTmaWarp) {
    if (a.bulk) cluster_arrive();
    cluster_wait();
  }
  // every rank's partial tile is here
  if (a.bulk) {
    const bool got = alone || units == 0 || mbar_wait(&recv, 0, &abort_flag, a.status, kStatusTimeoutDense);
    tc_fence_before();
    __syncthreads();  // and TMEM has been read
    tc_fence_after();
    if (!got) abort_flag = 1;
    cluster_arrive();  // received: the others' copies no longer read their shared memory
  } else {
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem, a.tmem_cols);
  const int todo = abort_flag ? 0 : units;
  for (int u = (int)threadIdx.x; u < todo; u += kThreads) {
    const int t = u / kGroups, g = u - t * kGroups, c = c0 + g * 8;
    if (c < a.N) {
      float f[8];
      add_parts(f, part + t * 128 + g * 8, a.split, stride);
      if (kGated) {
        float up[8];
        add_parts(up, part + t * 128 + 64 + g * 8, a.split, stride);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * sigmoid(f[i]) * up[i];
      } else {
        if (a.bias != nullptr) b.add_to(f, a.out_dtype);
        if (a.out_dtype == MOE_DTYPE_FP32)
          activate_all<true>(a.act, f);
        else
          activate_all<false>(a.act, f);
      }
      if (a.residual != nullptr) r.add_to(f, a.out_dtype);
      store8(f, a.d, (int64_t)(t0 + first + t) * a.ldd + c, a.out_dtype);
    }
    fetch(u + kThreads);
  }
  __syncwarp();
  if (a.bulk) cluster_wait();  // this CTA's copies have been received
}

// Rows of X a tile, tiles, parts of K and about how long it takes (us).
struct SmallPlan {
  int n, chunks, split;
  float us;
};

// The split with the least estimated time, fitted as plan_pair's: a stage takes
// 0.2 us and 0.0014 for each row of X (E4M3: 0.27 and 0.0005; where SMs hold two
// CTAs 1.4 and 1.25 times that), a launch 3.2 us and 0.05 for each row (two CTAs:
// 0.07).  4096 x 4096 at 64 rows: 26.2 us unsplit, 12.0 split by eight.  A split
// that does not fit in one round loses (192 rows: 26 us split by four, 19 by
// two).  Tiles of 128 rows measured no faster.
SmallPlan plan_small(const DenseGemm &g) {
  const bool e4m3 = g.dtype == MOE_DTYPE_E4M3;
  const int cols = g.epi == kEpiGated ? 64 : 128, kb = e4m3 ? 128 : 64;
  const int nkb = (g.K + kb - 1) / kb;
  SmallPlan p = {};
  p.chunks = (g.M + kChunk - 1) / kChunk;
  p.n = ((g.M + p.chunks - 1) / p.chunks + 15) / 16 * 16;
  const int64_t tiles = (int64_t)((g.N + cols - 1) / cols) * p.chunks;
  const float rows = (float)p.n;
  const float stage = e4m3 ? 0.27f + 0.0005f * rows : 0.2f + 0.0014f * rows;
  const float hbm = weight_us(g);
  for (int split = 1; split == 1 || (split <= kMaxSplit && 2 * split <= nkb); split *= 2) {
    const int64_t ctas = tiles * split, slots = 2 * num_sms();
    if (split > 1 && ctas > slots) break;
    const int64_t rounds = (ctas + slots - 1) / slots;
    const float stages = (float)(rounds * ((nkb + split - 1) / split));
    const bool two = ctas > num_sms();
    const float us = 3.2f + (two ? 0.07f : 0.05f) * rows +
                     stages * stage * (!two ? 1.0f : e4m3 ? 1.25f : 1.4f) + 0.5f * hbm;
    if (p.us == 0.f || us <= p.us) {
      p.us = us;
      p.split = split;
    }
  }
  return p;
}

template <bool kGated, bool kE4m3, bool kMn>
cudaError_t launch(const DenseGemm &g, cudaStream_t s) {
  auto kern = dense_small_kernel<kGated, kE4m3, kMn>;
  constexpr int kCols = kGated ? 64 : 128, kKb = kE4m3 ? 128 : 64;
  const SmallPlan plan = plan_small(g);

  SmallArgs a = {};
  a.T = g.M;
  a.N = g.N;
  a.K = g.K;
  a.n = plan.n;
  a.split = plan.split;
  const uint32_t stage = kWBytes + (uint32_t)a.n * 128u;
  // Two CTAs share an SM: one streams while the other adds and stores.
  a.stages = std::min<int>(kMaxStages, (int)(kRingRoom / stage));
  uint32_t cols = (uint32_t)a.n;
  a.sf_col = cols;
  if (kE4m3) cols += (uint32_t)a.stages * kSmallSfCols;
  a.tmem_cols = 32;
  while (a.tmem_cols < cols) a.tmem_cols *= 2;

  // Up to 16 rows: single stores to a place behind the ring (8 KB), as soon as
  // a CTA is done.  More: bulk copies, out of and into the ring's place, after
  // every CTA of the cluster is done (single stores took 4 us at 64 rows).
  a.own = (a.n + a.split - 1) / a.split;
  a.bulk = a.n > 16;
  const uint32_t ring_bytes = (uint32_t)a.stages * stage;
  const uint32_t part_bytes = (uint32_t)(a.split * a.own) * 512u;
  a.part_off = !a.bulk ? ring_bytes : (a.split == 1 ? 0u : (uint32_t)a.n * 512u);
  const size_t smem = 1024 + std::max(ring_bytes, a.part_off + part_bytes);

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
       : kMn  ? map_2d(&maps.w, g.dtype, CU_TENSOR_MAP_SWIZZLE_128B, g.b, g.K, g.N, g.ldb, kKb, 64)
              : map_2d(&maps.w, g.dtype, CU_TENSOR_MAP_SWIZZLE_128B, g.b, g.N, g.K, g.ldb, 128, kKb)) &&
      map_2d(&maps.x, g.dtype, CU_TENSOR_MAP_SWIZZLE_128B, g.a, g.M, g.K, g.lda, a.n, kKb);
  if (!ok) return cudaErrorInvalidValue;

  if (smem > kMostSmem) return cudaErrorInvalidValue;
  static std::atomic<bool> allowed[64];
  const cudaError_t e = allow_smem(kern, kMostSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((g.N + kCols - 1) / kCols * a.split), (unsigned)plan.chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

}  // namespace

DensePlan dense_small_plan(const DenseGemm &g) {
  const SmallPlan p = plan_small(g);
  return {p.n, g.epi == kEpiGated ? 64 : 128, p.split, p.us};
}

cudaError_t launch_dense_small(const DenseGemm &g, cudaStream_t s) {
  if (g.dtype == MOE_DTYPE_E4M3) return launch<false, true, false>(g, s);
  if (g.epi == kEpiGated) return launch<true, false, false>(g, s);
  return g.b_mn ? launch<false, false, true>(g, s) : launch<false, false, false>(g, s);
}

}  // namespace moe
