// Matrix products grouped by expert, on CTA pairs (tcgen05.mma.cta_group::2, sm_103a).
// Expert e owns rows [offsets[e], offsets[e+1]) and matrix W_e [N][K]:
//
//   kForward     y[p, n]     = sum over k of x[p, k] W_e[n, k]
//   kRowGrad     dx[p, k]    = sum over n of dy[p, n] W_e[n, k]
//   kWeightGrad  dW_e[n, k]  = sum over e's rows p of dy[p, n] x[p, k]
//
// The row counts are ragged, known on the device alone: every CTA reads the offsets
// and works out the tiles for itself.
//
// Rows products: the matrix is the MMA's M (tiles of 256 of its rows or columns, 128 in
// each CTA's shared memory), the expert's rows its N (32 to 256, split evenly over the
// expert's row tiles): an expert of few rows costs few, and its matrix streams at the
// rate of HBM all the same.  Rows past an expert's end are the next one's; their
// columns of the accumulator are not stored.  Of the tiles that do not fill a round of
// the clusters, the K stages are dealt out evenly: a cluster takes at most the end of
// one and the start of the next; pieces leave fp32 partial sums, and the last to
// finish adds them in the order of K, whichever it is.
//
// Weight gradient: dy's columns are the MMA's M, x's columns its N, and the depth runs
// over the expert's rows.  Both operands are MN-major as they lie in memory, and
// the last stage must not see the next expert's rows (nor what lies behind the last):
// each expert has tensor maps of its own that end with its rows, made on the device
// from one template (tensormap.replace), so TMA fills in zeros.
//
// Measured: eight experts of 4096 x 1536 with a row each 21.4 us (100 MB, 4.7 TB/s with
// launch and first copies); 8192 rows over 32 experts of 4096 x 7168 355 to 375 us (5.5 to 5.8
// TB/s); over 8 experts of 14336 x 4096 dx 590 and dW 623 us (1.63 and 1.54 PFLOP/s).
//
// CTA = 10 warps in both CTAs of the pair, as in dense_pair.cu: warps 0-7 epilogue,
// warp 8 TMA, warp 9 TMEM allocation and, in the even CTA, the MMAs.  Every wait is
// bounded; on expiry the CTA latches the status bit and leaves its loops.
#include <algorithm>
#include <type_traits>

#include "grouped.cuh"
#include "pair_tile.cuh"

namespace moe {

namespace {

enum { kForward = 0, kRowGrad = 1, kWeightGrad = 2 };

constexpr int kEpiWarps = 8;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
// kFine: its epilogue's threads hold 128 sums and 32 on their way, with registers that the
// other four warps (two of them idle) leave them: 2 x 208 + 88 = 3 x 168, what each of
// the three groups of 128 threads starts with.
template <bool kFine>
constexpr int kThreads = (kEpiWarps + (kFine ? 4 : 2)) * 32;
constexpr int kFineEpiRegs = 208, kFineOtherRegs = 88;
static_assert(2 * kFineEpiRegs + kFineOtherRegs <= 3 * 168, "more would be waited for without end");
constexpr int kTileM = 256;
constexpr int kTileN = 256;  // the most accumulator columns
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr uint32_t kStageBytes = kABytes + kTileN / 2 * kBK * 2;
// The weight gradient's results leave by way of shared memory, 4 KB for each epilogue
// warp, and one stage less fits.
template <int kMode>
struct Shape {
  static constexpr int stages = kMode == kWeightGrad ? 5 : 6;
  static constexpr uint32_t out_bytes = kMode == kWeightGrad ? 4096 : 0;
};
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxClusters = 80;  // (a GB300 has 76 pairs of SMs)
constexpr int kChunks = kTileN / 64;  // of 32 accumulator columns, to an epilogue warp
// The tensor cores' additions truncate, each by up to a step of the running sum, which adds
// up: 2.4e-6 of the result over 2048 products, 8 times what fp32 rounding leaves.  For fp32
// results (kFine) an accumulator takes 512 of depth and the epilogue's warps add them,
// rounding to nearest.
constexpr int kFineStages = 8;
// Pieces of a split tile: at most this many, of at least this many stages.
constexpr int kMaxParts = 8, kMinPart = 4;

template <int kMode>
constexpr size_t smem_bytes(int E) {
  typedef Shape<kMode> S;
  return 1024 + (size_t)S::stages * kStageBytes + kEpiWarps * S::out_bytes + (2 * S::stages + 5) * 8 +
         24 + (size_t)2 * (E + 1) * 4;
}
static_assert(smem_bytes<kForward>(kMaxE) <= 232448 && smem_bytes<kWeightGrad>(kMaxE) <= 232448,
              "shared memory per CTA");

struct GroupedMaps {
  CUtensorMap a;     // rows products: the matrices
  CUtensorMap b[8];  // rows products: boxes of 16, 32, ..., 128 rows
  CUtensorMap d;     // weight gradient
};

struct GroupedArgs {
  const int32_t *offsets;
  int R, E;
  int M;      // extent of the MMA's M over all tiles: columns of y or dx, N of dW
  int N;      // weight gradient: K of dW
  int nkb;    // rows products: stages of depth
  int mt, nt; // tiles of M; weight gradient: tiles of N
  int bn;     // weight gradient: accumulator columns
  int dtype, out_dtype;
  void *d;
  int64_t ldd;  // rows products
  int accumulate;
  const CUtensorMap *maps;
  float *part;       // places of part_cols x 256 fp32
  int part_chunks;   // part_cols / 32
  uint32_t *counters, *status;
};

typedef RowSchedule<kTileN, 32, kTileM, kMaxParts, kMinPart> RowTiles;

// The weight gradient's tiles: whole ones, in turn.
struct WeightTiles {
  const int32_t *seg, *first;
  int E, mt, nt, bn, N, nkb;
  int total, cid, ncl;
  static constexpr int pieces = 0;

  __device__ __forceinline__ void start() { total = first[E]; }
  __device__ __forceinline__ bool at(int i, Work *w) const {
    const int tile = i * ncl + cid;
    if (tile >= total) return false;
    const int e = expert_of(first, E, tile);
    const int at = tile - first[e], m = at / nt, n = at - m * nt;
    w->e = e;
    w->tile = tile;
    w->part = 0;
    w->parts = 1;
    w->a0 = m * kTileM;
    w->b0 = n * bn;
    w->n = min(bn, N - w->b0);
    w->k0 = 0;
    w->k1 = (seg[e + 1] - seg[e] + kBK - 1) / kBK;
    return true;
  }
};

__device__ __forceinline__ void fence_map_acquire(const CUtensorMap *m) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(m) : "memory");
}

// `and` over the epilogue's 256 threads.
__device__ __forceinline__ bool epi_all(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.and.pred b, 1, 256, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

// One block of 32 rows by 32 columns (lanes) of y or dx.
__device__ __forceinline__ void store_rows(void *d, int64_t ld, int dtype, int64_t row, int rows,
                                           int col, const float (&v)[32]) {
  if (dtype == MOE_DTYPE_FP32) {
    float *p = static_cast<float *>(d) + row * ld + col;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < rows) p[j * ld] = v[j];
  } else {
    uint16_t *p = static_cast<uint16_t *>(d) + row * ld + col;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t w = pack16(dtype, v[j], v[j + 1]);
      if (j < rows) p[j * ld] = (uint16_t)w;
      if (j + 1 < rows) p[(j + 1) * ld] = (uint16_t)(w >> 16);
    }
  }
}

template <int kMode, bool kFine>
__global__ void __launch_bounds__(kThreads<kFine>, 1)
    grouped_pair_kernel(const __grid_constant__ GroupedMaps maps,
                        const __grid_constant__ GroupedArgs a) {
  constexpr bool kWeights = kMode == kWeightGrad;
  constexpr bool kAMn = kMode != kForward, kBMn = kWeights;
  constexpr int kStages = Shape<kMode>::stages;
  constexpr uint32_t kOutBytes = Shape<kMode>::out_bytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *ring = smem;
  uint8_t *slots = ring + kStages * kStageBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(slots + kEpiWarps * kOutBytes);
  uint64_t *empty = full + kStages;
  uint64_t *tfull = empty + kStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *fin = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *last_flag = abort_flag + 1;
  int32_t *seg = reinterpret_cast<int32_t *>(tmem_slot + 4);
  int32_t *first = seg + a.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();  // the even CTA issues the MMAs
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
    if (kWeights)
      tma_prefetch_desc(&maps.d);
    else
      tma_prefetch_desc(&maps.a);
  }
  pdl_wait();
  pdl_launch_dependents();
  make_tables(a.offsets, a.E, a.R, 0, a.R, seg, first, a.status, [&](int m) {
    if (kWeights) return m > 0 || !a.accumulate ? a.mt * a.nt : 0;
    return RowTiles::row_tiles(m) * a.mt;
  });
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  typename std::conditional<kWeights, WeightTiles, RowTiles>::type sch;
  sch.seg = seg;
  sch.first = first;
  sch.E = a.E;
  sch.mt = a.mt;
  sch.nkb = a.nkb;
  if constexpr (kWeights) {
    sch.nt = a.nt;
    sch.bn = a.bn;
    sch.N = a.N;
  }
  sch.cid = blockIdx.x >> 1;
  sch.ncl = gridDim.x >> 1;
  sch.start();
  // accumulator columns of a tile, and those whose B a CTA holds
  auto columns = [&](const Work &w) { return kWeights ? a.bn : (w.n + 31) & ~31; };

  if (kFine && warp >= kEpiWarps) fewer_registers<kFineOtherRegs>();
  if (kFine && warp > kMmaWarp) {
    // (no work of its own)
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------------ TMA producer --
    const uint32_t full0 = cluster_addr(full, 0);
    uint32_t st = 0, ph = 0, issued = 0;
    bool ok = true;
    Work w;
    int known = -1;  // the expert whose maps this warp has acquired
    for (int i = 0; ok && sch.at(i, &w); ++i) {
      if (w.k1 <= w.k0) continue;
      const int half = columns(w) >> 1;
      const int boxes = (half + 63) >> 6;
      const uint32_t bytes = kABytes + (kBMn ? (uint32_t)boxes * 8192u : (uint32_t)half * 128u);
      const CUtensorMap *ma = kWeights ? a.maps + 2 * w.e : &maps.a;
      const CUtensorMap *mb = kWeights ? ma + 1 : &maps.b[(half >> 4) - 1];
      if (kWeights && w.e != known) {
        fence_map_acquire(ma);
        fence_map_acquire(mb);
        known = w.e;
      }
      const int m = w.a0 + (int)rank * kBM, n = w.b0 + (int)rank * half;
      for (int kb = w.k0; kb < w.k1; ++kb) {
        if (!mbar_wait_warp(&empty[st], ph ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) {
          ok = false;
          break;
        }
        const uint32_t bar = full0 + st * 8;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * bytes);
          uint8_t *da = ring + st * kStageBytes, *db = da + kABytes;
          const int k = kb * kBK;
          if (kWeights) {
            tma_load_2d_pair(da, ma, bar, m, k);
            tma_load_2d_pair(da + 8192, ma, bar, m + 64, k);
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(db + b * 8192, mb, bar, n + 64 * b, k);
          } else {
            if (kAMn) {
              tma_load_3d_pair(da, ma, bar, m, k, w.e);
              tma_load_3d_pair(da + 8192, ma, bar, m + 64, k, w.e);
            } else {
              tma_load_3d_pair(da, ma, bar, k, m, w.e);
            }
            tma_load_2d_pair(db, mb, bar, k, n);
          }
        }
        ++issued;
        if (++st == (uint32_t)kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (rank == 0) {
      // every copy of both CTAs completes on these barriers
      const uint32_t n = min(issued, (uint32_t)kStages);
      for (uint32_t i = 0; i < n; ++i) {
        st = st == 0 ? kStages - 1 : st - 1;
        if (st == (uint32_t)kStages - 1) ph ^= 1u;
        mbar_wait_drain(&full[st], ph);
      }
    } else if (!ok) {
      // the odd CTA's copies complete on the even CTA's barriers: after an
      // abort give copies in flight time to land before leaving
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------- MMA issuer --
    if (rank == 0) {
      constexpr uint32_t kAStep = kAMn ? 128 : 2, kBStep = kBMn ? 128 : 2;  // 16 of depth
      constexpr uint32_t kAHi = kAMn ? kDescHiMn : kDescHiK, kBHi = kBMn ? kDescHiMn : kDescHiK;
      const uint32_t a_lo = smem_u32(ring) >> 4 | (kAMn ? kDescLoMn : kDescLoK);
      const uint32_t b_lo = smem_u32(ring + kABytes) >> 4 | (kBMn ? kDescLoMn : kDescLoK);
      uint32_t st = 0, ph = 0, tl = 0;
      bool ok = true;
      Work w;
      for (int i = 0; ok && sch.at(i, &w); ++i) {
        if (w.k1 <= w.k0) continue;
        const uint32_t idesc = idesc_16(a.dtype, kAMn, kBMn, 2 * kBM, columns(w));
        for (int from = w.k0; ok && from < w.k1; from += kFine ? kFineStages : w.k1 - w.k0) {
          const int to = kFine ? min(from + kFineStages, w.k1) : w.k1;
          const uint32_t buf = tl & 1u, use = tl >> 1;
          ++tl;
          if (!mbar_wait_warp(&tempty[buf], (use & 1u) ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d0 = tmem_base + buf * kTileN;
          for (int kb = from; kb < to; ++kb) {
            if (!mbar_wait_warp(&full[st], ph, abort_flag, a.status, kStatusTimeoutDense)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t ad = a_lo + st * (kStageBytes >> 4), bd = b_lo + st * (kStageBytes >> 4);
            if (elect_one()) {
#pragma unroll
              for (uint32_t q = 0; q < 4; ++q)
                umma_16_pair(d0, ad + q * kAStep, kAHi, bd + q * kBStep, kBHi, idesc,
                             kb > from || q > 0 ? 1u : 0u);
              umma_commit_pair(&empty[st], 3);
            }
            if (++st == (uint32_t)kStages) {
              st = 0;
              ph ^= 1u;
            }
          }
          if (ok && elect_one()) umma_commit_pair(&tfull[buf], 3);
        }
      }
      if (elect_one()) umma_commit_pair(fin, 1);
      __syncwarp();
      mbar_wait_drain(fin, 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue --
    if (kFine) more_registers<kFineEpiRegs>();
    // warps w and w + 4 share 32 TMEM lanes and take every other 32 columns
    Slots<2> slot = {slots + warp * kOutBytes, 0, false};
    const int quad = warp & 3, turn = (warp >> 2) * 32;
    uint32_t tl = 0;
    Work w;
    for (int i = 0; sch.at(i, &w); ++i) {
      const bool none = w.k1 <= w.k0;  // an expert without rows: zeros
      const int m0 = w.a0 + (int)rank * kBM + quad * 32;
      const int cend = m0 < a.M ? w.n : 0;
      bool ok = true;
      uint32_t tb = 0;
      // the next accumulator
      auto take = [&]() {
        const uint32_t buf = tl & 1u, use = tl >> 1;
        ++tl;
        tb = tmem_base + ((uint32_t)(quad * 32) << 16) + buf * kTileN;
        ok = mbar_wait_warp(&tfull[buf], use & 1u, abort_flag, a.status, kStatusTimeoutDense);
        tc_fence_after();
      };
      auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed(cluster_addr(&tempty[(tl - 1) & 1u], 0));
      };
      // kFine: the sums of all accumulators; else the one accumulator is read where it is used
      float sums[kFine ? kChunks : 1][32];
      if constexpr (kFine) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sums[i][j] = 0.f;
        for (int from = w.k0; ok && from < w.k1; from += kFineStages) {
          take();
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            if (turn + 64 * i < w.n) {
              float v[32];
              tmem_ld32(tb + turn + 64 * i, v);
#pragma unroll
              for (int j = 0; j < 32; ++j) sums[i][j] += v[j];
            }
          }
          hand_back();
        }
      } else if (!none) {
        take();
      }
      // warps meet at a split tile: all of them leave there, or none
      if (!kWeights && i < sch.pieces) ok = epi_all(ok && !*abort_flag);
      if (!ok) break;
      // 32 columns of the accumulator, the warp's i-th
      auto columns_of = [&](int i, float (&v)[32]) {
        if constexpr (kFine) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = sums[i][j];
        } else {
          tmem_ld32(tb + turn + 64 * i, v);
        }
      };
      if constexpr (kWeights) {
        const bool wide = a.out_dtype == MOE_DTYPE_FP32;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c = turn + 64 * i;
          if (c >= cend) break;
          float v[32];
          if (none) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
          } else {
            columns_of(i, v);
          }
          Rows32 held;
          if (a.accumulate)
            held.load(static_cast<const char *>(a.d) +
                          (((int64_t)w.e * a.M + m0) * a.N + w.b0 + c) * (wide ? 4 : 2),
                      a.N, a.M - m0, a.N - w.b0 - c, a.out_dtype, lane);
          uint8_t *p = wide ? slot.take32(lane) : slot.take16(lane);
          if (a.accumulate) held.add_to(v, p, a.out_dtype, lane);
          if (wide)
            put32(p, lane, v);
          else
            put16(p, lane, a.out_dtype, v);
          send_3d(&maps.d, p, lane, w.b0 + c, m0, w.e);
        }
      } else {
        const int col = m0 + lane;
        bool last = true;
        auto place = [&](int part, int c) {
          const int s = sch.slot(sch.first_worker(w.tile) + part, w.tile);
          return a.part + ((size_t)(s * 2 + (int)rank) * a.part_chunks + c / 32) * (kBM * 32) +
                 quad * 1024 + lane * 4;
        };
        if (w.parts > 1) {
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int c = turn + 64 * i;
            if (c >= w.n) break;
            float v[32];
            columns_of(i, v);
            float *mine = place(w.part, c);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              __stcg(reinterpret_cast<float4 *>(mine + q * 128),
                     make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
          }
          epi_all(true);
          if (threadIdx.x == 0) *last_flag = arrive_last(a.counters + 2 * w.tile + rank, w.parts);
          epi_all(true);
          last = *last_flag != 0;
        }
        if (last) {
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int c = turn + 64 * i;
            if (c >= w.n) break;
            float v[32];
            if (w.parts == 1) {
              columns_of(i, v);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.f;
              // (two parts' loads at a time took longer: 24.7 us instead of 21.5 for eight
              // experts of 4096 x 1536 with a row each)
              for (int part = 0; part < w.parts; ++part) {
                const float *p = place(part, c);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  const float4 f = __ldcg(reinterpret_cast<const float4 *>(p + q * 128));
                  v[4 * q] += f.x;
                  v[4 * q + 1] += f.y;
                  v[4 * q + 2] += f.z;
                  v[4 * q + 3] += f.w;
                }
              }
            }
            if (col < a.M) store_rows(a.d, a.ldd, a.out_dtype, w.b0 + c, w.n - c, col, v);
          }
        }
      }
      if (!kFine && !none) hand_back();
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

// Each expert's maps of dy and x, ending with its rows.
struct MapTemplates {
  CUtensorMap dy, x;
};
__device__ __forceinline__ void make_map(CUtensorMap *to, const CUtensorMap &from, const void *base,
                                         int rows) {
  const uint4 *s = reinterpret_cast<const uint4 *>(&from);
  uint4 *d = reinterpret_cast<uint4 *>(to);
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = s[i];
  asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(to),
               "l"(base)
               : "memory");
  asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(to),
               "r"(rows)
               : "memory");
}
__global__ void grouped_maps_kernel(const __grid_constant__ MapTemplates t, const int32_t *offsets,
                                    int E, int R, const uint8_t *dy, int64_t dy_bytes,
                                    const uint8_t *x, int64_t x_bytes, CUtensorMap *maps) {
  pdl_wait();
  pdl_launch_dependents();
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e < E) {
    const int o = __ldg(offsets + e), end = __ldg(offsets + e + 1);
    if (o >= 0 && o < end && end <= R) {  // (the others are not used)
      make_map(maps + 2 * e, t.dy, dy + o * dy_bytes, end - o);
      make_map(maps + 2 * e + 1, t.x, x + o * x_bytes, end - o);
    }
  }
  asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}

// Clusters that can run at once (per device, queried once).
template <int kMode, bool kFine>
cudaError_t resident_clusters(int *out) {
  auto kern = grouped_pair_kernel<kMode, kFine>;
  static std::atomic<int> resident[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (resident[dev] == 0) {
    static std::atomic<bool> allowed[64];
    cudaError_t e = allow_smem(kern, smem_bytes<kMode>(kMaxE), allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(num_sms() / 2 * 2));
    cfg.blockDim = dim3(kThreads<kFine>);
    cfg.dynamicSmemBytes = smem_bytes<kMode>(kMaxE);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    resident[dev] = std::min(std::min(n, num_sms() / 2), kMaxClusters);
  }
  *out = resident[dev];
  return cudaSuccess;
}

template <int kMode, bool kFine>
cudaError_t start(const GroupedMaps &maps, const GroupedArgs &a, int clusters, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * clusters));
  cfg.blockDim = dim3(kThreads<kFine>);
  cfg.dynamicSmemBytes = smem_bytes<kMode>(a.E);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_pair_kernel<kMode, kFine>, maps, a);
}

// [E][rows][cols], dense.
bool map_3d(CUtensorMap *m, int dtype, CUtensorMapSwizzle sw, const void *p, int E, int64_t rows,
            int64_t cols, int box_rows, int box_cols) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)E};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * type_bytes(dtype),
                                 (cuuint64_t)rows * cols * type_bytes(dtype)};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  return encode_map(m, map_type(dtype), sw, p, 3, dims, strides, box);
}

// Accumulator columns of the largest tile of R rows.
int part_cols(int R) { return std::min(kTileN, (R + 31) / 32 * 32); }

template <int kMode, bool kFine>
cudaError_t rows_product(const GroupedGemm &g, cudaStream_t s) {
  int resident = 0;
  cudaError_t e = resident_clusters<kMode, kFine>(&resident);
  if (e != cudaSuccess) return e;
  const bool grad = kMode == kRowGrad;
  const int M = grad ? g.K : g.N, depth = grad ? g.N : g.K;
  GroupedArgs a = {};
  a.offsets = g.offsets;
  a.R = g.R;
  a.E = g.E;
  a.M = M;
  a.nkb = (depth + kBK - 1) / kBK;
  a.mt = (M + kTileM - 1) / kTileM;
  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.d = g.d;
  a.ldd = grad ? g.ldx : g.ldy;
  a.part = g.part;
  a.part_chunks = part_cols(g.R) / 32;
  a.counters = g.status + kSplitCounterWord;
  a.status = g.status;
  GroupedMaps maps = {};
  const CUtensorMapSwizzle in = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = grad ? map_3d(&maps.a, g.dtype, in, g.w, g.E, g.N, g.K, kBK, 64)
                 : map_3d(&maps.a, g.dtype, in, g.w, g.E, g.N, g.K, kBM, kBK);
  for (int i = 0; i < 8; ++i)
    ok = ok && map_2d(&maps.b[i], g.dtype, in, grad ? g.dy : g.x, g.R, depth, grad ? g.ldy : g.ldx,
                      16 * (i + 1), kBK);
  if (!ok) return cudaErrorInvalidValue;
  // at most this many tiles, each of which may be split
  const int64_t tiles = ((int64_t)std::min(g.E, g.R) + g.R / kTileN) * a.mt;
  const int64_t most = tiles * std::max(1, std::min(kMaxParts, a.nkb / kMinPart));
  return start<kMode, kFine>(maps, a, (int)std::min<int64_t>(resident, most), s);
}

}  // namespace

// Two pieces to a cluster, 256 x (rows of a tile) fp32 each.
size_t grouped_part_bytes(int R) {
  return (size_t)2 * kMaxClusters * kTileM * part_cols(R) * 4;
}

cudaError_t launch_grouped_rows(const GroupedGemm &g, bool grad, cudaStream_t s) {
  if (grad) return rows_product<kRowGrad, false>(g, s);
  return g.out_dtype == MOE_DTYPE_FP32 ? rows_product<kForward, true>(g, s)
                                       : rows_product<kForward, false>(g, s);
}

namespace {

template <bool kFine>
cudaError_t weight_grad(const GroupedGemm &g, cudaStream_t s) {
  int resident = 0;
  cudaError_t e = resident_clusters<kWeightGrad, kFine>(&resident);
  if (e != cudaSuccess) return e;
  const CUtensorMapSwizzle in = CU_TENSOR_MAP_SWIZZLE_128B;
  MapTemplates t;
  bool ok = map_2d(&t.dy, g.dtype, in, g.dy, g.R, g.N, g.ldy, kBK, 64) &&
            map_2d(&t.x, g.dtype, in, g.x, g.R, g.K, g.ldx, kBK, 64);
  GroupedMaps maps = {};
  const CUtensorMapSwizzle out =
      g.out_dtype == MOE_DTYPE_FP32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  ok = ok && map_3d(&maps.d, g.out_dtype, out, g.d, g.E, g.N, g.K, 32, 32);
  if (!ok) return cudaErrorInvalidValue;
  GroupedArgs a = {};
  a.offsets = g.offsets;
  a.R = g.R;
  a.E = g.E;
  a.M = g.N;
  a.N = g.K;
  a.bn = std::min(kTileN, (g.K + 63) / 64 * 64);
  a.mt = (g.N + kTileM - 1) / kTileM;
  a.nt = (g.K + a.bn - 1) / a.bn;
  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.d = g.d;
  a.accumulate = g.accumulate;
  a.maps = g.maps;
  a.status = g.status;
  const int threads = 128;
  e = launch_pdl(grouped_maps_kernel, dim3((unsigned)((g.E + threads - 1) / threads)),
                 dim3(threads), 0, s, t, g.offsets, g.E, g.R, static_cast<const uint8_t *>(g.dy),
                 g.ldy * 2, static_cast<const uint8_t *>(g.x), g.ldx * 2, g.maps);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)g.E * a.mt * a.nt;
  return start<kWeightGrad, kFine>(maps, a, (int)std::min<int64_t>(resident, tiles), s);
}

}  // namespace

cudaError_t launch_grouped_weight_grad(const GroupedGemm &g, cudaStream_t s) {
  return g.out_dtype == MOE_DTYPE_FP32 ? weight_grad<true>(g, s) : weight_grad<false>(g, s);
}

}  // namespace moe
