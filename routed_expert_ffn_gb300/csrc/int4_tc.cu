// Products with 4-bit weights on the tensor cores (tcgen05, sm_103a): y = act(x W^T +
// bias) + residual of one matrix, or y_p = W_e x_p for the rows p of each expert e.
//
// Bound: HBM for few rows, which reads half a byte for each weight.  To keep up an SM
// turns 48 codes a clock into 16-bit numbers, a good half of what its schedulers issue
// (13 instructions for a word of eight).  So every weight is unpacked once for all rows of
// a tile: 128 rows of W are the MMA's M, up to 64 rows of x its N, and the unpacked
// numbers go to TMEM, where the MMA reads its A operand: through shared memory they would
// be written and read once more, twice what it moves anyway.
//
// The numbers are code - 8, exact in 16 bits, not yet scaled: the sums of one group of
// columns are an accumulator of their own, which the epilogue's warps multiply by the
// group's scale (a lane is a row of W) and add in fp32 registers.  Neither codes nor scales
// are rounded, and the tensor cores' truncating additions go over 128 products at most.
//
// Depth goes by units of 256 columns (a row's 128 bytes of codes), unpacked in steps of 64
// (32 TMEM columns of 16-bit pairs) and accumulated in blocks of 128.  Tiles, and the depth
// of those that do not fill a round of the SMs, are dealt out as in grouped_pair.cu.
//
// CTA = 14 warps, one CTA an SM:
//   warps 0-3    scale and add the accumulators; the epilogue (32 TMEM lanes each)
//   warps 4-11   unpack, two sets of four (32 TMEM lanes each), every other step
//   warp 12      TMA: codes and rows of x
//   warp 13      TMEM allocation; one thread issues the MMAs
// Every wait is bounded; on expiry the CTA latches the status bit and leaves its loops.
#include <algorithm>

#include "grouped.cuh"
#include "int4.cuh"
#include "pair_ptx.cuh"

namespace moe {

namespace {

constexpr int kAddWarps = 4, kUnpackWarps = 8;
constexpr int kTmaWarp = kAddWarps + kUnpackWarps, kMmaWarp = kTmaWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kUnit = 256, kStep = 64, kSteps = kUnit / kStep;
constexpr uint32_t kCodeBytes = kBM * kUnit / 2;
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kABufs = 8, kAColsStep = kStep / 2;  // operand: [0, 256)
constexpr uint32_t kDCol = kABufs * kAColsStep;         // accumulators: [256, 512)
constexpr int kMaxCtas = 160;  // (a GB300 has 152 SMs)
constexpr int kMaxParts = 16;

// Rows of x of a tile at most, and where the accumulators of a block lie: one for each
// group, kGroup columns apart.
template <int kGroup, int kN>
struct Shape {
  static constexpr int x_step = kN * kStep * 2;  // bytes of x for one step
  static constexpr uint32_t stage = kCodeBytes + kSteps * x_step;
  static constexpr int stages = kN == 16 ? 8 : (kN == 32 ? 6 : 4);
  static constexpr uint32_t d_cols = kGroup == 128 ? 64 : 128;  // of a block
  static constexpr uint32_t d_bufs = (kTmemCols - kDCol) / d_cols;
  static constexpr int groups = 128 / kGroup;  // of a block
  static_assert(kN <= kGroup && kN <= 64, "accumulator columns");
};
template <int kGroup, int kN>
constexpr size_t smem_bytes(int E) {
  typedef Shape<kGroup, kN> S;
  return 1024 + (size_t)S::stages * S::stage + (2 * kMaxStages + 2 * kABufs + 2 * S::d_bufs + 1) * 8 +
         32 + (size_t)2 * (E + 1) * 4;
}
static_assert(smem_bytes<128, 16>(kMaxE) <= 232448 && smem_bytes<128, 32>(kMaxE) <= 232448 &&
                  smem_bytes<128, 64>(kMaxE) <= 232448,
              "shared memory per CTA");

struct TcMaps {
  CUtensorMap q;     // codes [E][N][K/2]
  CUtensorMap x[4];  // boxes of 16, 32, 48, 64 rows
};
struct TcArgs {
  const int32_t *offsets;
  int T, E, N, K;
  int mt, units, groups;
  int dtype, out_dtype, act;
  const uint16_t *scale;
  const void *bias, *residual;
  void *y;
  int64_t ldr, ldy;
  float *part;
  uint32_t *counters, *status;
};

// D[tmem] (+)= A[tmem] B[smem]^T: A's rows in the TMEM lanes, two elements to a column.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
      " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

template <bool kFp16>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (kFp16)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// A word of eight codes as code - 8, pairs in the order of the columns: a pair is a byte,
// its halves moved to the low bits of two 16-bit numbers, which the exponent of 128
// (bf16) or 1024 (fp16) makes 128 + code; less 136 that is exact.
template <bool kFp16>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t *to) {
  constexpr uint32_t kOne = kFp16 ? 0x64006400u : 0x43004300u;
  constexpr uint32_t kZero = kFp16 ? 0x64086408u : 0x43084308u;
  const uint32_t high = w >> 4;
#pragma unroll
  for (uint32_t b = 0; b < 4; ++b)
    to[b] = sub2<kFp16>((__byte_perm(w, high, 0x4000u + (0x400u | b << 8) + b) & 0x000f000fu) | kOne,
                        kZero);
}

// `and` over the adding warps' 128 threads.
__device__ __forceinline__ bool add_all(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.and.pred b, 1, 128, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

// A row's scales of one unit, as they lie.
template <int kGroup>
struct UnitScales {
  static constexpr int count = kUnit / kGroup;  // 8, 4 or 2
  uint32_t w[count / 2];
  __device__ __forceinline__ void load(const uint16_t *row, int unit, int groups) {
    const int g = unit * count;
    const uint16_t *p = row + g;
    if (groups % count == 0) {  // whole units, as aligned as they are long
      if constexpr (kGroup == 32) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
      } else if constexpr (kGroup == 64) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
      } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
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

template <bool kFp16, int kGroup, int kN>
__global__ void __launch_bounds__(kThreads, 1)
    int4_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a) {
  typedef Shape<kGroup, kN> S;
  typedef RowSchedule<kN, 16, kBM, kMaxParts, 1> Tiles;
  constexpr int kStages = S::stages;
  constexpr int kDtype = kFp16 ? MOE_DTYPE_FP16 : MOE_DTYPE_BF16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + kStages * S::stage);
  uint64_t *empty = full + kMaxStages;
  uint64_t *a_full = empty + kMaxStages;
  uint64_t *a_empty = a_full + kABufs;
  uint64_t *d_full = a_empty + kABufs;
  uint64_t *d_empty = d_full + S::d_bufs;
  uint64_t *fin = d_empty + S::d_bufs;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *last_flag = abort_flag + 1;
  int32_t *seg = reinterpret_cast<int32_t *>(tmem_slot + 4);
  int32_t *first = seg + a.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kUnpackWarps + 1);
    }
    for (uint32_t b = 0; b < kABufs; ++b) {
      mbar_init(&a_full[b], 4);
      mbar_init(&a_empty[b], 1);
    }
    for (uint32_t b = 0; b < S::d_bufs; ++b) {
      mbar_init(&d_full[b], 1);
      mbar_init(&d_empty[b], kAddWarps);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.x[0]);
  }
  pdl_wait();
  pdl_launch_dependents();
  make_tables(a.offsets, a.E, a.T, seg, first, a.status,
              [&](int m) { return Tiles::row_tiles(m) * a.mt; });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  Tiles sch;
  sch.seg = seg;
  sch.first = first;
  sch.E = a.E;
  sch.mt = a.mt;
  sch.nkb = a.units;
  sch.cid = blockIdx.x;
  sch.ncl = gridDim.x;
  sch.start();
  auto steps_of = [&](int unit) { return min(kSteps, (a.K - unit * kUnit + kStep - 1) / kStep); };
  Work w;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------ TMA producer --
    uint32_t st = 0, ph = 0, issued = 0;
    bool ok = true;
    for (int i = 0; ok && sch.at(i, &w); ++i) {
      const int n16 = (w.n + 15) & ~15;
      const CUtensorMap *mx = &maps.x[(n16 >> 4) - 1];
      for (int u = w.k0; u < w.k1; ++u) {
        if (!mbar_wait_warp(&empty[st], ph ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) {
          ok = false;
          break;
        }
        const int steps = steps_of(u);
        if (elect_one()) {
          uint8_t *to = ring + st * S::stage;
          mbar_arrive_expect_tx(&full[st], kCodeBytes + (uint32_t)(steps * n16 * kStep * 2));
          tma_load_3d(to, &maps.q, &full[st], u * (kUnit / 2), w.a0, w.e);
          for (int s = 0; s < steps; ++s)
            tma_load_2d(to + kCodeBytes + s * S::x_step, mx, &full[st], u * kUnit + s * kStep, w.b0);
        }
        ++issued;
        if (++st == (uint32_t)kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    const uint32_t n = min(issued, (uint32_t)kStages);
    for (uint32_t i = 0; i < n; ++i) {
      st = st == 0 ? kStages - 1 : st - 1;
      if (st == (uint32_t)kStages - 1) ph ^= 1u;
      mbar_wait_drain(&full[st], ph);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------- MMA issuer --
    const uint32_t b_lo = smem_u32(ring + kCodeBytes) >> 4 | kDescLoK;
    uint32_t st = 0, ph = 0, ab = 0, aph = 0, db = 0, dph = 0;
    bool ok = true;
    for (int i = 0; ok && sch.at(i, &w); ++i) {
      const uint32_t idesc = idesc_16(kDtype, false, false, kBM, (w.n + 15) & ~15);
      for (int u = w.k0; ok && u < w.k1; ++u) {
        if (!mbar_wait_warp(&full[st], ph, abort_flag, a.status, kStatusTimeoutDense)) {
          ok = false;
          break;
        }
        const int steps = steps_of(u);
        for (int s = 0; s < steps; ++s) {
          if ((s & 1) == 0 &&
              !mbar_wait_warp(&d_empty[db], dph ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) {
            ok = false;
            break;
          }
          if (!mbar_wait_warp(&a_full[ab], aph, abort_flag, a.status, kStatusTimeoutDense)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d0 = tmem_base + kDCol + db * S::d_cols, a0 = tmem_base + ab * kAColsStep;
            const uint32_t bd = b_lo + ((st * S::stage + (uint32_t)s * S::x_step) >> 4);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
              const uint32_t k = (uint32_t)(s & 1) * kStep + q * 16;  // in the block
              umma_ts(d0 + k / kGroup * kGroup, a0 + q * 8, (uint64_t)kDescHiK << 32 | (bd + 2 * q),
                      idesc, k % kGroup != 0 ? 1u : 0u);
            }
            umma_commit(&a_empty[ab]);
            if ((s & 1) == 1 || s + 1 == steps) umma_commit(&d_full[db]);
            if (s + 1 == steps) umma_commit(&empty[st]);
          }
          if (++ab == kABufs) {
            ab = 0;
            aph ^= 1u;
          }
          if ((s & 1) == 1 || s + 1 == steps) {
            if (++db == S::d_bufs) {
              db = 0;
              dph ^= 1u;
            }
          }
        }
        if (++st == (uint32_t)kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (elect_one()) umma_commit(fin);
    __syncwarp();
    mbar_wait_drain(fin, 0);
    __syncwarp();
  } else if (warp >= kAddWarps) {
    // ---------------------------------------------------------- unpackers --
    const int quad = warp & 3, set = (warp - kAddWarps) >> 2;
    const int r = quad * 32 + lane;
    const uint32_t to = tmem_base + ((uint32_t)(quad * 32) << 16);
    uint32_t st = 0, ph = 0, ab = 0, aph = 0;
    bool ok = true;
    for (int i = 0; ok && sch.at(i, &w); ++i) {
      for (int u = w.k0; u < w.k1; ++u) {
        if (!mbar_wait_warp(&full[st], ph, abort_flag, a.status, kStatusTimeoutDense)) {
          ok = false;
          break;
        }
        // this set's two steps of the unit: 32 bytes of the row each
        const uint8_t *row = ring + st * S::stage + r * 128;
        uint4 v[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            v[h][c] = *reinterpret_cast<const uint4 *>(
                row + (((4 * h + 2 * set + c) ^ (r & 7)) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        const int steps = steps_of(u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int s = 2 * h + set;
          if (s < steps) {
            const uint32_t at = ab + (uint32_t)s, b = at & (kABufs - 1);
            const uint32_t p = aph ^ (at >= kABufs ? 1u : 0u);
            uint32_t o[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              unpack8<kFp16>(v[h][c].x, o + 16 * c);
              unpack8<kFp16>(v[h][c].y, o + 16 * c + 4);
              unpack8<kFp16>(v[h][c].z, o + 16 * c + 8);
              unpack8<kFp16>(v[h][c].w, o + 16 * c + 12);
            }
            if (!mbar_wait_warp(&a_empty[b], p ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) {
              ok = false;
              break;
            }
            tc_fence_after();
            tmem_st32(to + b * kAColsStep, o);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a_full[b]);
          }
        }
        if (!ok) break;
        ab += (uint32_t)steps;
        if (ab >= kABufs) {
          ab -= kABufs;
          aph ^= 1u;
        }
        if (++st == (uint32_t)kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------- scaling, adding, epilogue --
    const int quad = warp;
    const uint32_t from = tmem_base + ((uint32_t)(quad * 32) << 16) + kDCol;
    uint32_t db = 0, dph = 0;
    bool ok = true;
    auto scales_of = [&](const Work &t) {
      const int n = min(t.a0 + quad * 32 + lane, a.N - 1);
      return a.scale + ((int64_t)t.e * a.N + n) * a.groups;
    };
    UnitScales<kGroup> next;
    Work w_next;
    bool more = sch.at(0, &w_next);
    if (more) next.load(scales_of(w_next), w_next.k0, a.groups);
    for (int i = 0; more;) {
      w = w_next;
      more = sch.at(++i, &w_next);
      float acc[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) acc[j] = 0.f;
      const uint16_t *row = scales_of(w);
      for (int u = w.k0; u < w.k1; ++u) {
        const UnitScales<kGroup> sc = next;
        if (u + 1 < w.k1)
          next.load(row, u + 1, a.groups);
        else if (more)
          next.load(scales_of(w_next), w_next.k0, a.groups);
        const int blocks = (steps_of(u) + 1) >> 1;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b < blocks) {
            ok = mbar_wait_warp(&d_full[db], dph, abort_flag, a.status, kStatusTimeoutDense);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < S::groups; ++g) {
              const int at = b * S::groups + g;
              if (u * UnitScales<kGroup>::count + at >= a.groups) break;  // never accumulated
              const float f = unpack16(kDtype, at & 1 ? sc.w[at / 2] >> 16 : sc.w[at / 2]).x;
#pragma unroll
              for (int c = 0; c < kN; c += 16) {
                float v[16];
                tmem_ld16f(from + db * S::d_cols + (uint32_t)(g * kGroup + c), v);
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(f, v[j], acc[c + j]);
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[db]);
            if (++db == S::d_bufs) {
              db = 0;
              dph ^= 1u;
            }
          }
        }
        if (!ok) break;
      }
      // warps meet at a split tile: all of them leave there, or none
      if (i <= sch.pieces) ok = add_all(ok && !*abort_flag);
      if (!ok) break;
      bool last = true;
      if (w.parts > 1) {
        auto place = [&](int part) {
          const int s = sch.slot(sch.first_worker(w.tile) + part, w.tile);
          return a.part + (size_t)s * (kBM * kN) + (quad * 32 + lane) * 4;
        };
        float *mine = place(w.part);
#pragma unroll
        for (int q = 0; q < kN / 4; ++q)
          __stcg(reinterpret_cast<float4 *>(mine + q * (kBM * 4)),
                 make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]));
        __threadfence();
        add_all(true);
        if (threadIdx.x == 0) {
          const uint32_t n = atomicAdd(a.counters + w.tile, 1u) + 1;
          if (n == (uint32_t)w.parts) a.counters[w.tile] = 0;  // nobody else comes
          __threadfence();
          *last_flag = n == (uint32_t)w.parts;
        }
        add_all(true);
        last = *last_flag != 0;
        __threadfence();
        if (last) {
#pragma unroll
          for (int j = 0; j < kN; ++j) acc[j] = 0.f;
          for (int part = 0; part < w.parts; ++part) {
            const float *p = place(part);
#pragma unroll
            for (int q = 0; q < kN / 4; ++q) {
              const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + q * (kBM * 4)));
              acc[4 * q] += v.x;
              acc[4 * q + 1] += v.y;
              acc[4 * q + 2] += v.z;
              acc[4 * q + 3] += v.w;
            }
          }
        }
      }
      const int n = w.a0 + quad * 32 + lane;
      if (last && n < a.N) {
        const bool wide = a.out_dtype == MOE_DTYPE_FP32;
        auto load = [&](const void *p, int64_t at) {
          return wide ? static_cast<const float *>(p)[at]
                      : unpack16(a.out_dtype, static_cast<const uint16_t *>(p)[at]).x;
        };
        if (a.bias != nullptr) {
          const float b = load(a.bias, n);
#pragma unroll
          for (int j = 0; j < kN; ++j) acc[j] += b;
        }
        if (wide)
          activate_all<true>(a.act, acc);
        else
          activate_all<false>(a.act, acc);
        if (a.residual != nullptr) {
#pragma unroll
          for (int j = 0; j < kN; ++j)
            if (j < w.n) acc[j] += load(a.residual, (int64_t)(w.b0 + j) * a.ldr + n);
        }
        const int64_t y0 = (int64_t)w.b0 * a.ldy + n;
        if (wide) {
          float *p = static_cast<float *>(a.y) + y0;
#pragma unroll
          for (int j = 0; j < kN; ++j)
            if (j < w.n) p[j * a.ldy] = acc[j];
        } else {
          uint16_t *p = static_cast<uint16_t *>(a.y) + y0;
#pragma unroll
          for (int j = 0; j < kN; ++j)
            if (j < w.n) p[j * a.ldy] = (uint16_t)pack16(a.out_dtype, acc[j], 0.f);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool kFp16, int kGroup, int kN>
cudaError_t start(const Int4Gemm &g, cudaStream_t s) {
  auto kern = int4_tc_kernel<kFp16, kGroup, kN>;
  static std::atomic<bool> allowed[64];
  cudaError_t e = allow_smem(kern, smem_bytes<kGroup, kN>(kMaxE), allowed);
  if (e != cudaSuccess) return e;
  TcArgs a = {};
  a.offsets = g.offsets;
  a.T = g.T;
  a.E = g.E;
  a.N = g.N;
  a.K = g.K;
  a.mt = (g.N + kBM - 1) / kBM;
  a.units = (g.K + kUnit - 1) / kUnit;
  a.groups = (g.K + kGroup - 1) / kGroup;
  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.act = g.act;
  a.scale = static_cast<const uint16_t *>(g.scale);
  a.bias = g.bias;
  a.residual = g.residual;
  a.y = g.y;
  a.ldr = g.ldr;
  a.ldy = g.ldy;
  a.part = g.part;
  a.counters = g.status + kSplitCounterWord;
  a.status = g.status;
  TcMaps maps = {};
  const cuuint64_t dims[3] = {(cuuint64_t)g.K / 2, (cuuint64_t)g.N, (cuuint64_t)g.E};
  const cuuint64_t strides[2] = {(cuuint64_t)g.K / 2, (cuuint64_t)g.N * (g.K / 2)};
  const cuuint32_t box[3] = {kUnit / 2, kBM, 1};
  bool ok = encode_map(&maps.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, g.q, 3,
                       dims, strides, box);
  for (int i = 0; i < kN / 16; ++i)
    ok = ok && map_2d(&maps.x[i], g.dtype, CU_TENSOR_MAP_SWIZZLE_128B, g.x, g.T, g.K, g.ldx,
                      16 * (i + 1), kStep);
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = ((int64_t)std::min(g.E, g.T) + g.T / kN) * a.mt;
  const int64_t most = std::min<int64_t>(tiles * std::min(kMaxParts, a.units),
                                         std::min(num_sms(), kMaxCtas));
  return launch_pdl(kern, dim3((unsigned)most), dim3(kThreads), smem_bytes<kGroup, kN>(g.E), s, maps,
                    a);
}

// Rows of a tile: as many as most experts have, if they are spread evenly.
template <bool kFp16, int kGroup>
cudaError_t by_rows(const Int4Gemm &g, cudaStream_t s) {
  const int rows = (g.T + g.E - 1) / g.E;
  if (rows <= 16) return start<kFp16, kGroup, 16>(g, s);
  if (rows <= 32 || kGroup == 32) return start<kFp16, kGroup, 32>(g, s);
  return start<kFp16, kGroup, kGroup == 32 ? 32 : 64>(g, s);
}
template <bool kFp16>
cudaError_t by_group(const Int4Gemm &g, cudaStream_t s) {
  if (g.group == 32) return by_rows<kFp16, 32>(g, s);
  return g.group == 64 ? by_rows<kFp16, 64>(g, s) : by_rows<kFp16, 128>(g, s);
}

}  // namespace

size_t int4_part_bytes(int T) {
  const int rows = T <= 16 ? 16 : (T <= 32 ? 32 : 64);
  return (size_t)2 * kMaxCtas * kBM * rows * 4;
}

cudaError_t launch_int4_tc(const Int4Gemm &g, cudaStream_t s) {
  return g.dtype == MOE_DTYPE_FP16 ? by_group<true>(g, s) : by_group<false>(g, s);
}

}  // namespace moe
