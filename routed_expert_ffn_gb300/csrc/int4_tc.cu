// Products with 4-bit weights on the tensor cores (tcgen05, sm_103a): y = act(x W^T +
// bias) + residual of one matrix, or y_p = W_e x_p for the rows p of each expert e.
//
// Bound: HBM for few rows, which reads half a byte for each weight.  To keep up an SM
// turns 48 codes a clock into 16-bit numbers, nine instructions for a word of eight.  So
// every weight is unpacked once for all rows of a tile: 128 rows of W are the MMA's M, up
// to 64 rows of x its N, and the unpacked numbers go to TMEM, where the MMA reads its A
// operand: through shared memory they would be written and read once more, twice what
// it moves anyway.  What a block costs now is the hand-over between the groups of warps (the
// MMAs of 256 x 128 codes by 64 rows take 670 clocks of about 1600).
//
// The numbers are code - 8, exact in 16 bits, not yet scaled: the sums of one group of
// columns are an accumulator of their own, which the epilogue's warps multiply by the
// group's scale (a lane is a row of W) and add in fp32 registers.  Neither codes nor scales
// are rounded, and the tensor cores' truncating additions go over 128 products at most.
//
// Depth goes by units of 256 columns (a row's 128 bytes of codes).  Tiles, and the depth
// of those that do not fill a round of the SMs, are dealt out as in grouped_pair.cu.
//
// CTA, one an SM:
//   warps 0-7    scale and add the accumulators; the epilogue (32 TMEM lanes each, and
//                half of the rows of x)
//   then         one or two sets of four warps that unpack (32 TMEM lanes each)
//   then         a warp for TMA (codes and rows of x), and one for TMEM's allocation, of
//                which one thread issues the MMAs
// Every wait is bounded; on expiry the CTA latches the status bit and leaves its loops.
// A wait takes some 100 clocks even when what it waits for is there, and each role of a block
// has two or three in a row: those that can be are asked for ahead (mbar_test).
//
// Measured: 14336 x 4096 with 16 rows 17 us, with 64 22, with 256 44; 32 experts of 4096 x 7168
// with 16 rows on average 149 us (3.4 TB/s).
#include <algorithm>

#include "grouped.cuh"
#include "int4.cuh"
#include "pair_ptx.cuh"

namespace moe {

namespace {

constexpr int kUnit = 256;
constexpr uint32_t kCodeBytes = kBM * kUnit / 2;
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kDCol = 256;  // operands: TMEM columns [0, 256), accumulators: [256, 512)
constexpr int kMaxCtas = 160;    // (a GB300 has 152 SMs)
constexpr int kMaxParts = 16;

// Rows of x of a tile at most (kN), and how depth is handed from one group of warps to
// the next: in blocks of `block` columns, unpacked into one of `bufs` operand buffers
// and accumulated into one of as many, where each group of columns has kN columns.
// A hand-over costs about 250 clocks whatever it hands over, and HBM brings 128 x 256
// codes in 680: blocks are as large as TMEM holds twice.
template <int kGroup, int kN>
struct Shape {
  // Sets of four unpacking warps: one is enough where the adding warps have the most to do
  // (203 rows of 7176 x 2080 in groups of 32: 53 us with two, 50 with one, 57 with four; 32
  // experts of 4096 x 7168 with 16 rows in groups of 64: 150, 158 and 190).
  static constexpr int sets = kN == 64 || (kN == 32 && kGroup == 32) ? 1 : 2;
  static constexpr int add_warps = 8, unpack_warps = 4 * sets;
  static constexpr int tma_warp = add_warps + unpack_warps, mma_warp = tma_warp + 1;
  static constexpr int threads = (mma_warp + 1) * 32;
  static constexpr int x_box = kN * 128;  // bytes of 64 columns of x
  static constexpr uint32_t stage = kCodeBytes + kUnit / 64 * x_box;
  static constexpr int stages = kN == 16 ? 8 : (kN == 32 ? 6 : 4);
  static constexpr int block = 256 / kGroup * kN <= 128 ? 256 : 128;
  static constexpr int blocks = kUnit / block;     // of a unit
  static constexpr int groups = block / kGroup;    // of a block
  static constexpr uint32_t a_cols = block / 2, d_cols = groups * kN;
  static constexpr uint32_t bufs = d_cols <= 64 && a_cols <= 64 ? 4 : 2;
  static_assert(bufs * a_cols <= kDCol && bufs * d_cols <= kTmemCols - kDCol, "TMEM columns");
};
template <int kGroup, int kN>
constexpr size_t smem_bytes(int E) {
  typedef Shape<kGroup, kN> S;
  return 1024 + (size_t)S::stages * S::stage + (2 * kMaxStages + 3 * S::bufs + 1) * 8 + 32 +
         (size_t)2 * (E + 1) * 4;
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
  int first;  // row of x that is the first of the rows made
  const float *factor;
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
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "n"(kDescHiK), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x kCols consecutive columns; nothing is there before tmem_ld_wait.
template <int kCols>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t *r) {
  if constexpr (kCols == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else {
    tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(r));
  }
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15])
      : "memory");
}

// `and` over the adding warps' 256 threads.
template <int kCount>
__device__ __forceinline__ bool add_all(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.and.pred b, 1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(kCount)
      : "memory");
  return r != 0;
}

template <int kGroup, int kN>
__global__ void __launch_bounds__(Shape<kGroup, kN>::threads, 1)
    int4_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a) {
  typedef Shape<kGroup, kN> S;
  typedef RowSchedule<kN, 16, kBM, kMaxParts, 1> Tiles;
  constexpr int kStages = S::stages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + kStages * S::stage);
  uint64_t *empty = full + kMaxStages;
  uint64_t *a_full = empty + kMaxStages;  // a block is unpacked
  uint64_t *done = a_full + S::bufs;      // it is multiplied: its operands are free, its sums there
  uint64_t *d_empty = done + S::bufs;     // they are read
  uint64_t *fin = d_empty + S::bufs;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *last_flag = abort_flag + 1;
  int32_t *seg = reinterpret_cast<int32_t *>(tmem_slot + 4);
  int32_t *first = seg + a.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], S::unpack_warps + 1);
    }
    for (uint32_t b = 0; b < S::bufs; ++b) {
      mbar_init(&a_full[b], S::unpack_warps);
      mbar_init(&done[b], 1);
      mbar_init(&d_empty[b], S::add_warps);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == S::mma_warp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == S::tma_warp && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.x[0]);
  }
  // The launch before this one made the rows of x, and waited for all before it: what
  // else is read here is there.
  pdl_launch_dependents();
  make_tables(a.offsets, a.E, a.T, a.first, min(a.T, a.first + kInt4Rows), seg, first, a.status,
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
  auto blocks_of = [&](int unit) {
    return min(S::blocks, (a.K - unit * kUnit + S::block - 1) / S::block);
  };
  Work w;
  uint32_t st = 0, ph = 0;    // stages of codes and rows
  uint32_t buf = 0, bph = 0;  // blocks

  if (warp == S::tma_warp) {
    // ------------------------------------------------------ TMA producer --
    uint32_t issued = 0;
    bool ok = true;
    auto copy_codes = [&](const Work &v, int u, uint32_t to) {
      const uint32_t n16 = (uint32_t)(v.n + 15) & ~15u;
      mbar_arrive_expect_tx(&full[to], kCodeBytes + kUnit / 64 * n16 * 128);
      tma_load_3d(ring + to * S::stage, &maps.q, &full[to], u * (kUnit / 2), v.a0, v.e);
    };
    auto copy_rows = [&](const Work &v, int u, uint32_t to) {
      const CUtensorMap *mx = &maps.x[((v.n + 15) >> 4) - 1];
#pragma unroll
      for (int s = 0; s < kUnit / 64; ++s)
        tma_load_2d(ring + to * S::stage + kCodeBytes + s * S::x_box, mx, &full[to],
                    u * kUnit + s * 64, v.b0 - a.first);
    };
    // the first round of codes does not wait for the rows
    uint32_t early = 0;
    for (int i = 0; early < (uint32_t)kStages && sch.at(i, &w); ++i)
      for (int u = w.k0; u < w.k1 && early < (uint32_t)kStages; ++u, ++early)
        if (elect_one()) copy_codes(w, u, early);
    pdl_wait();
    for (int i = 0; ok && sch.at(i, &w); ++i) {
      for (int u = w.k0; u < w.k1; ++u) {
        if (issued >= early &&
            !mbar_wait_warp(&empty[st], ph ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (issued >= early) copy_codes(w, u, st);
          copy_rows(w, u, st);
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
  } else if (warp == S::mma_warp) {
    // ------------------------------------------------------- MMA issuer --
    const uint32_t b_lo = smem_u32(ring + kCodeBytes) >> 4 | kDescLoK;
    bool ok = true;
    for (int i = 0; ok && sch.at(i, &w); ++i) {
      const uint32_t idesc = idesc_16(MOE_DTYPE_FP16, false, false, kBM, (w.n + 15) & ~15);
      for (int u = w.k0; ok && u < w.k1; ++u) {
        const bool rows_there = mbar_test(&full[st], ph);
        const int blocks = blocks_of(u);
        for (int b = 0; b < blocks; ++b) {
          // (the other two have been there for long when the operands come)
          const bool sums_free = mbar_test(&d_empty[buf], bph ^ 1u);
          if (!mbar_wait_warp(&a_full[buf], bph, abort_flag, a.status, kStatusTimeoutDense) ||
              (b == 0 && !mbar_wait_asked(rows_there, &full[st], ph, abort_flag, a.status,
                                          kStatusTimeoutDense)) ||
              !mbar_wait_asked(sums_free, &d_empty[buf], bph ^ 1u, abort_flag, a.status,
                               kStatusTimeoutDense)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            // (with the TMEM addresses known at compile time blocks took as long)
            const uint32_t d0 = tmem_base + kDCol + buf * S::d_cols, a0 = tmem_base + buf * S::a_cols;
            const uint32_t bd = b_lo + ((st * S::stage + (uint32_t)b * (S::block / 64) * S::x_box) >> 4);
#pragma unroll
            for (uint32_t q = 0; q < S::block / 16; ++q) {
              const uint32_t k = q * 16;  // in the block
              umma_ts(d0 + k / kGroup * kN, a0 + q * 8, bd + (k / 64 * S::x_box >> 4) + 2 * (q & 3),
                      idesc, k % kGroup != 0 ? 1u : 0u);
            }
            umma_commit(&done[buf]);
            if (b + 1 == blocks) umma_commit(&empty[st]);
          }
          if (++buf == S::bufs) {
            buf = 0;
            bph ^= 1u;
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
  } else if (warp >= S::add_warps) {
    // ---------------------------------------------------------- unpackers --
    // 32 rows to a warp; each set takes its share of a block's columns
    const Unpack unpack;
    const int quad = warp & 3, set = (warp - S::add_warps) >> 2;
    const int r = quad * 32 + lane;
    constexpr int kChunks = S::block / 32 / S::sets;  // of 32 columns, for a set
    const uint32_t to = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)set * (S::a_cols / S::sets);
    bool ok = true, codes_there = mbar_test(&full[st], ph), free = mbar_test(&done[buf], bph ^ 1u);
    for (int i = 0; ok && sch.at(i, &w); ++i) {
      for (int u = w.k0; ok && u < w.k1; ++u) {
        if (!mbar_wait_asked(codes_there, &full[st], ph, abort_flag, a.status, kStatusTimeoutDense)) {
          ok = false;
          break;
        }
        const uint8_t *row = ring + st * S::stage + r * 128;
        uint4 v[S::blocks][kChunks];
#pragma unroll
        for (int b = 0; b < S::blocks; ++b)
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            v[b][c] = *reinterpret_cast<const uint4 *>(
                row + ((((b * S::sets + set) * kChunks + c) ^ (r & 7)) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == (uint32_t)kStages) {
          st = 0;
          ph ^= 1u;
        }
        codes_there = mbar_test(&full[st], ph);
        const int blocks = blocks_of(u);
#pragma unroll
        for (int b = 0; b < S::blocks; ++b) {
          if (b < blocks) {
            // (the operands before these are multiplied)
            if (!mbar_wait_asked(free, &done[buf], bph ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              uint32_t o[16];
              unpack(v[b][c].x, o);
              unpack(v[b][c].y, o + 4);
              unpack(v[b][c].z, o + 8);
              unpack(v[b][c].w, o + 12);
              tmem_st16(to + buf * S::a_cols + (uint32_t)c * 16, o);
            }
            const uint32_t mine = buf;
            if (++buf == S::bufs) {
              buf = 0;
              bph ^= 1u;
            }
            free = mbar_test(&done[buf], bph ^ 1u);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a_full[mine]);
          }
        }
      }
    }
  } else {
    // ------------------------------------------- scaling, adding, epilogue --
    pdl_wait();
    // warps w and w + 4 share 32 TMEM lanes, each half of the rows of x
    constexpr int kHalf = kN / 2;
    const int quad = warp & 3, half = (warp >> 2) * kHalf;
    const uint32_t from = tmem_base + ((uint32_t)(quad * 32) << 16) + kDCol + half;
    bool ok = true;
    // A row's scales, two units ahead, of even and of odd units: what is done with a register
    // that a load is still to fill waits for it, a move included.
    UnitScales<kGroup, kUnit> even, odd;
    Work w_ask = {};
    int i_ask = 0, u_ask = 0;
    bool is_odd = false;
    const uint16_t *scale_row = nullptr;
    auto aim = [&]() {
      u_ask = sch.at(i_ask, &w_ask) ? w_ask.k0 : -1;
      scale_row = a.scale + ((int64_t)w_ask.e * a.N + min(w_ask.a0 + quad * 32 + lane, a.N - 1)) * a.groups;
    };
    auto ask = [&](UnitScales<kGroup, kUnit> &s) {
      if (u_ask < 0) return;
      s.load(scale_row, u_ask, a.groups);
      if (++u_ask == w_ask.k1) {
        ++i_ask;
        aim();
      }
    };
    aim();
    ask(even);
    ask(odd);
    for (int i = 0; sch.at(i, &w); ++i) {
      float acc[kHalf];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
      // asked for now, used at the tile's end: lane j's is that of row j
      const float factor =
          lane < kHalf && half + lane < w.n ? a.factor[w.b0 - a.first + half + lane] : 1.f;
      for (int u = w.k0; ok && u < w.k1; ++u) {
        float scales[kUnit / kGroup];
        auto take = [&](UnitScales<kGroup, kUnit> &s) {
#pragma unroll
          for (int g = 0; g < kUnit / kGroup; ++g) scales[g] = scale_half(a.dtype, s.w[g / 2], g & 1);
          ask(s);
        };
        if (is_odd)
          take(odd);
        else
          take(even);
        is_odd = !is_odd;
        const int blocks = blocks_of(u);
#pragma unroll
        for (int b = 0; b < S::blocks; ++b) {
          if (b < blocks) {
            ok = mbar_wait_warp(&done[buf], bph, abort_flag, a.status, kStatusTimeoutDense);
            if (!ok) break;
            tc_fence_after();
            // up to 32 columns on their way at a time: of several groups, or of one
            constexpr int kLoad = kHalf < 16 ? 8 : 16;
            static_assert(kHalf % kLoad == 0, "columns of a load");
            constexpr int kLoads = S::groups * (kHalf / kLoad);  // of a block
            constexpr int kOnce = kLoads < 32 / kLoad ? kLoads : 32 / kLoad;
#pragma unroll
            for (int l0 = 0; l0 < kLoads; l0 += kOnce) {
              uint32_t v[kOnce * kLoad];
#pragma unroll
              for (int l = 0; l < kOnce; ++l)
                tmem_ld_cols<kLoad>(from + buf * S::d_cols + (uint32_t)((l0 + l) / (kHalf / kLoad) * kN +
                                                                        (l0 + l) % (kHalf / kLoad) * kLoad),
                                    v + l * kLoad);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < kOnce * kLoad; ++k) asm volatile("" : "+r"(v[k]));  // not before
#pragma unroll
              for (int l = 0; l < kOnce; ++l) {
                const int g = b * S::groups + (l0 + l) / (kHalf / kLoad);
                const int c = (l0 + l) % (kHalf / kLoad) * kLoad;
#pragma unroll
                for (int j = 0; j < kLoad; ++j)
                  acc[c + j] = fmaf(scales[g], __uint_as_float(v[l * kLoad + j]), acc[c + j]);
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[buf]);
            if (++buf == S::bufs) {
              buf = 0;
              bph ^= 1u;
            }
          }
        }
      }
      // warps meet at a split tile: all of them leave there, or none
      if (i < sch.pieces) ok = add_all<S::add_warps * 32>(ok && !*abort_flag);
      if (!ok) break;
      bool last = true;
      if (w.parts > 1) {
        auto place = [&](int part) {
          const int s = sch.slot(sch.first_worker(w.tile) + part, w.tile);
          return a.part + (size_t)s * (kBM * kN) + (size_t)half * kBM + (quad * 32 + lane) * 4;
        };
        float *mine = place(w.part);
#pragma unroll
        for (int q = 0; q < kHalf / 4; ++q)
          __stcg(reinterpret_cast<float4 *>(mine + q * (kBM * 4)),
                 make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]));
        add_all<S::add_warps * 32>(true);
        if (threadIdx.x == 0) *last_flag = arrive_last(a.counters + w.tile, w.parts);
        add_all<S::add_warps * 32>(true);
        last = *last_flag != 0;
        if (last) {
#pragma unroll
          for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
          // several loads in flight, added in order
#pragma unroll 4
          for (int part = 0; part < w.parts; ++part) {
            const float *p = place(part);
#pragma unroll
            for (int q = 0; q < kHalf / 4; ++q) {
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
#pragma unroll
      for (int j = 0; j < kHalf; ++j) acc[j] *= __shfl_sync(0xffffffffu, factor, j);
      if (last && n < a.N) {
        const bool wide = a.out_dtype == MOE_DTYPE_FP32;
        auto load = [&](const void *p, int64_t at) {
          return wide ? static_cast<const float *>(p)[at]
                      : unpack16(a.out_dtype, static_cast<const uint16_t *>(p)[at]).x;
        };
        if (a.bias != nullptr) {
          const float b = load(a.bias, n);
#pragma unroll
          for (int j = 0; j < kHalf; ++j) acc[j] += b;
        }
        if (wide)
          activate_all<true>(a.act, acc);
        else
          activate_all<false>(a.act, acc);
        if (a.residual != nullptr) {
#pragma unroll
          for (int j = 0; j < kHalf; ++j)
            if (half + j < w.n) acc[j] += load(a.residual, (int64_t)(w.b0 + half + j) * a.ldr + n);
        }
        const int64_t y0 = (int64_t)(w.b0 + half) * a.ldy + n;
        if (wide) {
          float *p = static_cast<float *>(a.y) + y0;
#pragma unroll
          for (int j = 0; j < kHalf; ++j)
            if (half + j < w.n) p[j * a.ldy] = acc[j];
        } else {
          uint16_t *p = static_cast<uint16_t *>(a.y) + y0;
#pragma unroll
          for (int j = 0; j < kHalf; ++j)
            if (half + j < w.n) p[j * a.ldy] = (uint16_t)pack16(a.out_dtype, acc[j], 0.f);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == S::mma_warp) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int kGroup, int kN>
cudaError_t start(const Int4Gemm &g, cudaStream_t s) {
  auto kern = int4_tc_kernel<kGroup, kN>;
  static std::atomic<bool> allowed[64];
  cudaError_t e = allow_smem(kern, smem_bytes<kGroup, kN>(kMaxE), allowed);
  if (e != cudaSuccess) return e;
  TcArgs a = {};
  a.offsets = g.offsets;
  a.T = g.T;
  a.E = g.E;
  a.N = g.N;
  a.K = g.K;
  a.first = g.first;
  a.factor = g.factor;
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
  const int rows = std::min(g.T - g.first, kInt4Rows);
  TcMaps maps = {};
  const cuuint64_t dims[3] = {(cuuint64_t)g.K / 2, (cuuint64_t)g.N, (cuuint64_t)g.E};
  const cuuint64_t strides[2] = {(cuuint64_t)g.K / 2, (cuuint64_t)g.N * (g.K / 2)};
  const cuuint32_t box[3] = {kUnit / 2, kBM, 1};
  bool ok = encode_map(&maps.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, g.q, 3,
                       dims, strides, box);
  for (int i = 0; i < kN / 16; ++i)
    ok = ok && map_2d(&maps.x[i], MOE_DTYPE_FP16, CU_TENSOR_MAP_SWIZZLE_128B, g.xr, rows, int4_pitch(g.K),
                      int4_pitch(g.K), 16 * (i + 1), 64);
  if (!ok) return cudaErrorInvalidValue;
  // (rows of a tile are chosen by what int4_part_bytes counts on)
  if (g.part_bytes < (size_t)2 * kMaxCtas * kBM * kN * 4) return cudaErrorInvalidValue;
  const int64_t tiles = ((int64_t)std::min(g.E, rows) + rows / kN) * a.mt;
  const int64_t most = std::min<int64_t>(tiles * std::min(kMaxParts, a.units),
                                         std::min(num_sms(), kMaxCtas));
  return launch_pdl(kern, dim3((unsigned)most), dim3(Shape<kGroup, kN>::threads), smem_bytes<kGroup, kN>(g.E), s, maps,
                    a);
}

// Rows of a tile: what one pass takes.  Experts' rows vary, so that half of the most that an
// even spread gives 16 of would take two passes: 32 experts of 4096 x 7168 with 16 rows
// on average take 149 us in tiles of up to 32, 190 in tiles of 16 and 202 in tiles of 64; a
// matrix of 14336 x 4096 with 16 rows 17.8 and 16.7 us in tiles of 32 and 16.
template <int kGroup>
cudaError_t by_rows(const Int4Gemm &g, cudaStream_t s) {
  const int rows = (g.T + g.E - 1) / g.E;
  if (rows <= (g.E == 1 ? 16 : 8)) return start<kGroup, 16>(g, s);
  if (rows <= 32 || kGroup == 32) return start<kGroup, 32>(g, s);
  return start<kGroup, kGroup == 32 ? 32 : 64>(g, s);
}

}  // namespace

// Two pieces to a CTA, 128 x (rows of a tile) fp32 each; of up to 8 rows over any experts a
// tile has 16 rows, of up to 16 or of more than one expert's 32 at most.
size_t int4_part_bytes(int T) {
  const int rows = T <= 8 ? 16 : (T <= 32 ? 32 : 64);
  return (size_t)2 * kMaxCtas * kBM * rows * 4;
}

cudaError_t launch_int4_tc(const Int4Gemm &g, cudaStream_t s) {
  if (g.group == 32) return by_rows<32>(g, s);
  return g.group == 64 ? by_rows<64>(g, s) : by_rows<128>(g, s);
}

}  // namespace moe
