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
// Where there are too few tiles for the SMs, two pairs (a cluster of four) take
// the halves of K of one tile: each sends its partial sums of the other's half
// of the columns through distributed shared memory and finishes its own half.
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
//   warp 9     TMEM allocation; in the even CTA one thread issues the MMAs;
//   warp 10    E4M3 operands only: their block exponents, laid out as the
//              scale factors of block-scaled MMAs (kind::mxf8f6f4).
// Every wait is bounded; on expiry the CTA latches the status bit and leaves
// its loops, and both CTAs meet at a cluster barrier before TMEM is freed.
#include <algorithm>
#include <type_traits>

#include "dense.cuh"
#include "pair_tile.cuh"

namespace moe {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kSfWarp = kEpiWarps + 2;           // E4M3
// E4M3 leaves the last 64 TMEM columns to scale factors, four slots of four
// stages each: accumulators of 224 columns.
// The gradient of the gated product stores three tiles and turns two for each
// 32 columns: it has three output slots and a place to turn, and a stage less.
template <int kEpi, bool kE4m3>
struct Shape {
  static constexpr bool grad = kEpi == kEpiGatedGrad;
  static constexpr int threads = (kEpiWarps + 2 + (kE4m3 ? 1 : 0)) * 32;
  static constexpr int stages = kE4m3 || grad ? 5 : 6;
  static constexpr int acc = kE4m3 ? 224 : 256;  // columns of an accumulator
  static constexpr int kb = kE4m3 ? 128 : 64;    // K elements of a stage (128 bytes)
  static constexpr uint32_t sf_col = 2 * acc;
  static constexpr uint32_t out_bytes = grad ? 8192 : 4096;  // of an epilogue warp
  static constexpr int slots = grad ? 3 : 2;                 // of 32 x 32 16-bit values
};
typedef Shape<kEpiLinear, false> Shape16;
typedef Shape<kEpiLinear, true> Shape8;
static_assert(Shape8::sf_col + 4 * kSfCols <= 512, "TMEM columns");
constexpr int kMaxStages = 6;
constexpr int kSfGroup = 8;                       // stages to a hand-over of scale factors
constexpr int kSfBufs = 3;
constexpr uint32_t kSfBlock = 3 * 512;            // of four stages: A, twice B
constexpr int kTileM = 256;
constexpr int kTileN = 256;                      // the most columns of a tile
constexpr uint32_t kABytes = kBM * kBK * 2;      // 16 KB
constexpr uint32_t kBBytes = kTileN / 2 * kBK * 2;  // <= 16 KB
constexpr uint32_t kStageBytes = kABytes + kBBytes;
// Split-K: where a CTA's partial columns for the other pair leave, where the
// other pair's arrive (both in the ring's place), 16 KB for 32 columns.
constexpr uint32_t kChunkBytes = kBM * 32 * 4;
constexpr uint32_t kRecvOff = 4 * kChunkBytes;
constexpr uint32_t kTileBytes = 4096;            // 32 x 32 fp32
constexpr uint32_t kTmemCols = 512;
template <int kEpi, bool kE4m3>
constexpr size_t smem_bytes() {
  typedef Shape<kEpi, kE4m3> S;
  return 1024 + (size_t)S::stages * kStageBytes + kEpiWarps * S::out_bytes +
         (2 * kMaxStages + 6 + 2 * kSfBufs) * 8 + 16 +
         (kE4m3 ? 128 + kSfBufs * 2 * kSfBlock : 0);
}
static_assert(smem_bytes<kEpiLinear, false>() <= 232448 &&
                  smem_bytes<kEpiLinear, true>() <= 232448 &&
                  smem_bytes<kEpiGatedGrad, false>() <= 232448,
              "shared memory per CTA");
static_assert(2 * kRecvOff <= Shape8::stages * kStageBytes, "exchange buffers");
// Row tiles of a raster group: tiles that run together share the A rows of 8
// row tiles and the B rows of ~10 column tiles, ~20 MB at K = 4096: in L2.
constexpr int kGroupM = 8;

// One product of a launch.
struct Problem {
  int M, N, nkb;  // nkb: stages of K
  int mt, nt;     // row and column tiles
  int a_mn;       // (kMulti) whether A is MN-major
  int out_dtype;
  const void *residual;
  int64_t ldr;
};
struct ProblemMaps {
  CUtensorMap a, b, d;
};

// Up to three products in one launch (kMulti): a gradient's dX and dWs, which do
// not depend on each other, share one round-up to whole rounds and one tail.
// Clusters first take the tiles of product 0 in turn, then those of the others;
// the clusters that had a tile of product 0 less go on for more rounds.
template <bool kMulti>
struct PairMaps {
  ProblemMaps p[kMulti ? 3 : 1];
  CUtensorMap extra;  // preact, saved or dgu
};

template <bool kMulti>
struct PairArgs {
  Problem p[kMulti ? 3 : 1];
  int tiles0, tiles1, tiles;  // of product 0, of 1 and of 1 and 2 (kMulti)
  int shared_rounds;          // rounds of products 1 and 2 that every cluster takes
  int bn, cols;  // accumulator columns of a tile; output columns of a tile
  int split;     // pairs to a tile, K split between them (1 or 2)
  int kb_part;   // stages of K to a pair
  int dtype, act;
  const void *bias;
  const float *saved;
  int extra;  // kEpiLinear: store preact; kEpiGated: store saved
  const int8_t *a_scale, *b_scale;
  uint32_t *status;
};

// D (+)= (A * 2^sfa) (B * 2^sfb)^T over the pair, 32 of K.  Each CTA's TMEM
// holds the scale factors of its own rows of A and of all columns.
__device__ __forceinline__ void umma_mxf8_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                               uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %8, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %5, [%6], [%7], p;\n\t}" ::
          "r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 32 rows of 16 bytes from shared memory (both CTAs' own) to 4 columns of TMEM,
// repeated in the four groups of 32 lanes; in order with the MMAs that follow.
__device__ __forceinline__ void sf_copy_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}
// Its source: no swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sf(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
struct Tile {
  int p, m0, j;  // product, first row, column tile
};
__device__ __forceinline__ Tile tile_at(const Problem &q, int p, int tile) {
  const int per = kGroupM * q.nt;
  const int g = tile / per, r = tile - g * per;
  const int gm = min(kGroupM, q.mt - g * kGroupM);
  Tile t;
  t.p = p;
  t.j = r / gm;
  t.m0 = (g * kGroupM + r - t.j * gm) * kTileM;
  return t;
}
// Cluster c's i-th tile, of n clusters; false past its last.
template <bool kMulti>
__device__ __forceinline__ bool work_at(const PairArgs<kMulti> &a, int i, int c, int n, Tile *t) {
  int k = i * n + c;
  if (k < a.tiles0) {
    *t = tile_at(a.p[0], 0, k);
    return true;
  }
  if (!kMulti) return false;
  const int more = a.tiles0 % n;  // clusters with one tile of product 0 more
  const int j = i - a.tiles0 / n - (c < more ? 1 : 0);
  if (j < a.shared_rounds)
    k = j * n + c;
  else if (c >= more)
    k = a.shared_rounds * n + (j - a.shared_rounds) * (n - more) + c - more;
  else
    return false;
  if (k >= a.tiles) return false;
  *t = k < a.tiles1 ? tile_at(a.p[1], 1, k) : tile_at(a.p[kMulti ? 2 : 0], 2, k - a.tiles1);
  return true;
}

// 16 of the values, the first or the second half.
__device__ __forceinline__ void add16(float (&f)[16], const uint8_t *slot, int half, int lane) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 v = *reinterpret_cast<const float4 *>(slot + lane * 128 +
                                                       (((4 * half + c) ^ (lane & 7)) << 4));
    f[4 * c] += v.x;
    f[4 * c + 1] += v.y;
    f[4 * c + 2] += v.z;
    f[4 * c + 3] += v.w;
  }
}
// The bias of a tile's 256 columns, 8 to a lane; loaded a tile ahead.
struct TileBias {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void *p, int c, int N, int dtype, int lane) {
    c += lane * 8;
    if (c >= N) return;
    if (dtype == MOE_DTYPE_FP32) {
      const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + c);
      lo = __ldg(q);
      hi = __ldg(q + 1);
    } else {
      lo = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + c));
    }
  }
  // f[i] += the bias of column 32 `chunk` + i
  __device__ __forceinline__ void add_to(float (&f)[32], int chunk, int dtype) const {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const int from = chunk * 4 + l;
      if (dtype == MOE_DTYPE_FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[8 * l + i] += __uint_as_float(__shfl_sync(0xffffffffu, w[i], from));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = unpack16(dtype, __shfl_sync(0xffffffffu, w[i], from));
          f[8 * l + 2 * i] += u.x;
          f[8 * l + 2 * i + 1] += u.y;
        }
      }
    }
  }
};

// 32 rows of 16 fp32 values, loaded four lanes to a row (whole sectors; a lane to
// a row fetched them twice) and turned by way of shared memory so that lane r has
// row r.  Rows and columns past the ends are zero.
struct Tile16 {
  float4 v[4];
  __device__ __forceinline__ void load(const float *p, int64_t ld, int rows, int cols, int lane) {
    const int r = lane >> 2, c = (lane & 3) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = 8 * i + r < rows && c < cols
                 ? __ldg(reinterpret_cast<const float4 *>(p + (int64_t)(8 * i + r) * ld + c))
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void turn(uint8_t *to, int lane, float (&f)[16]) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4 *>(to + (8 * i + r) * 64 + ((c ^ ((r >> 1) & 3)) << 4)) = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 o =
          *reinterpret_cast<const float4 *>(to + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4));
      f[4 * i] = o.x;
      f[4 * i + 1] = o.y;
      f[4 * i + 2] = o.z;
      f[4 * i + 3] = o.w;
    }
    __syncwarp();
  }
};

// kExact: activations for fp32 results.  Kernels of their own: their code beside that
// of 16-bit results made the latter's epilogues 14% longer (2048 x 8192 x 1024 with
// SiLU 28.5 -> 32.6 us).
template <int kEpi, bool kAMn, bool kBMn, bool kE4m3, bool kMulti, bool kExact>
__global__ void __launch_bounds__(Shape<kEpi, kE4m3>::threads, 1)
    dense_pair_kernel(const __grid_constant__ PairMaps<kMulti> maps,
                      const __grid_constant__ PairArgs<kMulti> a) {
  typedef Shape<kEpi, kE4m3> S;
  constexpr int kStages = S::stages, kKb = S::kb;
  constexpr uint32_t kAcc = S::acc;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *ring = smem;
  uint8_t *slots = ring + kStages * kStageBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(slots + kEpiWarps * S::out_bytes);
  uint64_t *empty = full + kMaxStages;
  uint64_t *tfull = empty + kMaxStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *fin = tempty + 2;
  uint64_t *recv = fin + 1;
  uint64_t *sf_full = recv + 1;
  uint64_t *sf_empty = sf_full + kSfBufs;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sf_empty + kSfBufs);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  // E4M3: [kSfBufs][2][kSfBlock], 128-byte aligned
  uint8_t *sf_blocks = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(tmem_slot + 2) + 127) & ~static_cast<uintptr_t>(127));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank();
  const uint32_t rank = crank & 1u;  // in the pair; the even CTA issues the MMAs
  const uint32_t lead = crank & ~1u;
  const uint16_t pair_mask = (uint16_t)(3u << lead);
  const int kpart = (int)(crank >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);  // of both CTAs
    }
    for (int g = 0; g < kSfBufs; ++g) {
      mbar_init(&sf_full[g], 2);  // a warp of each CTA
      mbar_init(&sf_empty[g], 1);
    }
    mbar_init(fin, 1);
    mbar_init(recv, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&maps.p[0].a);
    tma_prefetch_desc(&maps.p[0].b);
    tma_prefetch_desc(&maps.p[0].d);
  }
  pdl_wait();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // this pair's stages of K (kMulti: all of each product's)
  const int k_first = min(a.p[0].nkb, kpart * a.kb_part);
  const int k_last = min(a.p[0].nkb, k_first + a.kb_part);
  auto stages_of = [&](int p) { return kMulti ? a.p[p].nkb : k_last - k_first; };
  const int half = a.bn >> 1;
  const int cid = blockIdx.x / (2 * a.split), ncl = gridDim.x / (2 * a.split);

  if (warp == kTmaWarp) {
    // ------------------------------------------------------ TMA producer --
    {
      const int b_boxes = (half + 63) >> 6;
      const uint32_t bytes =
          kABytes + (kBMn ? (uint32_t)b_boxes * 8192u : (uint32_t)half * 128u);
      const uint32_t full0 = cluster_addr(full, lead);
      uint32_t st = 0, ph = 0, issued = 0;
      uint8_t *da = ring;
      bool ok = true;
      Tile t;
      // the stages of a tile, A's majorness known at compile time
      auto fill = [&](auto a_mn, const CUtensorMap *ma, const CUtensorMap *mb, int m, int n,
                      int k_end) -> bool {
        for (int kb = k_first; kb < k_end; ++kb) {
          if (!mbar_wait_warp(&empty[st], ph ^ 1u, abort_flag, a.status, kStatusTimeoutDense))
            return false;
          const uint32_t bar = full0 + st * 8;
          if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * bytes);
          uint8_t *db = da + kABytes;
          const int k = kb * kKb;
          if (a_mn.value) {
            tma_load_2d_pair(da, ma, bar, m, k);
            tma_load_2d_pair(da + 8192, ma, bar, m + 64, k);
          } else {
            tma_load_2d_pair(da, ma, bar, k, m);
          }
          if (kEpi == kEpiGated) {
            // the even CTA holds the gate columns' rows, the odd CTA the up columns'
            tma_load_3d_pair(db, mb, bar, k, n, (int)rank);
          } else if (kBMn) {
            for (int i = 0; i < b_boxes; ++i)
              tma_load_2d_pair(db + i * 8192, mb, bar, n + 64 * i, k);
          } else {
            tma_load_2d_pair(db, mb, bar, k, n);
          }
          }
          ++issued;
          da += kStageBytes;
          if (++st == (uint32_t)kStages) {
            st = 0;
            ph ^= 1u;
            da = ring;
          }
        }
        return true;
      };
      for (int i = 0; ok && work_at(a, i, cid, ncl, &t); ++i) {
        const ProblemMaps *map = &maps.p[t.p];
        const int m = t.m0 + (int)rank * kBM;
        const int n = kEpi == kEpiGated ? t.j * a.cols : t.j * a.cols + (int)rank * half;
        const int k_end = k_first + stages_of(t.p);
        if (!kMulti || a.p[t.p].a_mn == (kAMn ? 1 : 0))
          ok = fill(std::integral_constant<bool, kAMn>(), &map->a, &map->b, m, n, k_end);
        else
          ok = fill(std::integral_constant<bool, !kAMn>(), &map->a, &map->b, m, n, k_end);
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
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------- MMA issuer --
    if (rank == 0) {
      constexpr uint32_t kBStep = kBMn ? 128 : 2;  // 16 of K, in 16 bytes
      // operand descriptors: the high words do not change, the low ones hold the
      // address in 16-byte units
      constexpr uint32_t kAHi = kAMn ? kDescHiMn : kDescHiK, kBHi = kBMn ? kDescHiMn : kDescHiK;
      static_assert(kDescHiMn == kDescHiK, "one high word for either A (kMulti)");
      const uint32_t b0 = smem_u32(ring + kABytes) >> 4 | (kBMn ? kDescLoMn : kDescLoK);
      uint32_t off = 0;
      uint32_t st = 0, ph = 0, tl = 0;
      // E4M3: scale factors go to TMEM in blocks of four stages, each block
      // while the products of the one before it run
      const int per_tile = (k_last - k_first + 3) / 4;
      int blocks = cid < a.tiles0 ? (a.tiles0 - cid + ncl - 1) / ncl * per_tile : 0, in_tile = 0;
      uint32_t sg = 0, sph = 0, filled = 0, used = 0;  // hand-over buffer; TMEM slots
      auto copy_block = [&]() -> bool {
        if (blocks == 0) return true;
        const uint32_t part = (uint32_t)in_tile % (kSfGroup / 4);
        if (part == 0 && !mbar_wait_warp(&sf_full[sg], sph, abort_flag, a.status, kStatusTimeoutDense))
          return false;
        tc_fence_after();
        const uint32_t to = tmem_base + Shape8::sf_col + (filled++ & 3u) * kSfCols;
        const uint64_t sd = sdesc_sf(smem_u32(sf_blocks + (sg * 2 + part) * kSfBlock));
        if (elect_one()) {
#pragma unroll
          for (uint32_t i = 0; i < 3; ++i) sf_copy_pair(to + 4 * i, sd + i * (512 >> 4));
        }
        --blocks;
        if (++in_tile == per_tile) in_tile = 0;
        if (part == kSfGroup / 4 - 1 || in_tile == 0) {
          if (elect_one()) umma_commit_pair(&sf_empty[sg], pair_mask);
          if (++sg == kSfBufs) {
            sg = 0;
            sph ^= 1u;
          }
        }
        return true;
      };
      bool ok = !kE4m3 || copy_block();
      Tile t;
      auto multiply = [&](auto a_mn, uint32_t d0, int k_count) -> bool {
        constexpr bool kMn = decltype(a_mn)::value;
        constexpr uint32_t kAStep = kMn ? 128 : 2;
        const uint32_t a0 = smem_u32(ring) >> 4 | (kMn ? kDescLoMn : kDescLoK);
        const uint32_t idesc = kE4m3 ? idesc_mxf8(2 * kBM, a.bn)
                                     : idesc_16(a.dtype, kMn, kBMn, 2 * kBM, a.bn);
        for (int ki = 0; ki < k_count; ++ki) {
          if (!mbar_wait_warp(&full[st], ph, abort_flag, a.status, kStatusTimeoutDense)) return false;
          uint32_t sf = 0, id = idesc;
          if (kE4m3) {
            if (ki % 4 == 0) ++used;
            sf = tmem_base + Shape8::sf_col + ((used - 1) & 3u) * kSfCols;
            id |= idesc_sf_byte((uint32_t)ki & 3u);
          }
          tc_fence_after();
          const uint32_t ad = a0 + off, bd = b0 + off;
          if (elect_one()) {
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
              const uint32_t acc = ((uint32_t)ki | q) != 0 ? 1u : 0u;
              if (kE4m3) {
                umma_mxf8_pair(d0, ad + 2 * q, kAHi, bd + 2 * q, kBHi, id, sf, sf + 4, acc);
              } else {
                umma_16_pair(d0, ad + q * kAStep, kAHi, bd + q * kBStep, kBHi, idesc, acc);
              }
            }
            umma_commit_pair(&empty[st], pair_mask);
          }
          if (kE4m3 && ki % 4 == 0 && !copy_block()) return false;
          off += kStageBytes >> 4;
          if (++st == (uint32_t)kStages) {
            st = 0;
            ph ^= 1u;
            off = 0;
          }
        }
        return true;
      };
      for (int i = 0; ok && work_at(a, i, cid, ncl, &t); ++i, ++tl) {
        const uint32_t buf = tl & 1u, use = tl >> 1;
        if (!mbar_wait_warp(&tempty[buf], (use & 1u) ^ 1u, abort_flag, a.status, kStatusTimeoutDense)) break;
        tc_fence_after();
        const uint32_t d0 = tmem_base + buf * kAcc;
        if (!kMulti || a.p[t.p].a_mn == (kAMn ? 1 : 0))
          ok = multiply(std::integral_constant<bool, kAMn>(), d0, stages_of(t.p));
        else
          ok = multiply(std::integral_constant<bool, !kAMn>(), d0, stages_of(t.p));
        if (!ok) break;
        if (elect_one()) umma_commit_pair(&tfull[buf], pair_mask);
      }
      if (elect_one()) umma_commit_pair(fin, (uint16_t)(1u << lead));
      __syncwarp();
      mbar_wait_drain(fin, 0);
    }
    __syncwarp();
  } else if (kE4m3 && warp == kSfWarp) {
    // ------------------------------------------------- scale factors --
    // A word of TMEM's scale factors holds four bytes: here those of four
    // successive 128-deep stages, chosen by the byte index in the MMA's
    // descriptor.  Lane l's word j of A's 512-byte block is row 32 j + l, word
    // j of B's block i column 128 i + 32 j + l (32 columns lie in one 128-row
    // block of W).  The MMA thread copies the blocks to TMEM in the order of its
    // products.  One hand-over for eight stages: it takes a release at cluster
    // scope, which measured 0.85 us (a stage takes 0.32).
    // Loads run one hand-over ahead.
    const int last = (a.p[0].N - 1) >> 7, nkb = a.p[0].nkb, total = a.tiles0;
    uint32_t nx[2][4], nw[2];
    auto load = [&](int tile, int kb) {
      const Tile t = tile_at(a.p[0], 0, tile);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = min(t.m0 + (int)rank * kBM + 32 * j + lane, a.p[0].M - 1);
        const int8_t *e = a.a_scale + (int64_t)r * nkb + kb;
        nx[0][j] = e8m0_4(e, nkb - kb);
        nx[1][j] = e8m0_4(e + 4, nkb - kb - 4);
      }
      // lane j: the words of 32 columns
      const int blk = min((t.j * a.cols + 32 * (lane & 7)) >> 7, last);
      const int8_t *e = a.b_scale + (int64_t)blk * nkb + kb;
      nw[0] = e8m0_4(e, nkb - kb);
      nw[1] = e8m0_4(e + 4, nkb - kb - 4);
    };
    uint32_t g = 0, ph = 0;
    int tile = cid, kb = k_first;
    if (tile < total) load(tile, kb);
    while (tile < total) {
      uint32_t x[2][4], w[2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = nx[i][j];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = __shfl_sync(0xffffffffu, nw[i], j);
      }
      kb += kSfGroup;
      if (kb >= k_last) {
        kb = k_first;
        tile += ncl;
      }
      if (tile < total) load(tile, kb);
      const bool free =
          mbar_wait(&sf_empty[g], ph ^ 1u, abort_flag, a.status, kStatusTimeoutDense);
      if (!__all_sync(0xffffffffu, free)) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 *to = reinterpret_cast<uint4 *>(sf_blocks + (g * 2 + i) * kSfBlock) + lane;
        to[0] = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
        to[32] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        to[64] = make_uint4(w[i][4], w[i][5], w[i][6], w[i][7]);
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&sf_full[g], lead));
      if (++g == kSfBufs) {
        g = 0;
        ph ^= 1u;
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue --
    // warps w and w + 4 share 32 TMEM lanes and take every other 32 columns
    Slots<S::slots> slot = {slots + warp * S::out_bytes, 0, false};
    uint8_t *turning = slot.base + S::slots * kSlotBytes;  // kEpiGatedGrad
    const int quad = warp & 3, turn = (warp >> 2) * 32;
    uint32_t tl = 0;
    Rows32 res;             // kEpiLinear: the residual of the next 32 columns
    Tile16 next_g, next_u;  // kEpiGatedGrad: of the next 16 columns
    auto bytes_of = [](int dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; };
    auto fetch = [&](const Problem &q, int c, int row) {
      if (kEpi == kEpiGatedGrad) {
        const float *sv = a.saved + (int64_t)(row - lane) * 2 * q.N + c;
        next_g.load(sv, 2 * (int64_t)q.N, q.M - (row - lane), q.N - c, lane);
        next_u.load(sv + q.N, 2 * (int64_t)q.N, q.M - (row - lane), q.N - c, lane);
      }
      if (kEpi == kEpiLinear && q.residual != nullptr)
        res.load(static_cast<const char *>(q.residual) +
                     ((int64_t)(row - lane) * q.ldr + c) * bytes_of(q.out_dtype),
                 q.ldr, q.M - (row - lane), q.N - c, q.out_dtype, lane);
    };
    TileBias bias = {}, next_bias = {};
    auto ahead = [&](const Tile &t) {
      if (kEpi == kEpiLinear && !kMulti && a.bias != nullptr)
        next_bias.load(a.bias, t.j * a.cols, a.p[0].N, a.p[0].out_dtype, lane);
    };
    Tile t, t_next;
    bool more = work_at(a, 0, cid, ncl, &t_next);
    if (more) ahead(t_next);
    for (int i = 0; more; ++tl) {
      t = t_next;
      const Problem &q = a.p[t.p];
      const ProblemMaps &map = maps.p[t.p];
      const uint32_t buf = tl & 1u, use = tl >> 1;
      bias = next_bias;
      more = work_at(a, ++i, cid, ncl, &t_next);
      if (more) ahead(t_next);
      const int row0 = t.m0 + (int)rank * kBM + quad * 32, row = row0 + lane;
      const int c0 = t.j * a.cols;
      int cfirst = c0, cend = c0 + a.cols;  // the columns this CTA finishes
      // of a cluster's only tile the first pair finishes the first half of the
      // columns, the second the rest
      const int mid = c0 + (a.cols / 32 + 1) / 2 * 32;
      if (a.split == 2 && kpart == 0) cend = mid;
      if (a.split == 2 && kpart == 1) cfirst = mid;
      fetch(q, cfirst + turn, row);
      bool ok = mbar_wait(&tfull[buf], use & 1u, abort_flag, a.status, kStatusTimeoutDense);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && a.split == 1) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(quad * 32) << 16) + buf * kAcc;
      if (a.split == 2) {
        // The others' partial sums go to the same CTA of the other pair, in
        // 32-column chunks (gated: g's chunk, then u's).
        const int ofirst = kpart == 0 ? mid : c0, oend = kpart == 0 ? c0 + a.cols : mid;
        constexpr int kPer = kEpi == kEpiGated ? 2 : 1;
        if (warp == 0 && lane == 0)
          mbar_arrive_expect_tx(recv, (uint32_t)((cend - cfirst) / 32 * kPer) * kChunkBytes);
        __syncwarp();
        cluster_arrive();  // this CTA's ring is done
        if (ok)
          for (int c = ofirst + turn; c < oend; c += 64) {
            uint8_t *p = ring + (uint32_t)((c - ofirst) / 32 * kPer) * kChunkBytes + quad * kTileBytes;
            float v[32];
            tmem_ld32(tb + (c - c0), v);
            put32(p, lane, v);
            if (kEpi == kEpiGated) {
              tmem_ld32(tb + half + (c - c0), v);
              put32(p + kChunkBytes, lane, v);
            }
          }
        fence_proxy_async_shared();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        cluster_wait();  // every ring is done
        if (ok && warp == 0 && lane == 0)
          bulk_send(cluster_addr(ring + kRecvOff, crank ^ 2u), ring,
                    (uint32_t)((oend - ofirst) / 32 * kPer) * kChunkBytes,
                    cluster_addr(recv, crank ^ 2u));
        __syncwarp();
        ok = mbar_wait(recv, 0, abort_flag, a.status, kStatusTimeoutDense) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      const uint8_t *others = ring + kRecvOff + quad * kTileBytes;
      const int cstart = cfirst;
      cend = row0 < q.M ? min(q.N, cend) : cfirst;
      for (int c = cfirst + turn; c < cend; c += 64) {
        float v[32];
        if (kEpi == kEpiLinear) {
          const Rows32 mine = res;
          if (q.residual != nullptr && c + 64 < cend) fetch(q, c + 64, row);
          tmem_ld32(tb + (c - c0), v);
          if (a.split == 2) add32(v, others + (uint32_t)((c - cstart) / 32) * kChunkBytes, lane);
          if (a.bias != nullptr) bias.add_to(v, (c - c0) / 32, q.out_dtype);
          if (a.extra) {
            uint8_t *p = slot.take32(lane);
            put32(p, lane, v);
            send_2d(&maps.extra, p, lane, c, row0);
          }
          activate_all<kExact>(a.act, v);
          const bool wide = q.out_dtype == MOE_DTYPE_FP32;
          uint8_t *p = wide ? slot.take32(lane) : slot.take16(lane);
          if (q.residual != nullptr) mine.add_to(v, p, q.out_dtype, lane);
          if (wide)
            put32(p, lane, v);
          else
            put16(p, lane, q.out_dtype, v);
          send_2d(&map.d, p, lane, c, row0);
        } else if (kEpi == kEpiGated) {
          float u[32];
          tmem_ld32(tb + (c - c0), v);
          tmem_ld32(tb + half + (c - c0), u);
          if (a.split == 2) {
            const uint8_t *o = others + (uint32_t)((c - cstart) / 32 * 2) * kChunkBytes;
            add32(v, o, lane);
            add32(u, o + kChunkBytes, lane);
          }
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
          send_2d(&map.d, p, lane, c, row0);
        } else {
          // dh = acc;  s = sigmoid(g):  h = g s u, dg = dh u s (1 + g (1 - s)), du = dh g s.
          // All three in 16 bits: they are the next products' operands, and keeping
          // more bits would take each product twice (high and low parts).  bf16
          // gradients end 0.0023 to 0.0025 off in the 2-norm, with the rounding of
          // the result alone 0.0016 to 0.0017.
          uint32_t wh[16], wg[16], wu[16];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float g[16], u[16], dh[16];
            next_g.turn(turning, lane, g);
            next_u.turn(turning, lane, u);
            if (hf == 0)
              fetch(q, c + 16, row);
            else if (c + 64 < cend)
              fetch(q, c + 64, row);
            tmem_ld16f(tb + (c - c0) + 16 * hf, dh);
            if (a.split == 2)
              add16(dh, others + (uint32_t)((c - cstart) / 32) * kChunkBytes, hf, lane);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float h[2], dg[2], du[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float s = sigmoid(g[i + k]), gs = g[i + k] * s;
                h[k] = gs * u[i + k];
                dg[k] = dh[i + k] * u[i + k] * s * (1.0f + g[i + k] * (1.0f - s));
                du[k] = dh[i + k] * gs;
              }
              wh[8 * hf + i / 2] = pack16(a.dtype, h[0], h[1]);
              wg[8 * hf + i / 2] = pack16(a.dtype, dg[0], dg[1]);
              wu[8 * hf + i / 2] = pack16(a.dtype, du[0], du[1]);
            }
          }
          uint8_t *p = slot.take16(lane);
          put16(p, lane, wh);
          send_2d(&map.d, p, lane, c, row0);
          p = slot.take16(lane);
          put16(p, lane, wg);
          send_3d(&maps.extra, p, lane, c, row0, 0);
          p = slot.take16(lane);
          put16(p, lane, wu);
          send_3d(&maps.extra, p, lane, c, row0, 1);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_relaxed(cluster_addr(&tempty[buf], lead));
    }
    // the slots outlive the copies that read them
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  if (a.split == 2 && warp >= kEpiWarps) {
    cluster_arrive();
    cluster_wait();
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

// How a product is laid out over the clusters, and about how long it takes (us).
struct PairPlan {
  int bn, cols, mt, nt, split, kb_part;
  int clusters;
  float us;
};

// Time of one stage (64 of K, E4M3 128) of a tile of bn columns.
float stage_us(bool e4m3, int bn) {
  return e4m3 ? 0.28f + 0.00035f * (float)bn : std::max(0.18f, 0.12f + 0.00062f * (float)bn);
}

// The plan with the least estimated time.  Fitted to the kernel on one GB300
// over 32 to 2048 rows, N of 1024 to 8192, K of 1024 to 14336: a stage takes
// 0.18 us up to 96 columns and 0.28 at 256 (E4M3: 0.30 at 64 and 0.36 at 224), a
// launch with its first copies and its last epilogue 5.8 us and 0.013 for each
// column, and half of the time that HBM needs for W is not hidden; a cluster's
// tiles are at least 0.45 us and 0.0085 for each column apart (their epilogues:
// 4096 x 4096 x 64 19.3 us in 64 columns, 13.8 in 256).  Splitting K in two costs
// 1.2 us (E4M3: 3.5) and halves a single round's stages: 4096 x 14336 at 512 rows
// 53.3 -> 42.4 us.
//
// Tried on the same shapes and slower or the same: two pairs of a cluster that
// share B by multicast (1024 x 4096 x 4096 26.9 us against 25.0: what an SM takes
// in limits, not L2), eight stages of 24 KB for narrow tiles, 12 or 16 epilogue
// warps, the residual two chunks ahead in registers.
PairPlan plan_pair(const DenseGemm &g, const int (&resident)[2]) {
  const bool e4m3 = g.dtype == MOE_DTYPE_E4M3, gated = g.epi == kEpiGated;
  const int kb = e4m3 ? Shape8::kb : Shape16::kb;
  const int nkb = (g.K + kb - 1) / kb;
  const float hbm = weight_us(g);
  PairPlan p = {};
  p.mt = (g.M + kTileM - 1) / kTileM;
  const int mt = p.mt;
  for (int split = 1; split <= 2; ++split) {
    // The first part in whole groups of eight stages, which E4M3's scale factors come
    // in (16 bits could split evenly: 33 stages are 24 and 9 so).
    const int part = split == 1 ? nkb : (nkb + 15) / 16 * 8;
    if (split == 2 && part >= nkb) continue;
    for (int bn = e4m3 ? Shape8::acc : Shape16::acc; bn >= 64; bn -= gated ? 64 : 32) {
      const int cols = gated ? bn / 2 : bn;
      const int nt = (g.N + cols - 1) / cols;
      const int64_t tiles = (int64_t)mt * nt;
      if (split == 2 && (tiles > resident[1] || cols < 64)) continue;  // one tile a cluster
      const int64_t rounds = (tiles + resident[split - 1] - 1) / resident[split - 1];
      const float once = e4m3 ? 5.2f + 0.01f * (float)bn : 5.8f + 0.013f * (float)bn;
      const float tile = (float)part * stage_us(e4m3, bn), drain = 0.45f + 0.0085f * (float)bn;
      const float us = once + (split == 1 ? 0.f : e4m3 ? 3.5f : 1.2f) + tile +
                       (float)(rounds - 1) * std::max(tile, drain) + 0.5f * hbm;
      if (p.us == 0.f || us < p.us) {
        p.us = us;
        p.bn = bn;
        p.cols = cols;
        p.nt = nt;
        p.split = split;
        p.kb_part = part;
        p.clusters = (int)std::min<int64_t>(resident[split - 1], tiles);
      }
    }
  }
  return p;
}

// Clusters of one and of two pairs that can run at once (per device, queried once).
template <int kEpi, bool kAMn, bool kBMn, bool kE4m3, bool kMulti, bool kExact = false>
cudaError_t resident_clusters(int (&out)[2]) {
  auto kern = dense_pair_kernel<kEpi, kAMn, kBMn, kE4m3, kMulti, kExact>;
  static std::atomic<int> resident[64][2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (resident[dev][0] == 0) {
    constexpr size_t kBytes = smem_bytes<kEpi, kE4m3>();
    static std::atomic<bool> allowed[64];
    cudaError_t e = allow_smem(kern, kBytes, allowed);
    if (e != cudaSuccess) return e;
    for (int p = 2; p >= 1; --p) {  // of one pair last: the one that says both are there
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)(2 * p);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3((unsigned)(num_sms() / (2 * p) * (2 * p)));
      cfg.blockDim = dim3(Shape<kEpi, kE4m3>::threads);
      cfg.dynamicSmemBytes = kBytes;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
      resident[dev][p - 1] = std::min(n, num_sms() / (2 * p));
    }
  }
  out[0] = resident[dev][0];
  out[1] = resident[dev][1];
  return cudaSuccess;
}

// Maps and arguments of one product in tiles of bn columns.
template <int kEpi>
bool set_problem(const DenseGemm &g, int bn, Problem *q, ProblemMaps *m) {
  const bool e4m3 = g.dtype == MOE_DTYPE_E4M3;
  const int kb = e4m3 ? Shape8::kb : Shape16::kb, half = bn / 2;
  const int cols = kEpi == kEpiGated ? half : bn;
  *q = {g.M, g.N, (g.K + kb - 1) / kb, (g.M + kTileM - 1) / kTileM, (g.N + cols - 1) / cols,
        g.a_mn ? 1 : 0, g.out_dtype, g.residual, g.ldr};
  const CUtensorMapSwizzle in = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = g.a_mn ? map_2d(&m->a, g.dtype, in, g.a, g.K, g.M, g.lda, kBK, 64)
                   : map_2d(&m->a, g.dtype, in, g.a, g.M, g.K, g.lda, kBM, kb);
  if (kEpi == kEpiGated)
    ok = ok && map_two(&m->b, g.dtype, in, g.b, g.N, g.K, g.ldb, g.ldb * g.N, half, kBK, 1);
  else
    ok = ok && (g.b_mn ? map_2d(&m->b, g.dtype, in, g.b, g.K, g.N, g.ldb, kBK, 64)
                       : map_2d(&m->b, g.dtype, in, g.b, g.N, g.K, g.ldb, half, kb));
  if (kEpi == kEpiGatedGrad)
    return ok && map_2d(&m->d, g.dtype, out_swizzle(g.dtype), g.h, g.M, g.N, g.N, 32, 32);
  return ok && map_2d(&m->d, g.out_dtype, out_swizzle(g.out_dtype), g.d, g.M, g.N, g.ldd, 32, 32);
}

template <int kEpi, bool kAMn, bool kBMn, bool kE4m3, bool kMulti, bool kExact = false>
cudaError_t start(const PairMaps<kMulti> &maps, const PairArgs<kMulti> &a, int clusters,
                  cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)(2 * a.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * a.split * clusters));
  cfg.blockDim = dim3(Shape<kEpi, kE4m3>::threads);
  cfg.dynamicSmemBytes = smem_bytes<kEpi, kE4m3>();
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, dense_pair_kernel<kEpi, kAMn, kBMn, kE4m3, kMulti, kExact>, maps,
                            a);
}

// `out` not null: only the plan.
template <int kEpi, bool kAMn, bool kBMn, bool kE4m3 = false, bool kExact = false>
cudaError_t launch(const DenseGemm &g, cudaStream_t s, DensePlan *out) {
  int resident[2];
  cudaError_t e = resident_clusters<kEpi, kAMn, kBMn, kE4m3, false, kExact>(resident);
  if (e != cudaSuccess) return e;
  const PairPlan plan = plan_pair(g, resident);
  if (out != nullptr) {
    *out = {kTileM, plan.cols, plan.split, plan.us};
    return cudaSuccess;
  }

  PairArgs<false> a = {};
  PairMaps<false> maps;
  bool ok = set_problem<kEpi>(g, plan.bn, &a.p[0], &maps.p[0]);
  a.tiles0 = a.p[0].mt * a.p[0].nt;
  a.bn = plan.bn;
  a.cols = plan.cols;
  a.split = plan.split;
  a.kb_part = plan.kb_part;
  a.dtype = g.dtype;
  a.act = g.act;
  a.bias = g.bias;
  a.saved = g.saved;
  a.a_scale = g.a_scale;
  a.b_scale = g.b_scale;
  a.status = g.status;
  maps.extra = maps.p[0].d;
  const CUtensorMapSwizzle wide = out_swizzle(MOE_DTYPE_FP32);
  if (kEpi == kEpiLinear && g.preact != nullptr) {
    a.extra = 1;
    ok = ok && map_2d(&maps.extra, MOE_DTYPE_FP32, wide, g.preact, g.M, g.N, g.N, 32, 32);
  } else if (kEpi == kEpiGated && g.saved != nullptr) {
    a.extra = 1;
    ok = ok && map_two(&maps.extra, MOE_DTYPE_FP32, wide, g.saved, g.M, g.N, 2 * (int64_t)g.N, g.N,
                       32, 32, 1);
  } else if (kEpi == kEpiGatedGrad) {
    ok = ok && map_two(&maps.extra, g.dtype, out_swizzle(g.dtype), g.dgu, g.M, g.N,
                       2 * (int64_t)g.N, g.N, 32, 32, 1);
  }
  if (!ok) return cudaErrorInvalidValue;
  return start<kEpi, kAMn, kBMn, kE4m3, false, kExact>(maps, a, plan.clusters, s);
}

cudaError_t pair_call(const DenseGemm &g, cudaStream_t s, DensePlan *out) {
  const bool exact = g.act != MOE_ACT_NONE && g.out_dtype == MOE_DTYPE_FP32;
  if (g.dtype == MOE_DTYPE_E4M3)
    return exact ? launch<kEpiLinear, false, false, true, true>(g, s, out)
                 : launch<kEpiLinear, false, false, true>(g, s, out);
  switch (g.epi) {
    case kEpiGated: return launch<kEpiGated, false, false>(g, s, out);
    case kEpiGatedGrad: return launch<kEpiGatedGrad, false, true>(g, s, out);
    default:
      if (g.a_mn) return launch<kEpiLinear, true, true>(g, s, out);
      if (g.b_mn) return launch<kEpiLinear, false, true>(g, s, out);
      return exact ? launch<kEpiLinear, false, false, false, true>(g, s, out)
                   : launch<kEpiLinear, false, false>(g, s, out);
  }
}

}  // namespace

DensePlan dense_pair_plan(const DenseGemm &g) {
  DensePlan p = {};
  return pair_call(g, nullptr, &p) == cudaSuccess ? p : DensePlan{};
}

cudaError_t launch_dense_pair(const DenseGemm &g, cudaStream_t s) {
  return pair_call(g, s, nullptr);
}

namespace {

// Tile width by plan_pair's figures, each product's tiles at their own depth; a
// tile takes 3.3 us at least (its epilogue).
struct MultiPlan {
  int bn;
  double us, cost[3];
};
MultiPlan plan_multi(const DenseGemm *g, int n, int ncl) {
  MultiPlan p = {};
  for (int w = Shape16::acc; w >= 64; w -= 32) {
    double c[3], sum = 0, most = 0;
    for (int i = 0; i < n; ++i) {
      const int64_t tiles = (int64_t)((g[i].M + kTileM - 1) / kTileM) * ((g[i].N + w - 1) / w);
      c[i] = std::max(3.3, (g[i].K + Shape16::kb - 1) / Shape16::kb * (double)stage_us(false, w));
      sum += (double)tiles * c[i];
      most = std::max(most, c[i]);
    }
    const double us = std::max(sum / ncl, most) + 0.5 * most + 0.02 * w;
    if (p.bn == 0 || us < p.us) {
      p.us = us;
      p.bn = w;
      for (int i = 0; i < n; ++i) p.cost[i] = c[i];
    }
  }
  return p;
}

}  // namespace

float dense_multi_us(const DenseGemm *g, int n) {
  if (n == 1) return dense_pair_us(g[0]);
  int resident[2];
  return resident_clusters<kEpiLinear, true, true, false, true>(resident) == cudaSuccess
             ? (float)plan_multi(g, n, resident[0]).us
             : 0.f;
}

cudaError_t launch_dense_multi(const DenseGemm *g, int n, cudaStream_t s) {
  if (n == 1) return launch_dense_pair(g[0], s);
  int resident[2];
  cudaError_t e = resident_clusters<kEpiLinear, true, true, false, true>(resident);
  if (e != cudaSuccess) return e;
  const int ncl = resident[0];
  const MultiPlan plan = plan_multi(g, n, ncl);
  const int bn = plan.bn;
  const double (&cost)[3] = plan.cost;
  PairArgs<true> a = {};
  PairMaps<true> maps;
  bool ok = true;
  for (int i = 0; i < n; ++i) ok = ok && set_problem<kEpiLinear>(g[i], bn, &a.p[i], &maps.p[i]);
  if (!ok) return cudaErrorInvalidValue;
  maps.extra = maps.p[0].d;
  if (n == 2) maps.p[2] = maps.p[1];
  a.tiles0 = a.p[0].mt * a.p[0].nt;
  a.tiles1 = a.p[1].mt * a.p[1].nt;
  a.tiles = a.tiles1 + (n == 3 ? a.p[2].mt * a.p[2].nt : 0);
  // Every cluster works for about the same time: those with a tile of product 0
  // more leave that much of the others' to the rest.
  const int more = a.tiles0 % ncl;
  const double other = cost[1];
  const double whole = ((double)a.tiles0 * cost[0] + (double)a.tiles * other) / ncl;
  const int all = (a.tiles + ncl - 1) / ncl;
  a.shared_rounds =
      more == 0 ? all
                : std::min(all, std::max(0, (int)((whole - (a.tiles0 / ncl + 1) * cost[0]) / other + 0.5)));
  a.bn = a.cols = bn;
  a.split = 1;
  a.dtype = g[0].dtype;
  a.act = MOE_ACT_NONE;
  a.status = g[0].status;
  const int used = (int)std::min<int64_t>(ncl, (int64_t)a.tiles0 + a.tiles);
  if (used < ncl) a.shared_rounds = 0;  // a tile each
  return start<kEpiLinear, true, true, false, true>(maps, a, used, s);
}

}  // namespace moe
