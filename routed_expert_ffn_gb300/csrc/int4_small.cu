// Products with 4-bit weights and few rows (decode): y = act(x W^T + bias) + residual of up to
// eight rows, or y_p = W_e x_p where experts have few rows each.
//
// Bound: HBM, which reads half a byte for each weight; next to it the instructions that
// unpack the codes, nine for a word of eight (int4.cuh).  Every weight is unpacked once
// for all rows and multiplied in the warp that loaded it, by mma.sync (16 rows of W by 16
// of depth by 8 rows of x, two clocks): a way through TMEM would only add to it
// (int4_tc.cu).  A group's sum is scaled in fp32 when it is complete: neither codes nor
// scales are rounded.
//
// Which k an operand element is does not matter as long as A and B agree.  A warp takes 16
// rows of W by chunks of 128 columns, a quad of lanes a row of W: nibbles j and j + 4 of
// a word, and x's elements j and j + 4 of the same eight, go together.  Each MMA must see
// one group alone: the lanes of a quad take words so that it does.
//
// One CTA of 16 warps on each SM.  It takes tiles of 16 kWarpRows rows of W: the warps that
// share rows split the depth by chunks and add their sums through shared memory.  Each warp
// has kAhead chunks of codes (8 KB) on their way to a ring of its own in shared memory, across
// tiles as well, the first of them before it looks at x; with loads to registers, four
// chunks ahead, 114688 x 4096 with 8 rows took 59 us instead of 53.
//
// x is taken as int4_rows.cu makes it (fp16, a power of two for each row).  Where the rows
// fit, kStaged, every CTA makes them for itself while its first codes are under way, which
// saves a launch.
//
// Experts: a pass takes up to eight of an expert's rows (as many as are staged); each CTA
// works through a stretch of all passes' tiles, which lie in the order of the experts, and stages
// rows when it comes to the next pass.
//
// Measured: 4096 x 4096 with one row 5.9 us, 14336 x 4096 with eight 14.3, 114688 x 4096 51
// (4.8 TB/s); 32 rows over 29 experts of 4096 x 1536 33.4 (2.9 TB/s: launch, offsets and first
// codes take 7, the fullest CTA's tiles a seventh more than the average's).  Scales twice as far
// ahead (groups of 64 and 32) and tiles finished one tile later, so that nobody waits for the
// slowest warp, gave nothing.
#include <algorithm>

#include "grouped.cuh"
#include "int4.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 8;  // chunks of codes under way for a warp
constexpr int kChunk = 128;
constexpr int kRows = kInt4SmallRows;
constexpr size_t kStagedBytes = 72 << 10;
constexpr uint32_t kRingBytes = kWarps * kAhead * 1024;

struct SmallArgs {
  int T, N, K;
  int tiles;
  int chunks, groups, pitch;
  int dtype, out_dtype, act;
  const uint8_t *x;  // kStaged: x itself, else the rows made
  const float *factor;
  const uint8_t *q;
  const uint16_t *scale;
  const void *bias, *residual;
  void *y;
  int64_t ldx, ldr, ldy;
  // experts: T is the most rows of a pass, `tiles` those of a matrix
  const int32_t *offsets;
  int R, E;
  uint32_t *status;
};

__device__ __forceinline__ void copy_codes(uint32_t to, const uint8_t *from) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// The first of the eight k in a chunk that word i of lane t stands for after regroup.
template <int kGroup>
__device__ __forceinline__ int k_of(int t, int i) {
  if (kGroup == 128) return 32 * t + 8 * i;
  if (kGroup == 64) {
    // words 0, 1 come from lanes 0 and 1 (group 0), 2 and 3 from lanes 2 and 3
    const int from = (t & 1) | (i & 2), w = (i & 1) | (t & 2);
    return 32 * from + 8 * w;
  }
  return 32 * i + 8 * t;  // group i, its word t
}

// Bytes of a staged row: four pieces of 64 bytes (word i of lanes 0 to 3) for each chunk,
// and 64 more, so that two rows' pieces lie in different banks.
__host__ __device__ constexpr int staged_pitch(int chunks) { return chunks * 256 + 64; }

// `rows` rows of x from row `first_row` on to shared memory as launch_int4_rows makes them, in that order; their
// factors to `factor`.  The warps share the rows evenly.
template <int kGroup>
__device__ __forceinline__ void stage_rows(const SmallArgs &a, int64_t first_row, int rows,
                                           uint8_t *to, float *factor, float *most) {
  const int per = rows == 1 ? kWarps : (rows == 2 ? kWarps / 2 : (rows <= 4 ? kWarps / 4 : kWarps / 8));
  const int warp = threadIdx.x >> 5, r = warp / per, first = warp % per * 32 + (threadIdx.x & 31);
  const bool mine = r < rows;
  const uint4 *row = reinterpret_cast<const uint4 *>(a.x + (first_row + (mine ? r : 0)) * a.ldx * 2);
  float up = 1.f;
  if (a.dtype == MOE_DTYPE_BF16) {
    float m = 0.f;
    if (mine)
#pragma unroll 4
      for (int c = first; c < a.K / 8; c += per * 32) m = fmaxf(m, finite_max_bf16(__ldg(row + c)));
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if ((threadIdx.x & 31) == 0) most[warp] = m;
    __syncthreads();
    for (int i = 0; i < per; ++i) m = fmaxf(m, most[warp / per * per + i]);
    const RowFactor f = row_factor(m);
    up = f.up;
    if (mine && first == 0) factor[r] = f.back;
  } else if (mine && first == 0) {
    factor[r] = 1.f;
  }
  if (!mine) return;
  to += r * staged_pitch(a.chunks);
#pragma unroll 4
  for (int p = first; p < a.chunks * 16; p += per * 32) {
    const int c = p >> 4, i = (p >> 2) & 3, t = p & 3;
    const int k = c * kChunk + k_of<kGroup>(t, i);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k < a.K) v = __ldg(row + k / 8);
    *reinterpret_cast<uint4 *>(to + c * 256 + i * 64 + t * 16) = row_piece(v, a.dtype, up);
  }
}

// y of the column n of W and the row `row` of x.
__device__ __forceinline__ void store(const SmallArgs &a, float v, int n, int64_t row) {
  const bool wide = a.out_dtype == MOE_DTYPE_FP32;
  auto load = [&](const void *p, int64_t at) {
    return wide ? static_cast<const float *>(p)[at]
                : unpack16(a.out_dtype, static_cast<const uint16_t *>(p)[at]).x;
  };
  if (a.bias != nullptr) v += load(a.bias, n);
  if (a.act != MOE_ACT_NONE) v = wide ? activate<true>(a.act, v) : activate<false>(a.act, v);
  if (a.residual != nullptr) v += load(a.residual, row * a.ldr + n);
  if (wide)
    static_cast<float *>(a.y)[row * a.ldy + n] = v;
  else
    static_cast<uint16_t *>(a.y)[row * a.ldy + n] = (uint16_t)pack16(a.out_dtype, v, 0.f);
}

// Sums of columns [from, from + cols) of the tile at n0, everything after them, and the
// rounding, by `threads` threads; a function of its own, as it is not worth a copy in each
// place.
template <int kWarpRows>
__device__ __noinline__ void finish(const SmallArgs &a, int n0, int64_t first_row, int rows,
                                    const float *red, const float *factors, int from, int cols,
                                    int thread, int threads) {
  constexpr int kCols = 16 * kWarpRows, kSplit = kWarps / kWarpRows;
  for (int j = thread; j < cols * rows; j += threads) {
    const int c = from + j % cols, r = j / cols, n = n0 + c;
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kSplit; ++s) v += red[(s * kRows + r) * (kCols + 1) + c];
    if (n < a.N) store(a, v * factors[r], n, first_row + r);
  }
}

// Passes over an expert's matrix: up to `most` of its rows each.
__host__ __device__ __forceinline__ int passes(int rows, int most) { return (rows + most - 1) / most; }

// kExperts: tiles of every pass of every expert in turn, a stretch of them to each CTA, which
// stages an expert's rows (kStaged) when it comes to them.
template <int kGroup, int kWarpRows, bool kStaged, bool kExperts>
__global__ void __launch_bounds__(kThreads, 1)
    int4_small_kernel(const __grid_constant__ SmallArgs a) {
  constexpr int kCols = 16 * kWarpRows, kSplit = kWarps / kWarpRows;
  __shared__ float red[2][kWarps * kRows * 17];
  __shared__ float most[kWarps], factors[kRows];
  extern __shared__ __align__(16) uint8_t dyn[];  // the warps' rings, then x (kStaged)
  uint8_t *staged = dyn + kRingBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp % kWarpRows, part = warp / kWarpRows;
  // not kStaged: the launch before this one made the rows of x, and waited for all before
  // it, so that the codes are there
  if (kStaged) pdl_wait();
  pdl_launch_dependents();
  const int32_t *seg = reinterpret_cast<const int32_t *>(staged + a.T * staged_pitch(a.chunks));
  const int32_t *first = seg + a.E + 1;
  int tile = blockIdx.x, end = a.tiles, step = gridDim.x;
  if constexpr (kExperts) {
    make_tables(a.offsets, a.E, a.R, 0, a.R, const_cast<int32_t *>(seg), const_cast<int32_t *>(first),
                a.status, [&](int m) { return passes(m, a.T) * a.tiles; });
    __syncthreads();
    const int64_t total = first[a.E];
    tile = (int)(total * blockIdx.x / gridDim.x);
    end = (int)(total * (blockIdx.x + 1) / gridDim.x);
    step = 1;
    if (tile == end) return;
  }
  // The expert of a tile, from that of one before it on, and the tile's first row of W.
  auto expert_at = [&](int tile, int e) {
    if (kExperts)
      while (first[e + 1] <= tile) ++e;
    return e;
  };
  auto n_of = [&](int tile, int e) {
    return (kExperts ? (tile - first[e]) % a.tiles : tile) * kCols;
  };
  const int e0 = kExperts ? expert_of(first, a.E, tile) : 0;

  // this warp's chunks of a tile, [c0, c0 + count)
  const int per = (a.chunks + kSplit - 1) / kSplit, c0 = part * per;
  const int count = max(0, min(per, a.chunks - c0));
  // In a chunk that K ends in, a lane past K keeps any codes: x is zero there.
  const bool skips = count > 0 && c0 + count == a.chunks && a.K - (a.chunks - 1) * kChunk <= 32 * t;

  // Codes on their way, across tiles: row g of this warp's 16 and, `down` bytes on, row g + 8.
  // A lane's 16 bytes lie in the ring where a quad's words can be read without bank conflicts.
  const uint32_t ring = smem_u32(dyn) + warp * (kAhead * 1024);
  const uint32_t put = ring + (g * 4 + (t ^ ((g >> 1) & 3))) * 16;
  int ask_tile = tile, ask_e = e0, to_ask = 0;
  uint32_t ask_slot = 0;
  const uint8_t *q = nullptr;
  int down = 0;
  auto ask = [&]() {
    if (to_ask == 0 && count > 0 && ask_tile < end) {
      ask_e = expert_at(ask_tile, ask_e);
      const int n = n_of(ask_tile, ask_e) + 16 * wr + g;
      const int n0 = min(n, a.N - 1), n1 = min(n + 8, a.N - 1);
      q = a.q + ((int64_t)ask_e * a.N + n0) * (a.K >> 1) + c0 * (kChunk / 2) + 16 * t;
      down = (n1 - n0) * (a.K >> 1);
      to_ask = count;
      ask_tile += step;
    }
    if (to_ask > 0) {
      if (to_ask > 1 || !skips) {
        copy_codes(put + ask_slot, q);
        copy_codes(put + ask_slot + 512, q + down);
      }
      q += kChunk / 2;
      --to_ask;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ask_slot = (ask_slot + 1024) & (kAhead * 1024 - 1);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) ask();

  // Scales, eight groups at a time, one such block ahead: lane l holds four of row l / 2.
  constexpr int kBlock = 8 * kGroup / kChunk;  // chunks: 8, 4 or 2
  int scale_tile = tile, scale_e = e0, scale_at = 0;  // group of the warp's range
  const int range = count > 0 ? min(count * (kChunk / kGroup), a.groups - c0 * (kChunk / kGroup)) : 0;
  const uint16_t *sc = nullptr;
  uint32_t next[4] = {};  // (as they come: whatever is done with them waits for them)
  auto ask_scales = [&]() {
    if (scale_tile >= end || range == 0) return;
    if (scale_at == 0) {
      scale_e = expert_at(scale_tile, scale_e);
      const int n = min(n_of(scale_tile, scale_e) + 16 * wr + (lane >> 1), a.N - 1);
      sc = a.scale + ((int64_t)scale_e * a.N + n) * a.groups + c0 * (kChunk / kGroup) + (lane & 1) * 4;
    }
    const int have = range - scale_at - (lane & 1) * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      next[k] = 0;
      if (k < have) next[k] = __ldg(sc + k);
    }
    sc += 8;
    scale_at += 8;
    if (scale_at >= range) {
      scale_at = 0;
      scale_tile += step;
    }
  };
  ask_scales();

  // the rows at hand: row `g` is this lane's; past the last one the sums are not used, and row 0
  // will do
  int64_t row0 = 0;
  int rows = a.T;
  if (kStaged) {
    if (!kExperts) stage_rows<kGroup>(a, 0, rows, staged, factors, most);  // (else as they come)
  } else {
    pdl_wait();
    if (threadIdx.x < a.T) factors[threadIdx.x] = a.factor[threadIdx.x];
  }
  __syncthreads();

  const Unpack unpack;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  int i = 0, e = e0, n0 = 0, staged_to = -1;
  uint32_t turn = 0, slot = 0;
  auto row_of_lane = [&]() {
    const int row = g < rows ? g : 0;
    return kStaged ? staged + row * staged_pitch(a.chunks) + t * 16 + c0 * 256
                   : a.x + ((int64_t)row * a.pitch + c0 * kChunk) * 2;
  };
  const uint8_t *x0 = row_of_lane(), *xp = x0;  // from this warp's first chunk on
  // By all threads, before a tile: its first row of W, and its rows of x.
  auto open = [&]() {
    e = expert_at(tile, e);
    n0 = n_of(tile, e);
    if (kExperts && tile >= staged_to) {
      const int pass = (tile - first[e]) / a.tiles;
      staged_to = first[e] + (pass + 1) * a.tiles;
      row0 = seg[e] + (int64_t)pass * a.T;
      rows = min(a.T, seg[e + 1] - (int)row0);
      __syncthreads();  // (everybody is done with the rows before)
      stage_rows<kGroup>(a, row0, rows, staged, factors, most);
      __syncthreads();
      x0 = row_of_lane();
    }
    xp = x0;
  };

  // The tile's sums: of this warp alone, or of all that share its rows.
  auto close = [&]() {
    float *to = red[turn] + part * kRows * (kCols + 1) + 16 * wr;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      to[(2 * t + (k & 1)) * (kCols + 1) + g + 8 * (k >> 1)] = sum[k];
      sum[k] = 0.f;
    }
    if (kSplit == 1) {
      __syncwarp();
      finish<kWarpRows>(a, n0, row0, rows, red[turn], factors, 16 * wr, 16, lane, 32);
    } else {
      __syncthreads();
      finish<kWarpRows>(a, n0, row0, rows, red[turn], factors, 0, kCols, threadIdx.x, kThreads);
    }
    turn ^= 1u;  // the other buffer was read before everybody arrived here
    tile += step;
  };

  if (count == 0) {
    while (tile < end) {
      open();
      close();
    }
    return;
  }
  while (tile < end) {
    if (i == 0) open();
    float scales[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) scales[k] = unpack16(a.dtype, next[k]).x;
    ask_scales();
    const int have = count - i;  // chunks of the tile from here on
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      if (j < have) {
        uint4 xv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          xv[k] = kStaged ? *reinterpret_cast<const uint4 *>(xp + k * 64)
                          : __ldg(reinterpret_cast<const uint4 *>(xp + k_of<kGroup>(t, k) * 2));
        xp += 256;
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        __syncwarp();
        uint32_t c[2][4];
        const uint8_t *codes = dyn + warp * (kAhead * 1024) + slot;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *row = codes + h * 512 + g * 64;
          const int turned = (g >> 1) & 3;
          if constexpr (kGroup == 128) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row + ((t ^ turned) << 4));
            c[h][0] = v.x;
            c[h][1] = v.y;
            c[h][2] = v.z;
            c[h][3] = v.w;
          } else if constexpr (kGroup == 64) {
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const uint2 v = *reinterpret_cast<const uint2 *>(
                  row + ((((t & 1) | k) ^ turned) << 4) + (t & 2) * 4);
              c[h][k] = v.x;
              c[h][k + 1] = v.y;
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              c[h][k] = *reinterpret_cast<const uint32_t *>(row + ((k ^ turned) << 4) + t * 4);
          }
        }
        slot = (slot + 1024) & (kAhead * 1024 - 1);
        // (eight products of one chain after the other would be waited for)
        constexpr int kChains = kGroup == 128 ? 2 : 1;
        constexpr int kWords = kGroup / 32;  // words to a group
        float group_sum[kChains][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t p0[4], p1[4];
          unpack(c[0][k], p0);
          unpack(c[1][k], p1);
          if (k % kWords == 0) {
            mma_first(group_sum[0], p0[0], p1[0], p0[1], p1[1], xv[k].x, xv[k].y);
            if (kChains == 2)
              mma_first(group_sum[kChains - 1], p0[2], p1[2], p0[3], p1[3], xv[k].z, xv[k].w);
            else
              mma(group_sum[0], p0[2], p1[2], p0[3], p1[3], xv[k].z, xv[k].w);
          } else {
            mma(group_sum[0], p0[0], p1[0], p0[1], p1[1], xv[k].x, xv[k].y);
            mma(group_sum[kChains - 1], p0[2], p1[2], p0[3], p1[3], xv[k].z, xv[k].w);
          }
          if (k % kWords == kWords - 1) {
            const int gr = j * (kChunk / kGroup) + k / kWords;  // of the block's eight
            const float f0 = __shfl_sync(0xffffffffu, scales[gr % 4], g * 2 + gr / 4);
            const float f1 = __shfl_sync(0xffffffffu, scales[gr % 4], g * 2 + 16 + gr / 4);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              float v = group_sum[0][m];
              if (kChains == 2) v += group_sum[kChains - 1][m];
              sum[m] = fmaf(m < 2 ? f0 : f1, v, sum[m]);
            }
          }
        }
        __syncwarp();  // (the words of this slot are read)
        ask();
      }
    }
    i += kBlock;
    if (i >= count) {
      i = 0;
      close();
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Experts' rows of a pass: as many as are staged.
int pass_rows(const Int4Gemm &g) {
  const int fit = (int)(kStagedBytes / staged_pitch((g.K + kChunk - 1) / kChunk));
  return std::min(std::min(g.T, kRows), fit);
}

template <int kGroup, int kWarpRows, bool kStaged, bool kExperts>
cudaError_t start(const Int4Gemm &g, cudaStream_t s) {
  auto kern = int4_small_kernel<kGroup, kWarpRows, kStaged, kExperts>;
  static std::atomic<bool> allowed[64];
  const size_t tables = kExperts ? (size_t)2 * (g.E + 1) * 4 : 0;
  const cudaError_t e = allow_smem(kern, kRingBytes + kStagedBytes + 2 * (kMaxE + 1) * 4, allowed);
  if (e != cudaSuccess) return e;
  SmallArgs a = {};
  a.T = kExperts ? pass_rows(g) : g.T;
  a.N = g.N;
  a.K = g.K;
  a.tiles = (g.N + 16 * kWarpRows - 1) / (16 * kWarpRows);
  a.chunks = (g.K + kChunk - 1) / kChunk;
  a.groups = (g.K + kGroup - 1) / kGroup;
  a.pitch = int4_pitch(g.K);
  a.offsets = g.offsets;
  a.R = g.T;
  a.E = g.E;
  a.status = g.status;
  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.act = g.act;
  a.x = static_cast<const uint8_t *>(kStaged ? g.x : g.xr);
  a.factor = g.factor;
  a.q = g.q;
  a.scale = static_cast<const uint16_t *>(g.scale);
  a.bias = g.bias;
  a.residual = g.residual;
  a.y = g.y;
  a.ldx = g.ldx;
  a.ldr = g.ldr;
  a.ldy = g.ldy;
  const size_t smem = kRingBytes + (kStaged ? (size_t)a.T * staged_pitch(a.chunks) : 0) + tables;
  const int64_t tiles = kExperts ? ((int64_t)std::min(g.E, g.T) + g.T / a.T) * a.tiles : a.tiles;
  return launch_pdl(kern, dim3((unsigned)std::min<int64_t>(tiles, num_sms())), dim3(kThreads), smem, s, a);
}

// The rows of a tile that take the least time: whole rounds of the SMs' tiles, each as long
// as its warps' chunks and about 0.6 chunks for its end.  Experts': as if all had rows; 29 of 128
// experts of 4096 x 1536 take 39.6 us in tiles of 64 rows, 33.4 of 128 and 34.8 of 256 (51 of 32,
// which are left out).
int warp_rows(const Int4Gemm &g) {
  const int chunks = (g.K + kChunk - 1) / kChunk;
  int best = 1;
  double least = 0;
  for (int wr = g.offsets != nullptr ? 4 : 1; wr <= kWarps; wr *= 2) {
    const int64_t tiles = (int64_t)((g.N + 16 * wr - 1) / (16 * wr)) * std::min(g.E, g.T);
    const int rounds = (int)((tiles + num_sms() - 1) / num_sms());
    const int split = kWarps / wr;
    const double us = (double)rounds * ((chunks + split - 1) / split + (split > 1 ? 0.6 : 0.2));
    if (least == 0 || us < least) {
      least = us;
      best = wr;
    }
  }
  return best;
}

template <int kGroup, bool kStaged, bool kExperts>
cudaError_t by_rows(const Int4Gemm &g, cudaStream_t s) {
  const int wr = warp_rows(g);
  if constexpr (!kExperts) {
    if (wr == 1) return start<kGroup, 1, kStaged, false>(g, s);
    if (wr == 2) return start<kGroup, 2, kStaged, false>(g, s);
  }
  if (wr == 4) return start<kGroup, 4, kStaged, kExperts>(g, s);
  if (wr == 8) return start<kGroup, 8, kStaged, kExperts>(g, s);
  return start<kGroup, 16, kStaged, kExperts>(g, s);
}
template <bool kStaged, bool kExperts>
cudaError_t by_group(const Int4Gemm &g, cudaStream_t s) {
  if constexpr (!kExperts) {
    if (g.group == 32) return by_rows<32, kStaged, false>(g, s);
  }
  return g.group == 64 ? by_rows<64, kStaged, kExperts>(g, s) : by_rows<128, kStaged, kExperts>(g, s);
}

}  // namespace

bool int4_staged(const Int4Gemm &g) {
  return (size_t)g.T * staged_pitch((g.K + kChunk - 1) / kChunk) <= kStagedBytes;
}

// Experts' rows: here, or by way of tcgen05, which takes up to 32 rows in a pass.  128 experts of
// 4096 x 1536, groups of 128: 8 rows over all of them 12.4 and 18.6 us, 32 rows 30.1 and 35.2, 128
// rows 70.6 and 89.3, 512 rows 115 and 136.  32 experts of 4096 x 7168, where five rows fit a pass,
// groups of 64: 64 rows 108 and 118 us, 128 rows 145 and 129.  Groups of 32 have four times
// the scales to bring to their lanes: 64 experts of 1536 x 4096 with 8 rows 19.7 and 18.2 us, with 64
// rows 60 and 46.
bool int4_few(const Int4Gemm &g) {
  if (g.group == 32) return false;
  const int most = pass_rows(g);
  return g.T <= most || (g.T + g.E - 1) / g.E <= most / 2;
}

cudaError_t launch_int4_small(const Int4Gemm &g, cudaStream_t s) {
  if (g.offsets != nullptr) return by_group<true, true>(g, s);
  return int4_staged(g) ? by_group<true, false>(g, s) : by_group<false, false>(g, s);
}

}  // namespace moe
