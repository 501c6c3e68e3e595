// Products with 4-bit weights and few rows (decode): y = act(x W^T + bias) + residual of
// one matrix, or y_p = W_e x_p for the rows p of each expert e.
//
// Bound: HBM, which reads half a byte for each weight; next to it the instructions
// that unpack the codes (a word of eight takes three shifts, four LOP3 and four
// subtractions), so every weight is unpacked once for all rows of a pass.
//
// Two codes become the two halves of a 32-bit register: masked, and given the
// exponent under which their bits count ones (bf16 128 + code, fp16 1024 + code); less
// 128 + 8 that is code - 8, exactly.  They are the A operand of mma.sync (16 rows of W
// by 16 of depth), x is B (8 rows of x): with one to 16 rows the tensor cores of
// tcgen05 would wait for the unpacking all the same, and its operands would have to
// go through shared or tensor memory.  A group's sum is scaled in fp32 when it is
// complete: neither codes nor scales are rounded.
//
// Which k an operand element is does not matter as long as A and B agree.  A lane
// takes 16 bytes of a row as they lie (32 codes): lane t of a quad those at
// 32 t of a chunk of 128; word i of them, nibbles j and j + 4, pairs with x's elements
// j and j + 4 of the same eight.  Groups of 32 or 64 end inside a chunk: the
// lanes of a quad exchange words so that each MMA sees one group alone.
//
// A CTA takes tiles of 16 kWarpRows rows of W: warps split the depth by chunks, each
// with kAhead chunks of codes in flight in registers, across tiles as well, and
// add their sums through shared memory.
#include <algorithm>

#include "int4.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;
constexpr int kChunk = 128;

struct SmallArgs {
  const int32_t *offsets;
  int T, E, N, K;
  int row_blocks;  // tiles of a matrix
  int chunks, groups;
  int dtype, out_dtype, act;
  const uint8_t *x;
  const uint8_t *q;
  const uint16_t *scale;
  const void *bias, *residual;
  void *y;
  int64_t ldx, ldr, ldy;
  uint32_t *status;
};

template <bool kFp16>
__device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
  uint32_t d;
  if (kFp16)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Nibbles j and j + 4 of a word as two numbers: (j = 0..3) of p[j].
template <bool kFp16>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&p)[4]) {
  constexpr uint32_t kOne = kFp16 ? 0x64006400u : 0x43004300u;   // 1024 or 128, twice
  constexpr uint32_t kZero = kFp16 ? 0x64086408u : 0x43084308u;  // 8 more
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = minus<kFp16>((w >> (4 * j) & 0x000f000fu) | kOne, kZero);
}
template <bool kFp16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (kFp16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Words of a quad's four lanes exchanged so that word i of every lane is of one group
// (kGroup 32: of group i; 64: words 0 and 1 of group 0, 2 and 3 of group 1).
template <int kGroup>
__device__ __forceinline__ void regroup(uint4 &v, int t) {
  if (kGroup == 128) return;
  // lanes t and t ^ 2 exchange two words
  {
    const bool high = (t & 2) != 0;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, high ? v.x : v.z, 2);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, high ? v.y : v.w, 2);
    v = high ? make_uint4(a, b, v.z, v.w) : make_uint4(v.x, v.y, a, b);
  }
  if (kGroup == 32) {
    // and lanes t and t ^ 1 one of each two
    const bool odd = (t & 1) != 0;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.y, 1);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, odd ? v.z : v.w, 1);
    v = odd ? make_uint4(a, v.y, b, v.w) : make_uint4(v.x, a, v.z, b);
  }
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

// One tile: 16 rows of W for each of kWarpRows warps, up to 8 kN rows of x.
struct SmallTile {
  int e, n0, row0, rows;
};

template <int kN, int kWarpRows>
struct SmallTiles {
  const int32_t *seg, *first;  // [E+1] (shared memory); null: one matrix
  int E, T, row_blocks, total;
  __device__ __forceinline__ SmallTile at(int tile) const {
    SmallTile t;
    int l = 0, begin = 0, end = T, base = 0;
    if (seg != nullptr) {
      int r = E;
      while (r - l > 1) {
        const int mid = (l + r) >> 1;
        if (first[mid] <= tile)
          l = mid;
        else
          r = mid;
      }
      begin = seg[l];
      end = seg[l + 1];
      base = first[l];
    }
    // the passes over one stretch of W follow each other
    const int passes = (end - begin + 8 * kN - 1) / (8 * kN);
    const int at = tile - base, block = at / passes, pass = at - block * passes;
    t.e = l;
    t.n0 = block * 16 * kWarpRows;
    t.row0 = begin + pass * 8 * kN;
    t.rows = min(8 * kN, end - t.row0);
    return t;
  }
};

// The tile's sums of all warps, then everything after them, rounded once.
template <int kN, int kWarpRows>
__device__ __noinline__ void finish(const SmallArgs &a, const SmallTile &t, const float *red) {
  constexpr int kCols = 16 * kWarpRows, kRows = 8 * kN, kSplit = kWarps / kWarpRows;
  for (int i = threadIdx.x; i < kCols * kRows; i += kThreads) {
    const int c = i % kCols, r = i / kCols;
    if (r >= t.rows || t.n0 + c >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kSplit; ++s) v += red[(s * kRows + r) * (kCols + 1) + c];
    const int n = t.n0 + c;
    const int64_t row = t.row0 + r;
    auto load = [&](const void *p, int64_t at) {
      if (a.out_dtype == MOE_DTYPE_FP32) return static_cast<const float *>(p)[at];
      return unpack16(a.out_dtype, static_cast<const uint16_t *>(p)[at]).x;
    };
    if (a.bias != nullptr) v += load(a.bias, n);
    if (a.act != MOE_ACT_NONE)
      v = a.out_dtype == MOE_DTYPE_FP32 ? activate<true>(a.act, v) : activate<false>(a.act, v);
    if (a.residual != nullptr) v += load(a.residual, row * a.ldr + n);
    if (a.out_dtype == MOE_DTYPE_FP32)
      static_cast<float *>(a.y)[row * a.ldy + n] = v;
    else
      static_cast<uint16_t *>(a.y)[row * a.ldy + n] = (uint16_t)pack16(a.out_dtype, v, 0.f);
  }
}

template <bool kFp16, int kGroup, int kN, int kWarpRows>
__global__ void __launch_bounds__(kThreads, 2)
    int4_small_kernel(const __grid_constant__ SmallArgs a) {
  constexpr int kCols = 16 * kWarpRows, kRows = 8 * kN, kSplit = kWarps / kWarpRows;
  constexpr int kRed = kSplit * kRows * (kCols + 1);
  __shared__ float red[2][kRed];
  extern __shared__ int32_t tables[];  // offsets: [E+1] and tile prefix sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp % kWarpRows, part = warp / kWarpRows;
  pdl_wait();
  pdl_launch_dependents();

  SmallTiles<kN, kWarpRows> tiles;
  tiles.E = a.E;
  tiles.T = a.T;
  tiles.row_blocks = a.row_blocks;
  tiles.seg = nullptr;
  tiles.first = nullptr;
  if (a.offsets != nullptr) {
    int32_t *seg = tables, *first = tables + a.E + 1;
    bool good = true;
    for (int i = threadIdx.x; i <= a.E; i += kThreads) {
      const int o = __ldg(a.offsets + i), before = i > 0 ? __ldg(a.offsets + i - 1) : 0;
      seg[i] = o;
      good = good && before >= 0 && o >= before && o <= a.T;
    }
    good = __syncthreads_and(good);
    if (warp == 0) {
      auto count = [&](int e) { return (seg[e + 1] - seg[e] + kRows - 1) / kRows * a.row_blocks; };
      const int per = (a.E + 31) / 32, e0 = min(a.E, lane * per), e1 = min(a.E, e0 + per);
      int sum = 0;
      if (good)
        for (int e = e0; e < e1; ++e) sum += count(e);
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int run = incl - sum;
      for (int e = e0; e < e1; ++e) {
        first[e] = run;
        if (good) run += count(e);
      }
      if (lane == 31) first[a.E] = incl;
      if (!good && lane == 0 && blockIdx.x == 0) atomicOr(a.status, kStatusBadOffsets);
    }
    __syncthreads();
    tiles.seg = seg;
    tiles.first = first;
    tiles.total = first[a.E];
  } else {
    tiles.total = (a.T + kRows - 1) / kRows * a.row_blocks;
  }

  // this warp's chunks of a tile: part, part + kSplit, ...
  const int count = part < a.chunks ? (a.chunks - part + kSplit - 1) / kSplit : 0;

  // Where the next codes to be asked for lie.
  struct Item {
    uint4 q0, q1;
    uint32_t s0, s1;
  };
  int ahead_tile = blockIdx.x, ahead_i = 0;
  const uint8_t *q0 = nullptr, *q1 = nullptr;
  const uint16_t *s0 = nullptr, *s1 = nullptr;
  auto aim = [&]() {
    if (ahead_tile >= tiles.total) return;
    const SmallTile w = tiles.at(ahead_tile);
    const int n = w.n0 + 16 * wr + g;
    const int64_t r0 = (int64_t)w.e * a.N + min(n, a.N - 1);
    const int64_t r1 = (int64_t)w.e * a.N + min(n + 8, a.N - 1);
    q0 = a.q + r0 * (a.K >> 1) + 16 * t;
    q1 = a.q + r1 * (a.K >> 1) + 16 * t;
    s0 = a.scale + r0 * a.groups;
    s1 = a.scale + r1 * a.groups;
  };
  auto ask = [&](Item &it) {
    if (ahead_tile >= tiles.total) return;
    const int c = part + ahead_i * kSplit;
    it.q0 = it.q1 = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
    if (c * kChunk + 32 * t < a.K) {
      it.q0 = load_codes(q0 + (int64_t)c * (kChunk / 2));
      it.q1 = load_codes(q1 + (int64_t)c * (kChunk / 2));
    }
    const int group = c * (kChunk / kGroup) + (kGroup == 128 ? 0 : (kGroup == 64 ? t >> 1 : t));
    it.s0 = it.s1 = 0;
    if (group < a.groups) {
      it.s0 = __ldg(s0 + group);
      it.s1 = __ldg(s1 + group);
    }
    if (++ahead_i == count) {
      ahead_i = 0;
      ahead_tile += gridDim.x;
      aim();
    }
  };

  Item item[kAhead];
  if (count > 0) {
    aim();
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ask(item[j]);
  }
  float sum[kN][4];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[n][i] = 0.f;
  int tile = blockIdx.x, i = 0;
  uint32_t turn = 0;
  SmallTile w = {};
  if (tile < tiles.total) w = tiles.at(tile);

  // The warp's sums to shared memory; the last warp's arrival completes the tile.
  auto close = [&]() {
    float *to = red[turn] + part * kRows * (kCols + 1) + 16 * wr;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        to[(8 * n + 2 * t + (k & 1)) * (kCols + 1) + g + 8 * (k >> 1)] = sum[n][k];
        sum[n][k] = 0.f;
      }
    }
    __syncthreads();
    finish<kN, kWarpRows>(a, w, red[turn]);
    turn ^= 1u;  // the other buffer was read before everybody arrived here
    tile += gridDim.x;
    if (tile < tiles.total) w = tiles.at(tile);
  };

  if (count == 0) {
    while (tile < tiles.total) close();
    return;
  }
  while (tile < tiles.total) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (tile >= tiles.total) break;
      const int c = part + i * kSplit;
      const uint8_t *xp[kN];
#pragma unroll
      for (int n = 0; n < kN; ++n)
        xp[n] = 8 * n + g < w.rows
                    ? a.x + ((int64_t)(w.row0 + 8 * n + g) * a.ldx + (int64_t)c * kChunk) * 2
                    : nullptr;
      uint4 c0 = item[j].q0, c1 = item[j].q1;
      const uint32_t sc0 = item[j].s0, sc1 = item[j].s1;
      regroup<kGroup>(c0, t);
      regroup<kGroup>(c1, t);
      ask(item[j]);
      float part_sum[kN][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        constexpr int kWords = kGroup / 32;  // words to a group
        if (k % kWords == 0) {
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m) part_sum[n][m] = 0.f;
        }
        uint32_t p0[4], p1[4];
        unpack<kFp16>(word(c0, k), p0);
        unpack<kFp16>(word(c1, k), p1);
        const int at = k_of<kGroup>(t, k);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (xp[n] != nullptr && c * kChunk + at < a.K)
            v = __ldg(reinterpret_cast<const uint4 *>(xp[n] + at * 2));
          mma<kFp16>(part_sum[n], p0[0], p1[0], p0[1], p1[1], __byte_perm(v.x, v.z, 0x5410),
                     __byte_perm(v.x, v.z, 0x7632));
          mma<kFp16>(part_sum[n], p0[2], p1[2], p0[3], p1[3], __byte_perm(v.y, v.w, 0x5410),
                     __byte_perm(v.y, v.w, 0x7632));
        }
        if (k % kWords == kWords - 1) {
          // lane t (of its quad) holds the scale of the group that its own codes are of
          uint32_t u0 = sc0, u1 = sc1;
          if (kGroup != 128) {
            const int from = (lane & ~3) | (kGroup == 64 ? (k & 2) : k);
            u0 = __shfl_sync(0xffffffffu, sc0, from);
            u1 = __shfl_sync(0xffffffffu, sc1, from);
          }
          const float f0 = unpack16(kFp16 ? MOE_DTYPE_FP16 : MOE_DTYPE_BF16, u0).x;
          const float f1 = unpack16(kFp16 ? MOE_DTYPE_FP16 : MOE_DTYPE_BF16, u1).x;
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            sum[n][0] = fmaf(f0, part_sum[n][0], sum[n][0]);
            sum[n][1] = fmaf(f0, part_sum[n][1], sum[n][1]);
            sum[n][2] = fmaf(f1, part_sum[n][2], sum[n][2]);
            sum[n][3] = fmaf(f1, part_sum[n][3], sum[n][3]);
          }
        }
      }
      if (++i == count) {
        i = 0;
        close();
      }
    }
  }
}

template <bool kFp16, int kGroup, int kN, int kWarpRows>
cudaError_t start(const Int4Gemm &g, cudaStream_t s) {
  SmallArgs a = {};
  a.offsets = g.offsets;
  a.T = g.T;
  a.E = g.E;
  a.N = g.N;
  a.K = g.K;
  a.row_blocks = (g.N + 16 * kWarpRows - 1) / (16 * kWarpRows);
  a.chunks = (g.K + kChunk - 1) / kChunk;
  a.groups = (g.K + kGroup - 1) / kGroup;
  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.act = g.act;
  a.x = static_cast<const uint8_t *>(g.x);
  a.q = g.q;
  a.scale = static_cast<const uint16_t *>(g.scale);
  a.bias = g.bias;
  a.residual = g.residual;
  a.y = g.y;
  a.ldx = g.ldx;
  a.ldr = g.ldr;
  a.ldy = g.ldy;
  a.status = g.status;
  const int64_t passes = g.offsets != nullptr ? (int64_t)std::min(g.E, g.T) + g.T / (8 * kN)
                                              : (g.T + 8 * kN - 1) / (8 * kN);
  const int64_t most = passes * a.row_blocks;
  const size_t smem = g.offsets != nullptr ? (size_t)2 * (g.E + 1) * 4 : 0;
  return launch_pdl(int4_small_kernel<kFp16, kGroup, kN, kWarpRows>,
                    dim3((unsigned)std::min<int64_t>(most, 2 * (int64_t)num_sms())), dim3(kThreads),
                    smem, s, a);
}

template <bool kFp16, int kGroup>
cudaError_t by_rows(const Int4Gemm &g, cudaStream_t s) {
  const bool one = g.T <= 8 * g.E;
  return one ? start<kFp16, kGroup, 1, 1>(g, s) : start<kFp16, kGroup, 2, 2>(g, s);
}
template <bool kFp16>
cudaError_t by_group(const Int4Gemm &g, cudaStream_t s) {
  if (g.group == 32) return by_rows<kFp16, 32>(g, s);
  return g.group == 64 ? by_rows<kFp16, 64>(g, s) : by_rows<kFp16, 128>(g, s);
}

}  // namespace

cudaError_t launch_int4_small(const Int4Gemm &g, cudaStream_t s) {
  return g.dtype == MOE_DTYPE_FP16 ? by_group<true>(g, s) : by_group<false>(g, s);
}

}  // namespace moe
