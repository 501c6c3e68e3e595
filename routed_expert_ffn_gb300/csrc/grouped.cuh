// Shared by the experts' ragged products (grouped_pair.cu) and their C ABI
// (api_grouped.cu).
#pragma once

#include "dense.cuh"

namespace moe {

// Rows [offsets[e], offsets[e+1]) of the row tensors belong to matrix e of w [E][N][K].
struct GroupedGemm {
  int R, E, N, K;
  int dtype;      // of every operand: MOE_DTYPE_BF16 or FP16
  int out_dtype;  // of the result
  const int32_t *offsets;
  const void *x, *w, *dy;     // x rows ldx apart, dy rows ldy apart
  int64_t ldx, ldy;
  void *d;                    // y (rows ldy apart), dx (rows ldx apart) or dw
  int accumulate;             // dw: added to what it holds
  float *part;                // partial sums of split tiles
  CUtensorMap *maps;          // dw: grouped_map_bytes(E)
  uint32_t *status;           // the workspace's status block
};

// Bytes of `part` for R rows.
size_t grouped_part_bytes(int R);
inline size_t grouped_map_bytes(int E) { return (size_t)E * 2 * sizeof(CUtensorMap); }

// What a cluster or CTA works on: stages [k0, k1) of a tile.
struct Work {
  int e;
  int a0;      // first row of the tile's stretch of the matrix
  int b0;      // first row of x, or column of dW
  int n;       // rows, or columns, of the tile
  int k0, k1;  // stages
  int parts, part, tile;
};

// first[e] <= tile < first[e + 1]
__device__ __forceinline__ int expert_of(const int32_t *first, int E, int tile) {
  int l = 0, r = E;
  while (r - l > 1) {
    const int mid = (l + r) >> 1;
    if (first[mid] <= tile)
      l = mid;
    else
      r = mid;
  }
  return l;
}

// The offsets (null: all T rows of one matrix), as far as they lie in rows [low, high), to
// seg [E+1], and the prefix sums of tiles(rows of an expert) to first [E+1], in shared
// memory; by all threads of the block, which meet afterwards.  Offsets that do not hold make
// no tiles, and a status bit.
template <typename Tiles>
__device__ __forceinline__ void make_tables(const int32_t *offsets, int E, int T, int low, int high,
                                            int32_t *seg, int32_t *first, uint32_t *status,
                                            Tiles tiles) {
  bool good = true;
  for (int i = threadIdx.x; i <= E; i += blockDim.x) {
    int o = i == 0 ? 0 : T;
    if (offsets != nullptr) {
      const int before = i > 0 ? __ldg(offsets + i - 1) : 0;
      o = __ldg(offsets + i);
      good = good && before >= 0 && o >= before && o <= T;
    }
    seg[i] = min(max(o, low), high);
  }
  good = __syncthreads_and(good);
  if (threadIdx.x < 32) {
    // a run of experts to a lane
    const int lane = threadIdx.x;
    const int per = (E + 31) / 32, e0 = min(E, lane * per), e1 = min(E, e0 + per);
    int sum = 0;
    if (good)
      for (int e = e0; e < e1; ++e) sum += tiles(seg[e + 1] - seg[e]);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int run = incl - sum;
    for (int e = e0; e < e1; ++e) {
      first[e] = run;
      if (good) run += tiles(seg[e + 1] - seg[e]);
    }
    if (lane == 31) first[E] = incl;
    if (!good && lane == 0 && blockIdx.x == 0) atomicOr(status, kStatusBadOffsets);
  }
}

// Tiles of kTile rows of an expert's matrix by up to kRows of its rows (a multiple of
// kAlign, split evenly), as worker `cid` of `ncl` sees them.  The tiles that do not
// fill a round of the workers come first, their stages dealt out evenly: at most the
// end of one tile and the start of the next to a worker, no more than kMaxParts
// pieces of a tile, of kMinPart stages at least.
template <int kRows, int kAlign, int kTile, int kMaxParts, int kMinPart>
struct RowSchedule {
  const int32_t *seg, *first;  // (shared memory)
  int E, mt, nkb;              // mt: tiles down a matrix; nkb: stages of its depth
  int total, rem, units, cid, ncl;
  int lo, hi, pieces;  // of this worker

  __host__ __device__ static int row_tiles(int m) { return (m + kRows - 1) / kRows; }

  __device__ __forceinline__ void start() {
    total = first[E];
    rem = total % ncl;
    pieces = 0;
    if (rem == 0) return;
    units = max((rem * nkb + ncl - 1) / ncl,
                max((nkb + kMaxParts - 1) / kMaxParts, min(kMinPart, nkb)));
    if (nkb - units < kMinPart) units = nkb;
    lo = min(rem * nkb, cid * units);
    hi = min(rem * nkb, lo + units);
    if (hi > lo) pieces = (hi - 1) / nkb - lo / nkb + 1;
  }
  // Where worker c keeps its partial sums of tile t.
  __device__ __forceinline__ int slot(int c, int t) const { return 2 * c + t - c * units / nkb; }
  __device__ __forceinline__ int first_worker(int t) const { return t * nkb / units; }

  __device__ __forceinline__ bool at(int i, Work *w) const {
    int tile;
    w->part = 0;
    w->parts = 1;
    w->k0 = 0;
    w->k1 = nkb;
    if (i < pieces) {
      tile = lo / nkb + i;
      w->k0 = max(lo - tile * nkb, 0);
      w->k1 = min(hi - tile * nkb, nkb);
      const int c = first_worker(tile);
      w->part = cid - c;
      w->parts = ((tile + 1) * nkb - 1) / units - c + 1;
    } else {
      tile = rem + (i - pieces) * ncl + cid;
      if (tile >= total) return false;
    }
    const int e = expert_of(first, E, tile);
    // the row tiles of one stretch of the matrix follow each other: they run together
    const int m = seg[e + 1] - seg[e], rt = row_tiles(m);
    const int at = tile - first[e], j = at / rt, r = at - j * rt;
    const int per = ((m + rt - 1) / rt + kAlign - 1) / kAlign * kAlign;  // (rt - 1) per < m
    w->e = e;
    w->tile = tile;
    w->a0 = j * kTile;
    w->b0 = seg[e] + r * per;
    w->n = min(per, m - r * per);
    return true;
  }
};

// One thread's arrival at a split tile's counter, after a barrier behind the writes of all whose
// part it is: true for the last of `parts`, which then sees the others' (after another
// barrier everybody behind it).
__device__ __forceinline__ bool arrive_last(uint32_t *counter, int parts) {
  uint32_t before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  if (before + 1 != (uint32_t)parts) return false;
  *counter = 0;  // nobody else comes
  return true;
}

cudaError_t launch_grouped_rows(const GroupedGemm &g, bool grad, cudaStream_t s);
cudaError_t launch_grouped_weight_grad(const GroupedGemm &g, cudaStream_t s);

}  // namespace moe
