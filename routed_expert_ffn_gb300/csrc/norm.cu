// Residual addition with root-mean-square norm, and its gradient.
//
//   s = x + residual            y = w * s * r,   r = (mean(s^2) + eps)^(-1/2)
//
// With n = s r and the loss's gradients dy of y and dres of s:
//
//   dx = dres + r (w dy - n mean(w dy n))        (the gradient of both x and residual)
//   dw = sum over the rows of dy n
//
// Everything between loads and stores is in 32 bits; s is normalised before
// it is rounded to the stored residual.
//
// Bound: HBM.  Forward: 3 row tensors read and written plus y (or its 8-bit
// codes); backward: 3 read, 1 written.  A row lives in the registers of one
// group of threads (kV chunks of 8 elements a thread), so every tensor is read
// once, and the mean costs a reduction in each warp and one exchange through
// shared memory.  Forward a CTA ends with its row (or few short ones); backward
// the CTAs stay and walk the rows, adding up dw in registers, and each thread
// copies its own chunks of the next rows to shared memory meanwhile (cp.async
// into a ring that no other thread touches): loads stay in flight through the
// reductions without taking registers.  The arithmetic is done on pairs (f32x2):
// with one instruction an element it took as long as the bytes.
#include <cuda_fp8.h>

#include <algorithm>

#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 512;

// ---------------------------------------------------------- pairs of fp32 --

typedef unsigned long long pair_t;  // (low word, high word)

__device__ __forceinline__ pair_t make_pair(float lo, float hi) {
  pair_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float lo_of(pair_t p) {
  return __uint_as_float((uint32_t)p);
}
__device__ __forceinline__ float hi_of(pair_t p) {
  return __uint_as_float((uint32_t)(p >> 32));
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
  pair_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
  pair_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) {
  pair_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// --------------------------------------------------------------- chunks --

// A chunk is 8 elements in pieces of 16 bytes: one piece of 8 (bf16, fp16) or
// two of 4 (fp32).  Piece i of a thread's chunk v is number (v * pieces + i) *
// group + thread of the row, so a warp's pieces lie side by side.
template <typename T>
struct Chunk {
  static constexpr int kPieces = sizeof(T) / 2;
  static constexpr int kEach = 8 / kPieces;  // elements of a piece
  uint4 a[kPieces];
};
template <typename T>
__device__ __forceinline__ int column(int v, int i, int group, int t) {
  return ((v * Chunk<T>::kPieces + i) * group + t) * Chunk<T>::kEach;
}

// `p`: the row.  Pieces past H (or all, where `live` is false) are zero.
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T *p, int v, int group, int t, int H,
                                               bool live) {
  Chunk<T> r;
#pragma unroll
  for (int i = 0; i < Chunk<T>::kPieces; ++i) {
    const int c = column<T>(v, i, group, t);
    r.a[i] = make_uint4(0, 0, 0, 0);
    // not the read-only path: outputs may overlay inputs row for row
    if (live && c < H)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.a[i].x), "=r"(r.a[i].y), "=r"(r.a[i].z), "=r"(r.a[i].w)
                   : "l"(p + c));
  }
  return r;
}

// A thread's ring in shared memory: `at` is this thread's 16 bytes of a chunk's
// first piece; the pieces of all threads of the CTA lie side by side.
template <typename T>
__device__ __forceinline__ void ring_fill(uint32_t at, const T *p, int v, int group, int t, int H,
                                          int threads) {
#pragma unroll
  for (int i = 0; i < Chunk<T>::kPieces; ++i) {
    const int c = column<T>(v, i, group, t);
    if (c < H)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + i * threads * 16),
                   "l"(p + c)
                   : "memory");
  }
}
template <typename T>
__device__ __forceinline__ Chunk<T> ring_read(uint32_t at, int v, int group, int t, int H,
                                              int threads, bool live) {
  Chunk<T> r;
#pragma unroll
  for (int i = 0; i < Chunk<T>::kPieces; ++i) {
    r.a[i] = make_uint4(0, 0, 0, 0);
    if (live && column<T>(v, i, group, t) < H)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.a[i].x), "=r"(r.a[i].y), "=r"(r.a[i].z), "=r"(r.a[i].w)
                   : "r"(at + i * threads * 16)
                   : "memory");
  }
  return r;
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `ahead` (at most 3) of this thread's fills have landed.
__device__ __forceinline__ void ring_wait(int ahead) {
  switch (ahead) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

__device__ __forceinline__ void to_pairs(const Chunk<__nv_bfloat16> &r, pair_t (&f)[4]) {
  const uint32_t w[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = make_pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void to_pairs(const Chunk<__half> &r, pair_t (&f)[4]) {
  const uint32_t w[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[i] = make_pair(v.x, v.y);
  }
}
__device__ __forceinline__ void to_pairs(const Chunk<float> &r, pair_t (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = make_pair(__uint_as_float(r.a[i].x), __uint_as_float(r.a[i].y));
    f[2 * i + 1] = make_pair(__uint_as_float(r.a[i].z), __uint_as_float(r.a[i].w));
  }
}

__device__ __forceinline__ Chunk<__nv_bfloat16> from_pairs(const pair_t (&f)[4], __nv_bfloat16) {
  Chunk<__nv_bfloat16> r;
  r.a[0] = make_uint4(pack_bf16x2(lo_of(f[0]), hi_of(f[0])), pack_bf16x2(lo_of(f[1]), hi_of(f[1])),
                      pack_bf16x2(lo_of(f[2]), hi_of(f[2])), pack_bf16x2(lo_of(f[3]), hi_of(f[3])));
  return r;
}
__device__ __forceinline__ Chunk<__half> from_pairs(const pair_t (&f)[4], __half) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(lo_of(f[i]), hi_of(f[i]));
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  Chunk<__half> r;
  r.a[0] = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}
__device__ __forceinline__ Chunk<float> from_pairs(const pair_t (&f)[4], float) {
  Chunk<float> r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.a[i] = make_uint4(__float_as_uint(lo_of(f[2 * i])), __float_as_uint(hi_of(f[2 * i])),
                        __float_as_uint(lo_of(f[2 * i + 1])), __float_as_uint(hi_of(f[2 * i + 1])));
  return r;
}
// Rounded to T, to the row `p`.
template <typename T>
__device__ __forceinline__ void store_chunk(T *p, const pair_t (&f)[4], int v, int group, int t,
                                            int H) {
  const Chunk<T> r = from_pairs(f, T());
#pragma unroll
  for (int i = 0; i < Chunk<T>::kPieces; ++i) {
    const int c = column<T>(v, i, group, t);
    if (c < H) *reinterpret_cast<uint4 *>(p + c) = r.a[i];
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// An fp32 sum with what its rounding left.
struct Kept {
  float hi, lo;
};
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// The warp's sum of hi (kTwo: hi + lo), not negative, added in integers: in units of
// 2^-25 of the largest lane's power of two, so that lanes within a factor of 4 of it
// lose nothing and the others half a unit.  Two reductions in hardware; shuffles with
// fp32 additions round at each of five steps (keeping what they round off took 74.4 us
// of 8192 x 7168 where this takes 69.3).  Sums below 2^-101, whose units are not normal
// numbers, infinities and NaN take the shuffles.
template <bool kTwo>
__device__ __forceinline__ Kept warp_sum_kept(Kept v) {
  constexpr uint32_t kLeast = 26u << 23;
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v.hi));
  if (m - kLeast >= 0x7f800000u - kLeast) return {warp_sum(v.hi), 0.f};
  const int e = 152 - (int)(m >> 23);
  const int units = __float2int_rn(v.hi * pow2(e)) + (kTwo ? __float2int_rn(v.lo * pow2(e)) : 0);
  const uint32_t s = __reduce_add_sync(0xffffffffu, (uint32_t)units);
  const float h = __uint2float_rn(s);
  return {h * pow2(-e), (float)(int)(s - __float2uint_rn(h)) * pow2(-e)};
}
// (hi + lo) / n rounded once; inv_n = 1 / n in fp32.
__device__ __forceinline__ float mean_of(Kept s, float n, float inv_n) {
  const float q = s.hi * inv_n;
  return fabsf(q) < INFINITY ? fmaf(fmaf(-q, n, s.hi) + s.lo, inv_n, q) : q;
}

// The power-of-two exponent of a block of 8-bit values with absolute maximum
// `amax` (of fp32 values): the least s with amax <= 448 * 2^s (448 = 1.75 * 2^8,
// the largest E4M3 value), at least -126; 0 for a block of zeros.
__device__ __forceinline__ int block_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0u) return 0;
  const int s = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(s, -126);
}

struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *y;
  uint8_t *q;
  int8_t *scale;
  int64_t x_stride, r_stride, y_stride;
  int T, H, group;  // group: threads to a row
  float eps, inv_h;  // inv_h: 1 / H
};

// y of a chunk as E4M3 codes.  A block of 128 elements lies in 16 neighbouring
// lanes (8 elements each) or, piece by piece, in 32 (fp32).
template <typename T>
__device__ __forceinline__ void store_codes(const NormArgs &a, const pair_t (&y)[4], int64_t row,
                                            int v, int t, bool live) {
  constexpr int kPieces = Chunk<T>::kPieces, kPairs = 4 / kPieces;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const pair_t *p = y + i * kPairs;
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) m = fmaxf(m, fmaxf(fabsf(lo_of(p[j])), fabsf(hi_of(p[j]))));
#pragma unroll
    for (int o = 64 / Chunk<T>::kEach; o > 0; o >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = block_exp(m);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    const int c = column<T>(v, i, a.group, t);
    if (!live || c >= a.H) continue;
    uint32_t w[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      w[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo_of(p[j]) * inv, hi_of(p[j]) * inv),
                                                __NV_SATFINITE, __NV_E4M3);
    uint8_t *q = a.q + row * a.H + c;
    if (kPairs == 4)
      *reinterpret_cast<uint2 *>(q) =
          make_uint2(w[0] | w[1] << 16, w[kPairs > 2 ? 2 : 0] | w[kPairs > 2 ? 3 : 0] << 16);
    else
      *reinterpret_cast<uint32_t *>(q) = w[0] | w[1] << 16;
    if ((c & 127) == 0) a.scale[row * ((a.H + 127) >> 7) + (c >> 7)] = (int8_t)e;
  }
}

// This thread's chunks of a row, s = x + residual: residual_out and, once the
// row's mean is known, y and its codes.  kOne: the row is the whole CTA's, else a
// warp's.
//
// y = (s r) w in fp32, r = rsqrtf(mean + eps).  The exponent of a block is a step
// of its largest y, and a mean off in its last bit can move y across that step
// (1 of 55 million blocks of 8192 x 7168 inputs, with plain fp32 sums here).  So
// the sum over threads keeps what its additions round off, the mean is rounded
// once, and y has the bits that the same fp32 operations give anywhere: what is
// left is the threads' own fp32 sums, a few squares each, whose errors are
// independent and some 2^-28 of the whole.
template <typename T, int kV, bool kOne>
__device__ __forceinline__ void norm_row(const NormArgs &a, const Chunk<T> (&rx)[kV],
                                         const Chunk<T> (&rr)[kV], const Chunk<T> (&rw)[kV],
                                         int64_t row, int t, bool live) {
  __shared__ Kept part[kNormThreads / 32];
  pair_t s[kV][4], sq = make_pair(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    pair_t r[4];
    to_pairs(rx[v], s[v]);
    to_pairs(rr[v], r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[v][i] = add2(s[v][i], r[i]);
      sq = fma2(s[v][i], s[v][i], sq);
    }
    if (a.residual_out != nullptr && live)
      store_chunk(static_cast<T *>(a.residual_out) + row * a.r_stride, s[v], v, a.group, t, a.H);
  }
  // A warp's row, too, by way of shared memory: with its sum left in registers 65536 x
  // 256 takes 34.6 us, so 33.2 (31.8 with fp32 additions that keep nothing; of long
  // coded rows 8192 x 7168 65.9 and 64.4, 5120 columns 45.7 and 47.3).
  const int mine = kOne ? t >> 5 : threadIdx.y, lane = t & 31;
  Kept sum = warp_sum_kept<false>({lo_of(sq) + hi_of(sq), 0.f});
  if (lane == 0) part[mine] = sum;
  __syncthreads();
  if (kOne) {
    sum = lane < a.group >> 5 ? part[lane] : Kept{0.f, 0.f};
    sum = warp_sum_kept<true>(sum);
  } else {
    sum = part[mine];
  }
  const float rstd = rsqrtf(mean_of(sum, (float)a.H, a.inv_h) + a.eps);
  const pair_t r2 = make_pair(rstd, rstd);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    pair_t w[4], y[4];
    to_pairs(rw[v], w);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(s[v][i], r2), w[i]);
    if (a.y != nullptr && live)
      store_chunk(static_cast<T *>(a.y) + row * a.y_stride, y, v, a.group, t, a.H);
    if (a.q != nullptr) store_codes<T>(a, y, row, v, t, live);
  }
}

// blockDim.x threads (whole warps) to a row, kOne: the CTA's only one, else a warp's.
// Registers are held down to 40 a thread of two chunks (64 of four): what hides the
// loads is other CTAs' rows (8192 x 7168 78.4 us with 48, 69.9 with 40).  CTAs that
// stayed and copied the next rows to shared memory meanwhile took 9.4 us for 1021 x
// 4104 (this 7.0), 44.9 for 8192 x 4096 (40.5), 17.0 for 16384 x 512 (15.0).
template <typename T, int kV, bool kOne>
__global__ void __launch_bounds__(kNormThreads, (kV == 2 ? 3 : 2) - (sizeof(T) == 4 ? 1 : 0))
    add_rms_norm_kernel(const NormArgs a) {
  const int t = threadIdx.x;
  const int64_t row =
      kOne ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = kOne || row < a.T;
  const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
  const T *res = static_cast<const T *>(a.residual) + row * a.r_stride;
  pdl_wait();
  Chunk<T> rx[kV], rr[kV], rw[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    rx[v] = load_chunk(x, v, a.group, t, a.H, live);
    rr[v] = load_chunk(res, v, a.group, t, a.H, live && a.residual != nullptr);
  }
#pragma unroll
  for (int v = 0; v < kV; ++v)
    rw[v] = load_chunk(static_cast<const T *>(a.weight), v, a.group, t, a.H, true);
  pdl_launch_dependents();
  norm_row<T, kV, kOne>(a, rx, rr, rw, row, t, live);
}

struct NormBwdArgs {
  const void *dy, *dres, *sum, *weight;
  void *dx;
  float *part;  // [CTAs][H]
  int64_t dy_stride, s_stride, dx_stride;
  int T, H, group, rows, depth;
  float eps;
};

// CTA b's group g walks rows b * rows + g, + gridDim.x * rows, ... with `depth`
// - 1 rows on their way to its ring.  dy n is kept per column in registers, joined
// over the CTA's groups through shared memory at the end and left as one row of
// partials for the second kernel: a fixed order, so the sums do not change from
// run to run.
template <typename T, int kV>
__global__ void __launch_bounds__(kNormThreads) add_rms_norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float2 s_part[2][kNormThreads / 32];
  extern __shared__ uint4 s_ring[];
  // wide or fp32 rows leave no registers for the weight: it is read from L1
  constexpr bool kKeepWeight = kV == 2 && sizeof(T) == 2, kKeepProduct = kV == 2;
  const int sub = threadIdx.x / a.group, t = threadIdx.x - sub * a.group;
  const int warps = a.group >> 5, threads = blockDim.x;
  const T *dy = static_cast<const T *>(a.dy), *sm = static_cast<const T *>(a.sum);
  const T *dr = static_cast<const T *>(a.dres), *wt = static_cast<const T *>(a.weight);
  const uint32_t chunk = (uint32_t)threads * 16u * (uint32_t)Chunk<T>::kPieces;
  const uint32_t ring = smem_u32(s_ring) + threadIdx.x * 16u;
  pdl_wait();
  pdl_launch_dependents();
  auto weight = [&](int v) {
    Chunk<T> r;
#pragma unroll
    for (int i = 0; i < Chunk<T>::kPieces; ++i) {
      const int c = column<T>(v, i, a.group, t);
      r.a[i] = c < a.H ? __ldg(reinterpret_cast<const uint4 *>(wt + c)) : make_uint4(0, 0, 0, 0);
    }
    return r;
  };
  Chunk<T> rw[kV];
  pair_t acc[kV][4];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    if (kKeepWeight) rw[v] = weight(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[v][i] = make_pair(0.f, 0.f);
  }
  auto fill = [&](int64_t row, int slot) {
    if (row < a.T) {
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const uint32_t at = ring + (uint32_t)(slot * 3 * kV + v) * chunk;
        ring_fill(at, sm + row * a.s_stride, v, a.group, t, a.H, threads);
        ring_fill(at + kV * chunk, dy + row * a.dy_stride, v, a.group, t, a.H, threads);
        if (dr != nullptr)
          ring_fill(at + 2 * kV * chunk, dr + row * a.s_stride, v, a.group, t, a.H, threads);
      }
    }
    ring_commit();
  };
  const int64_t step = (int64_t)gridDim.x * a.rows;
  int64_t row = (int64_t)blockIdx.x * a.rows + sub, ahead = row;
  for (int i = 0; i + 1 < a.depth; ++i, ahead += step) fill(ahead, i);
  int slot = 0, next = a.depth - 1, buf = 0;
  const float inv_h = 1.0f / (float)a.H;
  // every group makes the same number of trips (the barrier is the CTA's)
  for (int64_t r0 = (int64_t)blockIdx.x * a.rows; r0 < a.T;
       r0 += step, row += step, ahead += step, buf ^= 1) {
    fill(ahead, next);  // of depth 1 the row itself
    ring_wait(a.depth - 1);
    const bool live = row < a.T;
    pair_t s[kV][4], d[kV][4], wd[kV][4];
    pair_t p0 = make_pair(0.f, 0.f), p1 = p0;  // sum s^2, sum w dy s
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const uint32_t at = ring + (uint32_t)(slot * 3 * kV + v) * chunk;
      pair_t w[4];
      to_pairs(ring_read<T>(at, v, a.group, t, a.H, threads, live), s[v]);
      to_pairs(ring_read<T>(at + kV * chunk, v, a.group, t, a.H, threads, live), d[v]);
      to_pairs(kKeepWeight ? rw[v] : weight(v), w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const pair_t x = mul2(w[i], d[v][i]);
        if (kKeepProduct) wd[v][i] = x;
        p0 = fma2(s[v][i], s[v][i], p0);
        p1 = fma2(x, s[v][i], p1);
      }
    }
    float2 p = make_float2(warp_sum(lo_of(p0) + hi_of(p0)), warp_sum(lo_of(p1) + hi_of(p1)));
    if ((threadIdx.x & 31) == 0) s_part[buf][threadIdx.x >> 5] = p;
    __syncthreads();  // two buffers: the next trip writes the other one
    p = make_float2(0.f, 0.f);
    for (int i = 0; i < warps; ++i) {
      const float2 o = s_part[buf][sub * warps + i];
      p.x += o.x;
      p.y += o.y;
    }
    const float r = 1.0f / sqrtf(p.x * inv_h + a.eps);
    // n mean(w dy n) = s m, m = r^2 sum(w dy s) / H
    const float m = p.y * inv_h * r * r;
    const pair_t r2 = make_pair(r, r), m2 = make_pair(-m, -m);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const uint32_t at = ring + (uint32_t)(slot * 3 * kV + 2 * kV + v) * chunk;
      pair_t e[4], o[4], w[4];
      if (!kKeepProduct) to_pairs(weight(v), w);
      to_pairs(ring_read<T>(at, v, a.group, t, a.H, threads, live && dr != nullptr), e);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const pair_t x = kKeepProduct ? wd[v][i] : mul2(w[i], d[v][i]);
        o[i] = fma2(r2, fma2(s[v][i], m2, x), e[i]);
        acc[v][i] = fma2(d[v][i], mul2(s[v][i], r2), acc[v][i]);
      }
      if (live) store_chunk(static_cast<T *>(a.dx) + row * a.dx_stride, o, v, a.group, t, a.H);
    }
    slot = slot + 1 == a.depth ? 0 : slot + 1;
    next = next + 1 == a.depth ? 0 : next + 1;
  }
  if (a.part == nullptr) return;
  // this thread's columns in the order of T's pieces, as fp32
  auto leave = [&](float *to) {
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int kPairs = 4 / Chunk<T>::kPieces;
        const int c = column<T>(v, i / kPairs, a.group, t) + i % kPairs * 2;
        if (c < a.H) *reinterpret_cast<float2 *>(to + c) = make_float2(lo_of(acc[v][i]), hi_of(acc[v][i]));
      }
  };
  float *out = a.part + (int64_t)blockIdx.x * a.H;
  if (a.rows == 1) return leave(out);
  float *s_dw = reinterpret_cast<float *>(s_ring);  // [rows][H]
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // no thread's ring is in use
  leave(s_dw + (int64_t)sub * a.H);
  __syncthreads();
  for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
    float w = 0.f;
    for (int g = 0; g < a.rows; ++g) w += s_dw[(int64_t)g * a.H + c];
    out[c] = w;
  }
}

// Column sums of `part` [n][ld] over its n rows, in a fixed order: 32 columns
// a CTA, 32 rows at a time (of which four in flight a thread).
__global__ void __launch_bounds__(1024)
    column_sum_kernel(const float *part, int n, int cols, int64_t ld, float *out) {
  __shared__ float s[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  pdl_wait();
  pdl_launch_dependents();
  float v = 0.f;
  if (c < cols) {
    int r = ry;
    for (; r + 96 < n; r += 128) {
      const float *p = part + (int64_t)r * ld + c;
      const float a0 = p[0], a1 = p[32 * ld], a2 = p[64 * ld], a3 = p[96 * ld];
      v += a0;
      v += a1;
      v += a2;
      v += a3;
    }
    for (; r < n; r += 32) v += part[(int64_t)r * ld + c];
  }
  s[ry][cx] = v;
  __syncthreads();
  // warp w: column w of the CTA, lane l its row lane l
  v = warp_sum(s[cx][ry]);
  const int col = blockIdx.x * 32 + ry;
  if (cx == 0 && col < cols) out[col] = v;
}

int round_up(int v, int m) { return (v + m - 1) / m * m; }

constexpr size_t kRingRoom = 200 * 1024;

// Rows of a ring: up to four where `per_sm` CTAs of an SM have room for at least
// two, else two of a CTA that has the SM to itself, or one.
int ring_depth(size_t row_bytes, int per_sm) {
  const int d = (int)(kRingRoom / per_sm / row_bytes);
  return d >= 2 ? std::min(d, 4) : (2 * row_bytes <= kRingRoom ? 2 : 1);
}

template <typename T>
cudaError_t norm_forward(NormArgs a, cudaStream_t s) {
  const int nch = a.H / 8;
  // Two chunks a thread, four in rows that 512 threads do not hold else, and where
  // long rows are coded (8192 x 7168 to E4M3: 72.3 us of two, 69.8 of four; 5120
  // columns 53.1 and 52.0, without codes 50.4 and 50.9).
  const int v = nch > 2 * kNormThreads || (a.q != nullptr && nch > 640) ? 4 : 2;
  a.group = round_up((nch + v - 1) / v, 32);
  // a warp's rows four to a CTA (65536 x 256: 31.6 us, of one 34.4)
  const int rows = a.group == 32 ? 4 : 1;
  const dim3 grid((unsigned)((a.T + rows - 1) / rows)), block((unsigned)a.group, (unsigned)rows);
  if (rows > 1) return launch_pdl(add_rms_norm_kernel<T, 2, false>, grid, block, 0, s, a);
  return v == 2 ? launch_pdl(add_rms_norm_kernel<T, 2, true>, grid, block, 0, s, a)
                : launch_pdl(add_rms_norm_kernel<T, 4, true>, grid, block, 0, s, a);
}

// Threads to a row, rows to a CTA and CTAs of the backward pass: two an SM while
// their registers fit (8192 x 4096: 49 us of two, 69 of one; 8192 x 7168, whose
// 448 threads do not fit twice: 86 of two, 80 of one).
void norm_bwd_shape(int T, int H, int sms, int *v, int *group, int *rows, int *per_sm, int *ctas) {
  const int nch = H / 8;
  *v = nch <= 2 * kNormThreads ? 2 : 4;
  *group = round_up((nch + *v - 1) / *v, 32);
  *rows = std::max(1, 256 / *group);
  *per_sm = *group * *rows <= 256 ? 2 : 1;
  *ctas = std::min((T + *rows - 1) / *rows, *per_sm * sms);
}

template <typename T, int kV>
cudaError_t launch_norm_bwd(const NormBwdArgs &a, dim3 grid, dim3 block, size_t smem,
                            cudaStream_t s) {
  if (smem > kRingRoom) return cudaErrorInvalidValue;
  static std::atomic<bool> allowed[64];
  const cudaError_t e = allow_smem(add_rms_norm_bwd_kernel<T, kV>, kRingRoom, allowed);
  return e != cudaSuccess
             ? e
             : launch_pdl(add_rms_norm_bwd_kernel<T, kV>, grid, block, smem, s, a);
}

template <typename T>
cudaError_t norm_backward(NormBwdArgs a, float *dweight, cudaStream_t s) {
  int v, per_sm, ctas;
  norm_bwd_shape(a.T, a.H, num_sms(), &v, &a.group, &a.rows, &per_sm, &ctas);
  const size_t row_bytes = (size_t)3 * v * a.group * a.rows * 8 * sizeof(T);
  a.depth = ring_depth(row_bytes, per_sm);
  const size_t smem = std::max((size_t)a.depth * row_bytes,
                               a.rows > 1 ? (size_t)a.rows * a.H * 4 : 0);
  const dim3 grid((unsigned)ctas), block((unsigned)(a.group * a.rows));
  cudaError_t e = v == 2 ? launch_norm_bwd<T, 2>(a, grid, block, smem, s)
                         : launch_norm_bwd<T, 4>(a, grid, block, smem, s);
  if (e == cudaSuccess && dweight != nullptr)
    e = launch_column_sum(a.part, ctas, a.H, a.H, dweight, s);
  return e;
}

}  // namespace

cudaError_t launch_column_sum(const float *part, int n, int cols, int64_t ld, float *out,
                              cudaStream_t s) {
  return launch_pdl(column_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, s, part, n,
                    cols, ld, out);
}

size_t norm_bwd_part_bytes(const moe_norm_desc_t &d) {
  int v, group, rows, per_sm, ctas;
  norm_bwd_shape(d.T, d.H, kRouteSizingSms, &v, &group, &rows, &per_sm, &ctas);
  return (size_t)ctas * d.H * 4;
}

cudaError_t launch_add_rms_norm(const moe_norm_desc_t &d, const void *x, const void *residual,
                                const void *weight, void *residual_out, void *y, uint8_t *q,
                                int8_t *scale, cudaStream_t s) {
  NormArgs a = {x, residual, weight, residual_out, y, q, scale, d.x_stride, d.residual_stride,
                d.y_stride, d.T, d.H, 0, d.eps, 1.0f / (float)d.H};
  switch (d.dtype) {
    case MOE_DTYPE_BF16: return norm_forward<__nv_bfloat16>(a, s);
    case MOE_DTYPE_FP16: return norm_forward<__half>(a, s);
    default: return norm_forward<float>(a, s);
  }
}

cudaError_t launch_add_rms_norm_backward(const moe_norm_desc_t &d, const void *dy, const void *dres,
                                         const void *sum, const void *weight, void *dx,
                                         float *dweight, float *part, cudaStream_t s) {
  NormBwdArgs a = {dy, dres, sum, weight, dx, dweight != nullptr ? part : nullptr, d.y_stride,
                   d.residual_stride, d.x_stride, d.T, d.H, 0, 0, 0, d.eps};
  switch (d.dtype) {
    case MOE_DTYPE_BF16: return norm_backward<__nv_bfloat16>(a, dweight, s);
    case MOE_DTYPE_FP16: return norm_backward<__half>(a, dweight, s);
    default: return norm_backward<float>(a, dweight, s);
  }
}

}  // namespace moe
