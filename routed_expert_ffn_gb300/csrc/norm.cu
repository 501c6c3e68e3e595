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
// once, and the mean costs one shuffle reduction and one exchange through
// shared memory.
#include <cuda_fp8.h>

#include <algorithm>

#include "moe_internal.cuh"

namespace moe {

namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormBwdThreads = 512;

// 8 consecutive elements as loaded: 16 bytes (bf16, fp16) or 32 (fp32).
template <typename T>
struct Raw8 {
  uint4 a[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T *p) {
  Raw8<T> r;
  // not the read-only path: outputs may overlay inputs row for row
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.a[i].x), "=r"(r.a[i].y), "=r"(r.a[i].z), "=r"(r.a[i].w)
                 : "l"(reinterpret_cast<const uint4 *>(p) + i));
  return r;
}
template <typename T>
__device__ __forceinline__ Raw8<T> zero_raw() {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.a[i] = make_uint4(0, 0, 0, 0);
  return r;
}

__device__ __forceinline__ void to_float(const Raw8<__nv_bfloat16> &r, float (&f)[8]) {
  const uint32_t w[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void to_float(const Raw8<__half> &r, float (&f)[8]) {
  const uint32_t w[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void to_float(const Raw8<float> &r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(r.a[i].x);
    f[4 * i + 1] = __uint_as_float(r.a[i].y);
    f[4 * i + 2] = __uint_as_float(r.a[i].z);
    f[4 * i + 3] = __uint_as_float(r.a[i].w);
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                             pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(__half *p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The power-of-two exponent of a block of 8-bit values with absolute maximum
// `amax`: the least s with amax <= 448 * 2^s (448 = 1.75 * 2^8, the largest
// E4M3 value), at least -126; 0 for a block of zeros.
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
  int T, H, group, rows;  // threads to a row, rows to a CTA
  float eps;
};

// kV: chunks of 8 elements a thread.  A CTA takes `rows` rows, `group` threads
// (whole warps) to each; thread i of a group holds chunks i, i + group, ..., so
// the 128 elements that share an 8-bit scale lie in 16 neighbouring lanes.
template <typename T, int kV>
__global__ void __launch_bounds__(kV == 4 ? kNormMaxThreads / 2 : kNormMaxThreads)
    add_rms_norm_kernel(const NormArgs a) {
  __shared__ float s_part[kNormMaxThreads / 32];
  const int sub = threadIdx.x / a.group, t = threadIdx.x - sub * a.group;
  const int64_t row = (int64_t)blockIdx.x * a.rows + sub;
  const bool live = row < a.T;
  const int nch = a.H >> 3;
  const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
  const T *res = static_cast<const T *>(a.residual) + row * a.r_stride;
  pdl_wait();
  Raw8<T> rx[kV], rr[kV], rw[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = t + v * a.group;
    const bool in = live && c < nch;
    rx[v] = in ? load_raw(x + c * 8) : zero_raw<T>();
    rr[v] = in && a.residual != nullptr ? load_raw(res + c * 8) : zero_raw<T>();
  }
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = t + v * a.group;
    rw[v] = c < nch ? load_raw(static_cast<const T *>(a.weight) + c * 8) : zero_raw<T>();
  }
  pdl_launch_dependents();
  float s[kV][8];
  float sq = 0.f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    float r[8];
    to_float(rx[v], s[v]);
    to_float(rr[v], r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[v][i] += r[i];
      sq = fmaf(s[v][i], s[v][i], sq);
    }
    const int c = t + v * a.group;
    if (a.residual_out != nullptr && live && c < nch)
      store8(static_cast<T *>(a.residual_out) + row * a.r_stride + c * 8, s[v]);
  }
  sq = warp_sum(sq);
  const int warps = a.group >> 5;
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = sq;
  __syncthreads();
  float sum = 0.f;
  for (int i = 0; i < warps; ++i) sum += s_part[sub * warps + i];
  const float rstd = 1.0f / sqrtf(sum / (float)a.H + a.eps);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = t + v * a.group;
    const bool in = live && c < nch;
    float w[8], y[8];
    to_float(rw[v], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = s[v][i] * rstd * w[i];
    if (a.y != nullptr && in) store8(static_cast<T *>(a.y) + row * a.y_stride + c * 8, y);
    if (a.q != nullptr) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int e = block_exp(m);
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      if (in) {
        uint32_t w2[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = make_float2(y[2 * i] * inv, y[2 * i + 1] * inv);
          w2[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)
                        << (16 * (i & 1));
        }
        *reinterpret_cast<uint2 *>(a.q + row * a.H + c * 8) = make_uint2(w2[0], w2[1]);
        if ((c & 15) == 0) a.scale[row * ((a.H + 127) >> 7) + (c >> 4)] = (int8_t)e;
      }
    }
  }
}

struct NormBwdArgs {
  const void *dy, *dres, *sum, *weight;
  void *dx;
  float *part;  // [CTAs][H]
  int64_t dy_stride, s_stride, dx_stride;
  int T, H, group, rows;
  float eps;
};

// Persistent: CTA b's group g walks rows b * rows + g, + gridDim.x * rows, ...
// with the next row's loads in flight while this row is reduced.  dy n is kept
// per column in registers, joined over the CTA's groups through shared memory
// at the end and left as one row of partials for the second kernel: a fixed
// order, so the sums do not change from run to run.
template <typename T, int kV>
__global__ void __launch_bounds__(kNormBwdThreads) add_rms_norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float2 s_part[2][kNormBwdThreads / 32];
  extern __shared__ float s_dw[];  // [rows][H] when rows > 1
  const int sub = threadIdx.x / a.group, t = threadIdx.x - sub * a.group;
  const int nch = a.H >> 3, warps = a.group >> 5;
  const T *dy = static_cast<const T *>(a.dy), *sm = static_cast<const T *>(a.sum);
  const T *dr = static_cast<const T *>(a.dres);
  pdl_wait();
  // Two chunks of 16 bits leave room for the next row's loads and the weight
  // in registers; wider rows or types load each row when its turn comes.
  constexpr bool kAhead = kV == 2 && sizeof(T) == 2;
  const T *wt = static_cast<const T *>(a.weight);
  Raw8<T> rw[kV];
  float acc[kV][8];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = t + v * a.group;
    if (kAhead) rw[v] = c < nch ? load_raw(wt + c * 8) : zero_raw<T>();
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.f;
  }
  pdl_launch_dependents();
  auto fetch = [&](Raw8<T>(&to)[kV], const T *from, int64_t row, int64_t stride) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = t + v * a.group;
      to[v] = from != nullptr && row < a.T && c < nch ? load_raw(from + row * stride + c * 8)
                                                      : zero_raw<T>();
    }
  };
  auto weight = [&](int v, float(&w)[8]) {
    const int c = t + v * a.group;
    if (kAhead) {
      to_float(rw[v], w);
    } else {
      Raw8<T> r = zero_raw<T>();
      if (c < nch)
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
          r.a[i] = __ldg(reinterpret_cast<const uint4 *>(wt + c * 8) + i);
      to_float(r, w);
    }
  };
  const int64_t step = (int64_t)gridDim.x * a.rows;
  int64_t row = (int64_t)blockIdx.x * a.rows + sub;
  Raw8<T> ns[kV], nd[kV], nr[kV];
  if (kAhead) {
    fetch(ns, sm, row, a.s_stride);
    fetch(nd, dy, row, a.dy_stride);
    fetch(nr, dr, row, a.s_stride);
  }
  const float inv_h = 1.0f / (float)a.H;
  // every group makes the same number of trips (the barrier is the CTA's)
  const int64_t first = (int64_t)blockIdx.x * a.rows;
  int buf = 0;
  for (int64_t r0 = first; r0 < a.T; r0 += step, row += step, buf ^= 1) {
    Raw8<T> cs[kV], cd[kV], cr[kV];
    if (kAhead) {
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        cs[v] = ns[v];
        cd[v] = nd[v];
        cr[v] = nr[v];
      }
      fetch(ns, sm, row + step, a.s_stride);
      fetch(nd, dy, row + step, a.dy_stride);
      fetch(nr, dr, row + step, a.s_stride);
    } else {
      fetch(cs, sm, row, a.s_stride);
      fetch(cd, dy, row, a.dy_stride);
    }
    float2 p = make_float2(0.f, 0.f);  // sum s^2, sum w dy s
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      float s[8], d[8], w[8];
      to_float(cs[v], s);
      to_float(cd[v], d);
      weight(v, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p.x = fmaf(s[i], s[i], p.x);
        p.y = fmaf(w[i] * d[i], s[i], p.y);
      }
    }
    p.x = warp_sum(p.x);
    p.y = warp_sum(p.y);
    if ((threadIdx.x & 31) == 0) s_part[buf][threadIdx.x >> 5] = p;
    __syncthreads();  // two buffers: the next trip writes the other one
    float2 q = make_float2(0.f, 0.f);
    for (int i = 0; i < warps; ++i) {
      const float2 o = s_part[buf][sub * warps + i];
      q.x += o.x;
      q.y += o.y;
    }
    const float r = 1.0f / sqrtf(q.x * inv_h + a.eps);
    const float mr = q.y * inv_h * r * r;  // times s: n mean(w dy n) = s r * (r sum(w dy s) / H)
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = t + v * a.group;
      const bool in = row < a.T && c < nch;
      float s[8], d[8], w[8], e[8], o[8];
      to_float(cs[v], s);
      to_float(cd[v], d);
      weight(v, w);
      if (!kAhead)
        cr[v] = in && dr != nullptr ? load_raw(dr + row * a.s_stride + c * 8) : zero_raw<T>();
      to_float(cr[v], e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = fmaf(r, w[i] * d[i] - s[i] * mr, e[i]);
        acc[v][i] = fmaf(d[i], s[i] * r, acc[v][i]);
      }
      if (in) store8(static_cast<T *>(a.dx) + row * a.dx_stride + c * 8, o);
    }
  }
  if (a.part == nullptr) return;
  float *out = a.part + (int64_t)blockIdx.x * a.H;
  if (a.rows > 1) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = t + v * a.group;
      if (c < nch) store8(s_dw + (int64_t)sub * a.H + c * 8, acc[v]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      float w = 0.f;
      for (int g = 0; g < a.rows; ++g) w += s_dw[(int64_t)g * a.H + c];
      out[c] = w;
    }
  } else {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = t + v * a.group;
      if (c < nch) store8(out + c * 8, acc[v]);
    }
  }
}

// Column sums of `part` [n][ld] over its n rows, in a fixed order: 32 columns
// a CTA, 8 rows at a time.
__global__ void __launch_bounds__(256)
    column_sum_kernel(const float *part, int n, int cols, int64_t ld, float *out, int accumulate) {
  __shared__ float s[8][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  pdl_wait();
  pdl_launch_dependents();
  float v = 0.f;
  if (c < cols)
    for (int r = ry; r < n; r += 8) v += part[(int64_t)r * ld + c];
  s[ry][cx] = v;
  __syncthreads();
  if (ry == 0 && c < cols) {
    for (int i = 1; i < 8; ++i) v += s[i][cx];
    out[c] = accumulate ? out[c] + v : v;
  }
}

int round_up(int v, int m) { return (v + m - 1) / m * m; }

template <typename T>
cudaError_t norm_forward(NormArgs a, cudaStream_t s) {
  const int nch = a.H / 8;
  // Few rows: latency counts, one chunk a thread where 1024 threads hold the
  // row.  Many rows: four chunks a thread keep more loads in flight for each
  // barrier.
  const bool few = a.T <= 2 * num_sms();
  int v = few ? (nch <= kNormMaxThreads ? 1 : 2) : 4;
  if (nch <= 32) v = 1;
  a.group = round_up((nch + v - 1) / v, 32);
  a.rows = few ? 1 : std::max(1, 256 / a.group);
  const dim3 grid((unsigned)((a.T + a.rows - 1) / a.rows)), block((unsigned)(a.group * a.rows));
  switch (v) {
    case 1: return launch_pdl(add_rms_norm_kernel<T, 1>, grid, block, 0, s, a);
    case 2: return launch_pdl(add_rms_norm_kernel<T, 2>, grid, block, 0, s, a);
    default: return launch_pdl(add_rms_norm_kernel<T, 4>, grid, block, 0, s, a);
  }
}

// Threads to a row, rows to a CTA and CTAs of the backward pass.
void norm_bwd_shape(int T, int H, int sms, int *v, int *group, int *rows, int *ctas) {
  const int nch = H / 8;
  *v = nch <= 2 * kNormBwdThreads ? 2 : 4;
  *group = round_up((nch + *v - 1) / *v, 32);
  *rows = std::max(1, 256 / *group);
  // the joined column sums of the CTA's groups go through shared memory
  while (*rows > 1 && (size_t)*rows * H * 4 > 48 * 1024) *rows /= 2;
  *ctas = std::min((T + *rows - 1) / *rows, 2 * sms);
}

template <typename T>
cudaError_t norm_backward(NormBwdArgs a, float *dweight, cudaStream_t s) {
  int v, ctas;
  norm_bwd_shape(a.T, a.H, num_sms(), &v, &a.group, &a.rows, &ctas);
  const size_t smem = a.rows > 1 ? (size_t)a.rows * a.H * 4 : 0;
  const dim3 grid((unsigned)ctas), block((unsigned)(a.group * a.rows));
  cudaError_t e = v == 2 ? launch_pdl(add_rms_norm_bwd_kernel<T, 2>, grid, block, smem, s, a)
                         : launch_pdl(add_rms_norm_bwd_kernel<T, 4>, grid, block, smem, s, a);
  if (e == cudaSuccess && dweight != nullptr)
    e = launch_column_sum(a.part, ctas, a.H, a.H, dweight, 0, s);
  return e;
}

}  // namespace

cudaError_t launch_column_sum(const float *part, int n, int cols, int64_t ld, float *out,
                              int accumulate, cudaStream_t s) {
  return launch_pdl(column_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, s, part, n,
                    cols, ld, out, accumulate);
}

size_t norm_bwd_part_bytes(const moe_norm_desc_t &d) {
  int v, group, rows, ctas;
  norm_bwd_shape(d.T, d.H, kRouteSizingSms, &v, &group, &rows, &ctas);
  return (size_t)ctas * d.H * 4;
}

cudaError_t launch_add_rms_norm(const moe_norm_desc_t &d, const void *x, const void *residual,
                                const void *weight, void *residual_out, void *y, uint8_t *q,
                                int8_t *scale, cudaStream_t s) {
  NormArgs a = {x, residual, weight, residual_out, y, q, scale, d.x_stride, d.residual_stride,
                d.y_stride, d.T, d.H, 0, 0, d.eps};
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
                   d.residual_stride, d.x_stride, d.T, d.H, 0, 0, d.eps};
  switch (d.dtype) {
    case MOE_DTYPE_BF16: return norm_backward<__nv_bfloat16>(a, dweight, s);
    case MOE_DTYPE_FP16: return norm_backward<__half>(a, dweight, s);
    default: return norm_backward<float>(a, dweight, s);
  }
}

}  // namespace moe
