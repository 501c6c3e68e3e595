// C ABI of the dense half of a transformer block: argument validation and the
// sequence of launches of each call.  Declarations and the meaning of every
// argument are in include/moe.h.
#include <stdint.h>

#include <initializer_list>

#include "dense.cuh"

namespace moe {

namespace {

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A workspace of at least `need` bytes, aligned to 256.
moe_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// Whether `out` is at the address of one of `others` that the call still reads, or
// writes too (null: no argument).
bool lies_on(const void *out, std::initializer_list<const void *> others) {
  for (const void *p : others)
    if (out != nullptr && out == p) return true;
  return false;
}

// A row stride in elements: 0 (dense) becomes `cols`; otherwise at least
// `cols` and a multiple of `mult`.
bool fix_stride(int64_t *stride, int64_t cols, int mult) {
  if (*stride == 0) *stride = cols;
  return *stride >= cols && *stride % mult == 0 && *stride < ((int64_t)1 << 36);
}

// A validated copy of the descriptor with its strides filled in.
moe_status_t norm_desc(const moe_norm_desc_t *in, moe_norm_desc_t *d) {
  if (in == nullptr) return MOE_ERR_INVALID_ARG;
  *d = *in;
  if (d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_FP16 && d->dtype != MOE_DTYPE_FP32)
    return MOE_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (d->T < 0 || d->T > kMaxT || d->H < 8 || d->H > 16384 || d->H % 8 != 0)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!fix_stride(&d->x_stride, d->H, 8) || !fix_stride(&d->residual_stride, d->H, 8) ||
      !fix_stride(&d->y_stride, d->H, 8))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status_t linear_desc(const moe_linear_desc_t *in, moe_linear_desc_t *d) {
  if (in == nullptr) return MOE_ERR_INVALID_ARG;
  *d = *in;
  const bool e4m3 = d->dtype == MOE_DTYPE_E4M3;
  if (d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_FP16 && !e4m3) return MOE_ERR_INVALID_ARG;
  if (d->out_dtype != (e4m3 ? (int32_t)MOE_DTYPE_BF16 : d->dtype) &&
      d->out_dtype != MOE_DTYPE_FP32)
    return MOE_ERR_INVALID_ARG;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  const int32_t most = 1 << 18;
  if (d->T < 0 || d->T > kMaxT || d->N < 8 || d->N > most || d->N % 8 != 0 || d->K < 8 ||
      d->K > most || d->K % (e4m3 ? 16 : 8) != 0)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!fix_stride(&d->x_stride, d->K, e4m3 ? 16 : 8) || !fix_stride(&d->residual_stride, d->N, 8) ||
      !fix_stride(&d->y_stride, d->N, 8))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

size_t pad(size_t n) { return (n + 1023) / 1024 * 1024; }

// After the status block: dz and the column partials of the gradient.
struct LinearWs {
  size_t dz, part, total;
};
LinearWs linear_ws(const moe_linear_desc_t &d) {
  LinearWs w;
  w.dz = w.part = w.total = kStatusPad;
  if (d.dtype == MOE_DTYPE_E4M3) return w;  // no gradient
  w.part += d.act == MOE_ACT_NONE ? 0 : pad((size_t)d.T * d.N * 2);
  w.total = w.part + pad((size_t)act_grad_slices(d.T, d.N) * d.N * 4);
  return w;
}

moe_status_t ffn_desc(const moe_ffn_desc_t *d) {
  if (d == nullptr) return MOE_ERR_INVALID_ARG;
  if (d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_FP16) return MOE_ERR_INVALID_ARG;
  const int32_t most = 1 << 17;
  if (d->T < 0 || d->T > kMaxT || d->H < 8 || d->H > most || d->H % 8 != 0 || d->I < 8 ||
      d->I > most || d->I % 8 != 0)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

struct FfnWs {
  size_t h, dgu, total;
};
FfnWs ffn_ws(const moe_ffn_desc_t &d) {
  FfnWs w;
  w.h = kStatusPad;
  w.dgu = w.h + pad((size_t)d.T * d.I * 2);
  w.total = w.dgu + pad((size_t)d.T * d.I * 4);
  return w;
}

uint8_t *at(void *ws, size_t off) { return static_cast<uint8_t *>(ws) + off; }

// D[M,N] = A B with fp32 accumulators: the fields every product shares.
DenseGemm product(int M, int N, int K, int dtype, const void *a, int64_t lda, bool a_mn,
                  const void *b, int64_t ldb, bool b_mn, void *d, int64_t ldd, int out_dtype,
                  void *ws) {
  DenseGemm g = {};
  g.M = M;
  g.N = N;
  g.K = K;
  g.epi = kEpiLinear;
  g.dtype = dtype;
  g.out_dtype = out_dtype;
  g.act = MOE_ACT_NONE;
  g.a = a;
  g.lda = lda;
  g.a_mn = a_mn;
  g.b = b;
  g.ldb = ldb;
  g.b_mn = b_mn;
  g.d = d;
  g.ldd = ldd;
  g.status = static_cast<uint32_t *>(ws);
  return g;
}

// A forward product by the kernel that is estimated to take less: the one for
// few rows reads W at the rate of HBM but X once for each 128 columns; the
// tiled one wants 256 rows for each 64 to 256 columns.  4096 x 4096 (us, few
// rows against tiled): 32 rows 9.6 and 14.1, 128 rows 14.9 and 14.8, 192 rows
// 19.0 and 14.7.  preact and saved are stored by the tiled kernel only.
bool by_few_rows(const DenseGemm &g) {
  return g.M <= kSmallRows && g.preact == nullptr && g.saved == nullptr &&
         dense_small_us(g) <= dense_pair_us(g);
}
cudaError_t forward(const DenseGemm &g, cudaStream_t s) {
  return by_few_rows(g) ? launch_dense_small(g, s) : launch_dense_pair(g, s);
}

constexpr int kGradSmallRows = 64;
constexpr float kLaunchUs = 4.f;

// The products of a gradient, dx first where there is one (`with_dx`).
// In one launch with the others dx's tiles may be the longest, as deep as W has
// rows: of few rows it is a launch of the kernel for few rows where that is estimated
// to save more than a launch takes.  16 rows of 6336 x 400: 23.8 us in one, 12.0
// apart; of 2368 x 4600 19.7 and 20.6; 128 rows of 4096 x 4096 24.4 and 30.0.
cudaError_t gradients(const DenseGemm *g, int n, bool with_dx, cudaStream_t s) {
  if (!with_dx || g[0].M > kGradSmallRows) return launch_dense_multi(g, n, s);
  const float apart = dense_small_us(g[0]) + (n > 1 ? dense_multi_us(g + 1, n - 1) + kLaunchUs : 0.f);
  if (apart >= dense_multi_us(g, n)) return launch_dense_multi(g, n, s);
  const cudaError_t e = launch_dense_small(g[0], s);
  return e != cudaSuccess || n == 1 ? e : launch_dense_multi(g + 1, n - 1, s);
}

// dw[M,N] (+)= a^T b over T rows.
DenseGemm weight_grad(int M, int N, int T, int dtype, const void *a, int64_t lda, const void *b,
                      int64_t ldb, void *dw, int dw_dtype, int accumulate, void *ws) {
  DenseGemm g = product(M, N, T, dtype, a, lda, true, b, ldb, true, dw, N, dw_dtype, ws);
  if (accumulate) {
    g.residual = dw;
    g.ldr = N;
  }
  return g;
}

// The gradient of a weight over no rows: zeros, or what is accumulated.
cudaError_t no_rows(void *dw, int64_t n, int dw_dtype, int accumulate, cudaStream_t s) {
  if (dw == nullptr || accumulate) return cudaSuccess;
  return cudaMemsetAsync(dw, 0, (size_t)n * (dw_dtype == MOE_DTYPE_FP32 ? 4 : 2), s);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_norm_workspace_size(const moe_norm_desc_t *in) {
  moe_norm_desc_t d;
  if (norm_desc(in, &d) != MOE_OK) return 0;
  return kStatusPad + norm_bwd_part_bytes(d);
}

moe_status_t moe_add_rms_norm(const moe_norm_desc_t *in, const void *x, const void *residual,
                              const void *weight, void *residual_out, void *y, void *y_q,
                              int8_t *scale_exp, moe_stream_t stream) {
  moe_norm_desc_t d;
  moe_status_t st = norm_desc(in, &d);
  if (st != MOE_OK) return st;
  if (d.T == 0) return MOE_OK;  // empty tensors may have no address
  if (!ok_ptr(x) || !ok_opt(residual) || !ok_ptr(weight) || !ok_opt(residual_out) || !ok_opt(y) ||
      !ok_opt(y_q))
    return MOE_ERR_INVALID_ARG;
  if ((y_q == nullptr) != (scale_exp == nullptr) || (y == nullptr && y_q == nullptr))
    return MOE_ERR_INVALID_ARG;
  // in place means row for row
  if (residual_out == x && d.residual_stride != d.x_stride) return MOE_ERR_INVALID_ARG;
  if (y == x && d.y_stride != d.x_stride) return MOE_ERR_INVALID_ARG;
  if (y != nullptr && y == residual && d.y_stride != d.residual_stride) return MOE_ERR_INVALID_ARG;
  if (lies_on(y_q, {x, residual, residual_out, y})) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  return cuda_status(launch_add_rms_norm(d, x, residual, weight, residual_out, y,
                                         static_cast<uint8_t *>(y_q), scale_exp,
                                         (cudaStream_t)stream));
}

moe_status_t moe_add_rms_norm_backward(const moe_norm_desc_t *in, const void *dy,
                                       const void *dresidual, const void *sum, const void *weight,
                                       void *dx, float *dweight, void *workspace, size_t ws_bytes,
                                       moe_stream_t stream) {
  moe_norm_desc_t d;
  moe_status_t st = norm_desc(in, &d);
  if (st != MOE_OK) return st;
  if ((st = check_ws(workspace, ws_bytes, kStatusPad + norm_bwd_part_bytes(d))) != MOE_OK) return st;
  float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kStatusPad);
  if (!ok_opt(dweight)) return MOE_ERR_INVALID_ARG;
  if (d.T == 0) {
    if (dweight == nullptr) return MOE_OK;
    if ((st = check_device()) != MOE_OK) return st;
    return cuda_status(launch_column_sum(part, 0, d.H, d.H, dweight, (cudaStream_t)stream));
  }
  if (!ok_ptr(dy) || !ok_opt(dresidual) || !ok_ptr(sum) || !ok_ptr(weight) || !ok_ptr(dx))
    return MOE_ERR_INVALID_ARG;
  if (dx == dy && d.x_stride != d.y_stride) return MOE_ERR_INVALID_ARG;
  if (dx == dresidual && d.x_stride != d.residual_stride) return MOE_ERR_INVALID_ARG;
  if (dx == sum) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  return cuda_status(launch_add_rms_norm_backward(d, dy, dresidual, sum, weight, dx, dweight, part,
                                                  (cudaStream_t)stream));
}

size_t moe_linear_workspace_size(const moe_linear_desc_t *in) {
  moe_linear_desc_t d;
  return linear_desc(in, &d) == MOE_OK ? linear_ws(d).total : 0;
}

moe_status_t moe_linear_plan(const moe_linear_desc_t *in, int32_t with_preact,
                             moe_linear_plan_t *plan) {
  moe_linear_desc_t d;
  moe_status_t st = linear_desc(in, &d);
  if (st != MOE_OK) return st;
  if (plan == nullptr || d.T == 0) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  DenseGemm g = product(d.T, d.N, d.K, d.dtype, nullptr, d.x_stride, false, nullptr, d.K, false,
                        nullptr, d.y_stride, d.out_dtype, nullptr);
  g.act = d.act;
  float preact;
  if (with_preact) g.preact = &preact;
  const bool few = by_few_rows(g);
  const DensePlan p = few ? dense_small_plan(g) : dense_pair_plan(g);
  if (p.us == 0.f) return MOE_ERR_CUDA;
  plan->kernel = few ? MOE_LINEAR_FEW_ROWS : MOE_LINEAR_TILES;
  plan->tile_rows = p.rows;
  plan->tile_cols = p.cols;
  plan->split = p.split;
  return MOE_OK;
}

moe_status_t moe_linear(const moe_linear_desc_t *in, const void *x, const int8_t *x_scale,
                        const void *w, const int8_t *w_scale, const void *bias,
                        const void *residual, float *preact, void *y, void *workspace,
                        size_t ws_bytes, moe_stream_t stream) {
  moe_linear_desc_t d;
  moe_status_t st = linear_desc(in, &d);
  if (st != MOE_OK) return st;
  const LinearWs L = linear_ws(d);
  if ((st = check_ws(workspace, ws_bytes, L.total)) != MOE_OK) return st;
  if (d.T == 0) return MOE_OK;  // empty tensors may have no address
  const bool e4m3 = d.dtype == MOE_DTYPE_E4M3;
  if (!ok_ptr(x) || !ok_ptr(w) || !ok_opt(bias) || !ok_opt(residual) || !ok_opt(preact) ||
      !ok_ptr(y))
    return MOE_ERR_INVALID_ARG;
  if ((x_scale != nullptr) != e4m3 || (w_scale != nullptr) != e4m3) return MOE_ERR_INVALID_ARG;
  if (e4m3 && preact != nullptr) return MOE_ERR_INVALID_ARG;
  if (residual == y && d.residual_stride != d.y_stride) return MOE_ERR_INVALID_ARG;
  if (y == x || y == w || lies_on(preact, {x, w, bias, y})) return MOE_ERR_INVALID_ARG;
  if (preact != nullptr && preact == residual &&
      (d.out_dtype != MOE_DTYPE_FP32 || d.residual_stride != d.N))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  DenseGemm g = product(d.T, d.N, d.K, d.dtype, x, d.x_stride, false, w, d.K, false, y, d.y_stride,
                        d.out_dtype, workspace);
  g.a_scale = x_scale;
  g.b_scale = w_scale;
  g.act = d.act;
  g.bias = bias;
  g.residual = residual;
  g.ldr = d.residual_stride;
  g.preact = preact;
  return cuda_status(forward(g, s));
}

moe_status_t moe_linear_backward(const moe_linear_desc_t *in, const void *dy, const void *x,
                                 const void *w, const float *preact, void *dx, void *dw,
                                 int32_t dw_dtype, float *dbias, int32_t accumulate,
                                 void *workspace, size_t ws_bytes, moe_stream_t stream) {
  moe_linear_desc_t d;
  moe_status_t st = linear_desc(in, &d);
  if (st != MOE_OK) return st;
  if (d.dtype == MOE_DTYPE_E4M3) return MOE_ERR_INVALID_ARG;
  if (dw_dtype != d.dtype && dw_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  const LinearWs L = linear_ws(d);
  if ((st = check_ws(workspace, ws_bytes, L.total)) != MOE_OK) return st;
  const bool act = d.act != MOE_ACT_NONE;
  if (!ok_opt(dw) || !ok_opt(dbias)) return MOE_ERR_INVALID_ARG;
  if (d.T > 0) {
    if (!ok_ptr(dy) || !ok_opt(dx) || (act ? !ok_ptr(preact) : preact != nullptr))
      return MOE_ERR_INVALID_ARG;
    if ((dx != nullptr && !ok_ptr(w)) || (dw != nullptr && !ok_ptr(x))) return MOE_ERR_INVALID_ARG;
    if (dx != nullptr && (dx == dy || dx == x || dx == w)) return MOE_ERR_INVALID_ARG;
    // dx and dw are of one launch, after that of dbias; with an activation neither reads dy
    const void *w_read = dx != nullptr ? w : nullptr, *x_read = dw != nullptr ? x : nullptr;
    if (lies_on(dw, {x, w_read, dx, act ? nullptr : dy}) ||
        lies_on(dbias, {dy, preact, x_read, w_read, dx, dw}))
      return MOE_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != MOE_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  float *part = reinterpret_cast<float *>(at(workspace, L.part));
  const void *dz = act ? at(workspace, L.dz) : dy;
  const int64_t ldz = act ? d.N : d.y_stride;
  if (d.T == 0) {
    cudaError_t e = no_rows(dbias, d.N, MOE_DTYPE_FP32, accumulate, s);
    if (e == cudaSuccess) e = no_rows(dw, (int64_t)d.N * d.K, dw_dtype, accumulate, s);
    return cuda_status(e);
  }
  cudaError_t e = cudaSuccess;
  if (dbias != nullptr || (act && (dx != nullptr || dw != nullptr)))
    e = launch_act_grad(dy, d.y_stride, preact, d.T, d.N, d.act, d.dtype,
                        dx != nullptr || dw != nullptr ? at(workspace, L.dz) : nullptr, part,
                        static_cast<uint32_t *>(workspace) + kBiasCounterWord, dbias, accumulate, s);
  DenseGemm g[2];
  int n = 0;
  if (dx != nullptr)
    g[n++] = product(d.T, d.K, d.N, d.dtype, dz, ldz, false, w, d.K, true, dx, d.x_stride, d.dtype,
                     workspace);
  if (dw != nullptr)
    g[n++] = weight_grad(d.N, d.K, d.T, d.dtype, dz, ldz, x, d.x_stride, dw, dw_dtype, accumulate,
                         workspace);
  if (e == cudaSuccess && n > 0) e = gradients(g, n, dx != nullptr, s);
  return cuda_status(e);
}

size_t moe_gated_ffn_workspace_size(const moe_ffn_desc_t *d) {
  return ffn_desc(d) == MOE_OK ? ffn_ws(*d).total : 0;
}

moe_status_t moe_gated_ffn(const moe_ffn_desc_t *d, const void *x, const void *w13, const void *w2,
                           const void *residual, float *saved, void *y, void *workspace,
                           size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = ffn_desc(d);
  if (st != MOE_OK) return st;
  const FfnWs L = ffn_ws(*d);
  if ((st = check_ws(workspace, ws_bytes, L.total)) != MOE_OK) return st;
  if (d->T == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(w13) || !ok_ptr(w2) || !ok_opt(residual) || !ok_opt(saved) ||
      !ok_ptr(y))
    return MOE_ERR_INVALID_ARG;
  if (y == x || y == w13 || y == w2) return MOE_ERR_INVALID_ARG;
  if (lies_on(saved, {x, w13, w2, residual, y})) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  DenseGemm up = product(d->T, d->I, d->H, d->dtype, x, d->H, false, w13, d->H, false,
                         at(workspace, L.h), d->I, d->dtype, workspace);
  up.epi = kEpiGated;
  up.saved = saved;
  cudaError_t e = forward(up, s);
  DenseGemm down = product(d->T, d->H, d->I, d->dtype, at(workspace, L.h), d->I, false, w2, d->I,
                           false, y, d->H, d->dtype, workspace);
  down.residual = residual;
  down.ldr = d->H;
  if (e == cudaSuccess) e = forward(down, s);
  return cuda_status(e);
}

moe_status_t moe_gated_ffn_backward(const moe_ffn_desc_t *d, const void *dy, const void *x,
                                    const void *w13, const void *w2, const float *saved, void *dx,
                                    void *dw13, void *dw2, int32_t dw_dtype, int32_t accumulate,
                                    void *workspace, size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = ffn_desc(d);
  if (st != MOE_OK) return st;
  if (dw_dtype != d->dtype && dw_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  const FfnWs L = ffn_ws(*d);
  if ((st = check_ws(workspace, ws_bytes, L.total)) != MOE_OK) return st;
  if (!ok_opt(dw13) || !ok_opt(dw2)) return MOE_ERR_INVALID_ARG;
  if (d->T > 0) {
    if (!ok_ptr(dy) || !ok_ptr(w2) || !ok_ptr(saved) || !ok_opt(dx)) return MOE_ERR_INVALID_ARG;
    if ((dx != nullptr && !ok_ptr(w13)) || (dw13 != nullptr && !ok_ptr(x)))
      return MOE_ERR_INVALID_ARG;
    if (dx != nullptr && (dx == dy || dx == x || dx == w13 || dx == w2)) return MOE_ERR_INVALID_ARG;
    // the three are of one launch, which reads neither w2 nor saved
    const void *w13_read = dx != nullptr ? w13 : nullptr;
    if (lies_on(dw13, {x, w13_read, dw2 != nullptr ? dy : nullptr, dx, dw2}) ||
        lies_on(dw2, {dy, w13_read, dw13 != nullptr ? x : nullptr, dx}))
      return MOE_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != MOE_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  void *h = at(workspace, L.h), *dgu = at(workspace, L.dgu);
  const int T = d->T, H = d->H, I = d->I;
  if (T == 0) {
    cudaError_t e = no_rows(dw13, 2 * (int64_t)I * H, dw_dtype, accumulate, s);
    if (e == cudaSuccess) e = no_rows(dw2, (int64_t)H * I, dw_dtype, accumulate, s);
    return cuda_status(e);
  }
  DenseGemm g[3];
  int n = 0;
  if (dx != nullptr)
    g[n++] = product(T, H, 2 * I, d->dtype, dgu, 2 * (int64_t)I, false, w13, H, true, dx, H,
                     d->dtype, workspace);
  if (dw13 != nullptr)
    g[n++] = weight_grad(2 * I, H, T, d->dtype, dgu, 2 * (int64_t)I, x, H, dw13, dw_dtype,
                         accumulate, workspace);
  if (dw2 != nullptr)
    g[n++] = weight_grad(H, I, T, d->dtype, dy, H, h, I, dw2, dw_dtype, accumulate, workspace);
  if (n == 0) return MOE_OK;
  DenseGemm up = product(T, I, H, d->dtype, dy, H, false, w2, I, true, nullptr, 0, d->dtype,
                         workspace);
  up.epi = kEpiGatedGrad;
  up.saved = const_cast<float *>(saved);
  up.dgu = dgu;
  up.h = h;
  cudaError_t e = launch_dense_pair(up, s);
  if (e == cudaSuccess) e = gradients(g, n, dx != nullptr, s);
  return cuda_status(e);
}

}  // extern "C"
