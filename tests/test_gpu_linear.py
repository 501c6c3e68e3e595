"""The matrix product with bias, activation and residual (moe_linear) and its
gradients against 64-bit formulas (needs a GB300)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe
from dense_ref import (activation, assert_within, dequantize, half_step, product_bound, rel_l2,
                       tiny)

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_ffn_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def randn(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float32) * std).to(dtype).cuda()


def status_ok(ws):
    st, raw = moe.moe_get_device_status(ws)
    assert st == moe.MOE_OK, (st, raw)


def forward_bound(x, w, bias, residual, act, out, dtype):
    """(result, bound) of act(x w^T + b) + r in 64 bits, rounded once to `dtype`."""
    K = x.shape[1]
    z = x @ w.t()
    e = product_bound(x, w, K)
    if bias is not None:
        z = z + bias
        e = e + z.abs() * 2.0 ** -24 + bias.abs() * 2.0 ** -24
    y = activation(z, act)
    # slopes are below 1.13; the activation itself is good to 2^-16 of its argument
    e = 1.13 * e + (0 if act == "none" else 1) * z.abs() * 2.0 ** -16
    if residual is not None:
        y = y + residual
        e = e + y.abs() * 2.0 ** -24
    return z, y, e + (y.abs() + e) * half_step(dtype) + tiny(dtype)


# rows around the tiles' edges, columns and depths that no tile divides
SHAPES = [(0, 64, 64), (1, 8, 8), (1, 1024, 2048), (2, 136, 4096), (7, 264, 72), (16, 4096, 520),
          (33, 1000, 1032), (64, 512, 7168), (129, 4104, 136), (255, 768, 264), (256, 256, 64),
          (257, 320, 200), (300, 264, 2056), (513, 2048, 1024), (1000, 776, 1032), (2047, 1032, 8)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_forward(T, N, K, dtype):
    x, w = randn(1, T, K, dtype=dtype), randn(2, N, K, std=K ** -0.5, dtype=dtype)
    b, r = randn(3, N, dtype=dtype), randn(4, T, N, dtype=dtype)
    d = moe.linear_desc(T, N, K, moe.dtype_of(x))
    ws = moe.alloc_workspace(d)
    y = torch.full((T, N), 3.0, dtype=dtype, device="cuda")
    moe.moe_linear(d, x, w, b, r, y, ws)
    status_ok(ws)
    _, want, bound = forward_bound(x.double(), w.double(), b.double(), r.double(), "none", y, dtype)
    assert_within(y, want, bound, "y")
    moe.moe_linear(d, x, w, None, None, y, ws)
    _, want, bound = forward_bound(x.double(), w.double(), None, None, "none", y, dtype)
    assert_within(y, want, bound, "y without bias and residual")


@pytest.mark.parametrize("act", moe.ACT_NAMES)
@pytest.mark.parametrize("T,N,K", [(3, 264, 520), (300, 1000, 264)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_activations_and_preact(T, N, K, act, out):
    x, w = randn(11, T, K), randn(12, N, K, std=4 * K ** -0.5)
    b, r = randn(13, N, dtype=out), randn(14, T, N, dtype=out)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, act=act, out_dtype=moe.dtype_of(b))
    ws = moe.alloc_workspace(d)
    y, z = torch.empty(T, N, dtype=out, device="cuda"), torch.empty(T, N, device="cuda")
    moe.moe_linear(d, x, w, b, r, y, ws, preact=z)
    status_ok(ws)
    wz, want, bound = forward_bound(x.double(), w.double(), b.double(), r.double(), act, y, out)
    assert_within(y, want, bound, "y")
    zb = product_bound(x.double(), w.double(), K) + (wz.abs() + b.double().abs()) * 2.0 ** -23
    assert_within(z, wz, zb, "preact")
    again = torch.empty_like(y)
    moe.moe_linear(d, x, w, b, r, again, ws)
    torch.cuda.synchronize()
    # the pre-activation is stored by the tiled kernel alone: the sums' order may differ
    assert_within(again, want, bound, "y without preact")


@pytest.mark.parametrize("T", [5, 310])
def test_strides_in_place_and_neighbours(T):
    """Rows inside wider buffers: what lies past a row's end and past the last row is neither
    read (it is NaN) nor written."""
    N, K = 520, 264
    xw = torch.full((T + 3, K + 40), float("nan"), dtype=BF16, device="cuda")
    xw[:T, 8:8 + K] = randn(21, T, K)
    yw = torch.full((T + 3, N + 24), float("nan"), dtype=BF16, device="cuda")
    yw[:T, :N] = randn(22, T, N)
    w, b = randn(23, N, K, std=K ** -0.5), randn(24, N)
    x, y = xw[:T, 8:8 + K], yw[:T, :N]
    _, want, bound = forward_bound(x.double(), w.double(), b.double(), y.double(), "silu", y, BF16)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, "silu", x_stride=K + 40,
                        residual_stride=N + 24, y_stride=N + 24)
    ws = moe.alloc_workspace(d)
    moe.moe_linear(d, x, w, b, y, y, ws)
    status_ok(ws)
    assert_within(y, want, bound, "y in place")
    assert bool(torch.isnan(yw[T:]).all()) and bool(torch.isnan(yw[:T, N:]).all())


@pytest.mark.parametrize("T", [4, 300])
def test_infinities_stay_in_their_row(T):
    N, K = 264, 520
    x, w = randn(31, T, K), randn(32, N, K, std=K ** -0.5)
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    moe.moe_linear(d, x, w, None, None, y, ws)
    status_ok(ws)
    assert not bool(torch.isfinite(y[1]).any()) or bool((w[:, 3] == 0).any())
    assert bool(torch.isnan(y[2]).all())
    keep = [i for i in range(T) if i not in (1, 2)]
    _, want, bound = forward_bound(x[keep].double(), w.double(), None, None, "none", y, BF16)
    assert_within(y[keep], want, bound, "the other rows")


def quantized(t, rows):
    """E4M3 codes and exponents of t in rows x 128 blocks (plain torch)."""
    R, C = t.shape
    nr, nc = -(-R // rows), -(-C // 128)
    p = torch.zeros(nr * rows, nc * 128, dtype=torch.float32, device=t.device)
    p[:R, :C] = t.float()
    p = p.view(nr, rows, nc, 128)
    e = torch.ceil(torch.log2((p.abs().amax(dim=(1, 3)) / 448).clamp(min=2.0 ** -15)))
    q = (p / torch.exp2(e)[:, None, :, None]).view(nr * rows, nc * 128)[:R, :C]
    return (q.clamp(-448, 448).to(torch.float8_e4m3fn).contiguous(),
            e.to(torch.int8).contiguous())


@pytest.mark.parametrize("T,N,K", [(0, 64, 64), (1, 8, 16), (1, 1024, 2048), (5, 264, 80), (16, 512, 7168),
                                   (70, 1000, 528), (200, 136, 1040), (300, 776, 2064),
                                   (513, 4096, 1024)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_e4m3(T, N, K, out):
    # blocks of very different sizes: wrong scales show
    x, w = randn(41, T, K, dtype=FP32), randn(42, N, K, std=K ** -0.5, dtype=FP32)
    x = x * torch.exp2(torch.randint(-6, 7, (T, 1), device="cuda").float())
    x = x * torch.exp2(torch.arange(K, device="cuda").div(128, rounding_mode="floor") % 5).float()
    w = w * torch.exp2(torch.arange(N, device="cuda").div(128, rounding_mode="floor") % 3)[:, None]
    b, r = randn(43, N, dtype=out), randn(44, T, N, dtype=out)
    (xq, xe), (wq, we) = quantized(x, 1), quantized(w, 128)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_E4M3, "gelu_tanh", out_dtype=moe.dtype_of(b))
    ws = moe.alloc_workspace(d)
    y = torch.empty(T, N, dtype=out, device="cuda")
    moe.moe_linear(d, xq, wq, b, r, y, ws, x_scale=xe, w_scale=we)
    status_ok(ws)
    _, want, bound = forward_bound(dequantize(xq, xe), dequantize(wq, we, 128), b.double(),
                                   r.double(), "gelu_tanh", y, out)
    assert_within(y, want, bound, "y")


def test_e4m3_reads_what_the_norm_and_the_quantiser_write():
    T, H, N = 37, 1152, 640
    x, g, w = randn(51, T, H), randn(52, H), randn(53, N, H, std=H ** -0.5)
    q = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    e = torch.empty(T, H // 128, dtype=torch.int8, device="cuda")
    moe.moe_add_rms_norm(moe.norm_desc(T, H, moe.MOE_DTYPE_BF16), x, None, g, None, None, q, e)
    wq = torch.empty(N, H, dtype=torch.uint8, device="cuda")
    we = torch.empty(N // 128, H // 128, dtype=torch.int8, device="cuda")
    moe.moe_quantize_fp8(w, 1, N, H, wq, we)
    d = moe.linear_desc(T, N, H, moe.MOE_DTYPE_E4M3)
    ws = moe.alloc_workspace(d)
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    moe.moe_linear(d, q, wq, None, None, y, ws, x_scale=e, w_scale=we)
    status_ok(ws)
    _, want, bound = forward_bound(dequantize(q, e), dequantize(wq, we, 128), None, None, "none", y,
                                   BF16)
    assert_within(y, want, bound, "y")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "relu"])
@pytest.mark.parametrize("T,N,K", [(0, 64, 72), (1, 8, 8), (5, 264, 136), (64, 520, 256),
                                   (200, 1000, 264), (515, 264, 1032), (1030, 512, 512)])
def test_backward(T, N, K, act, dtype):
    x, w = randn(61, T, K, dtype=dtype), randn(62, N, K, std=K ** -0.5, dtype=dtype)
    dy = randn(63, T, N, std=0.5, dtype=dtype)
    z = x.float() @ w.float().t()
    d = moe.linear_desc(T, N, K, moe.dtype_of(x), act=act)
    ws = moe.alloc_workspace(d)
    dx, dw = torch.empty_like(x), torch.full_like(w, 5.0)
    db = torch.full((N,), 5.0, device="cuda")
    moe.moe_linear_backward(d, dy, x, w, z, dx, dw, db, ws)
    status_ok(ws)
    zd = z.double().requires_grad_()
    dz, = torch.autograd.grad(activation(zd, act), zd, dy.double())
    # dz in fp32: the slope is good to 2^-16 of its own size (at most 1.13), then one rounding
    ez = dy.double().abs() * (0 if act == "none" else 2.0 ** -16)
    er = ez + (0 if act == "none" else half_step(dtype)) * (dz.abs() + ez) + tiny(dtype)
    xd, wd = x.double(), w.double()
    want = dz @ wd
    e = er @ wd.abs() + product_bound(dz, wd.t(), N)
    assert_within(dx, want, e + (want.abs() + e) * half_step(dtype) + tiny(dtype), "dx")
    want_w = dz.t() @ xd
    e = er.t() @ xd.abs() + product_bound(dz.t(), xd.t(), T)
    assert_within(dw, want_w, e + (want_w.abs() + e) * half_step(dtype) + tiny(dtype), "dw")
    # in the 2-norm each of the two roundings is off by at most half a step
    if T > 1:
        assert rel_l2(dx, want) <= 2 * half_step(dtype)
        assert rel_l2(dw, want_w) <= 2 * half_step(dtype)
    assert_within(db, dz.sum(0), ez.sum(0) + dz.abs().sum(0) * (T + 16) * 2.0 ** -24 + 1e-30, "dbias")


def test_backward_accumulates_in_fp32_and_repeats_bit_for_bit():
    T, N, K = 300, 264, 136
    x, w, dy = randn(71, T, K), randn(72, N, K), randn(73, T, N)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    once, twice = torch.empty(N, K, device="cuda"), torch.empty(N, K, device="cuda")
    b1, b2 = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    moe.moe_linear_backward(d, dy, x, w, None, None, once, b1, ws)
    moe.moe_linear_backward(d, dy, x, w, None, None, twice, b2, ws)
    torch.cuda.synchronize()
    assert torch.equal(once, twice) and torch.equal(b1, b2)
    moe.moe_linear_backward(d, dy, x, w, None, None, twice, b2, ws, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(twice, once + once) and torch.equal(b2, b1 + b1)


def test_backward_against_differences():
    """L = sum(dy * y): dL/dh along the signs of dx and of dw, by central differences."""
    T, N, K = 40, 72, 64
    # values on coarse grids: x + v 2^-6 and w + u 2^-10 are exact in bf16
    x = randn(81, T, K).mul(4).round().div(4).clamp(-3.75, 3.75)
    w = randn(83, N, K).mul(4).round().clamp(-15, 15).div(64)
    dy = randn(85, T, N).mul(4).round().div(4)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, act="silu", out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)

    def loss(x_, w_, z=None):
        y = torch.empty(T, N, device="cuda")
        moe.moe_linear(d, x_, w_, None, None, y, ws, preact=z)
        return float((y.double() * dy.double()).sum())

    z = torch.empty(T, N, device="cuda")
    loss(x, w, z)
    dx, dw = torch.empty_like(x), torch.empty(N, K, device="cuda")
    moe.moe_linear_backward(d, dy, x, w, z, dx, dw, None, ws)
    ady = dy.double().abs()
    off = product_bound(x.double(), w.double(), K) + z.double().abs() * 2.0 ** -16
    noise = float((ady * off).sum())
    for grad, h in ((dx, 2.0 ** -6), (dw, 2.0 ** -10)):
        v = grad.sign().to(BF16)
        if grad is dx:
            plus, minus, dz = loss(x + h * v, w), loss(x - h * v, w), v.double() @ w.double().t()
        else:
            plus, minus, dz = loss(x, w + h * v), loss(x, w - h * v), x.double() @ v.double().t()
        along = float((grad.double() * v.double()).sum())
        # the difference's cubic term: h^2/6 times SiLU's third derivative (below 0.32) times
        # |dz|^3; the gradient's two roundings; the losses' own error over the step
        cubic = float((ady * dz.abs() ** 3).sum()) * h * h / 6 * 0.32
        assert abs((plus - minus) / (2 * h) - along) <= cubic + 2 * half_step(BF16) * along + noise / h


def test_captured_in_a_graph_and_on_another_stream():
    T, N, K = 24, 512, 1024
    x, w, r = randn(91, T, K), randn(92, N, K), randn(93, T, N)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    want, y = torch.empty_like(r), torch.empty_like(r)
    moe.moe_linear(d, x, w, None, r, want, ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_linear(d, x, w, None, r, y, ws, stream=st)
    st.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_linear(d, x, w, None, r, y, ws)
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, FP32), (FP16, FP16)])
@pytest.mark.parametrize("T,N,K", [(150, 264, 14344), (200, 520, 7176), (300, 264, 4104),
                                   (513, 1000, 8200), (700, 72, 2056)])
def test_deep_products(T, N, K, dtype, out):
    """Few tiles and many terms: K is split between CTA pairs."""
    x, w = randn(81, T, K, dtype=dtype), randn(82, N, K, std=K ** -0.5, dtype=dtype)
    b, r = randn(83, N, dtype=out), randn(84, T, N + 16, dtype=out)[:, :N]
    d = moe.linear_desc(T, N, K, moe.dtype_of(x), "silu", out_dtype=moe.dtype_of(b),
                        residual_stride=N + 16)
    ws = moe.alloc_workspace(d)
    y = torch.full((T, N), 3.0, dtype=out, device="cuda")
    moe.moe_linear(d, x, w, b, r, y, ws)
    status_ok(ws)
    _, want, bound = forward_bound(x.double(), w.double(), b.double(), r.double(), "silu", y, out)
    assert_within(y, want, bound, "y")


@pytest.mark.parametrize("T,N,K", [(200, 136, 7184), (300, 392, 4112), (513, 264, 9216)])
def test_deep_e4m3(T, N, K):
    x, w = randn(85, T, K, dtype=FP32), randn(86, N, K, std=K ** -0.5, dtype=FP32)
    x = x * torch.exp2(torch.arange(K, device="cuda").div(128, rounding_mode="floor") % 7).float()
    r = randn(87, T, N)
    (xq, xe), (wq, we) = quantized(x, 1), quantized(w, 128)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_E4M3)
    ws = moe.alloc_workspace(d)
    y = torch.full((T, N), 3.0, dtype=BF16, device="cuda")
    moe.moe_linear(d, xq, wq, None, r, y, ws, x_scale=xe, w_scale=we)
    status_ok(ws)
    _, want, bound = forward_bound(dequantize(xq, xe), dequantize(wq, we, 128), None, r.double(),
                                   "none", y, BF16)
    assert_within(y, want, bound, "y")


@pytest.mark.parametrize("T,N,K", [(4100, 264, 136), (700, 136, 4104), (700, 4104, 136), (260, 2056, 2056)])
def test_backward_of_unequal_products(T, N, K):
    """dx's terms are N, dw's T: one launch holds tiles of very different depth."""
    x, w = randn(91, T, K), randn(92, N, K, std=K ** -0.5)
    dy = randn(93, T, N, std=0.5)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    dx, dw = torch.empty_like(x), torch.zeros(N, K, device="cuda")
    for i in (1, 2):  # dw accumulates
        moe.moe_linear_backward(d, dy, x, w, None, dx, dw, None, ws, accumulate=True)
        status_ok(ws)
        want = dy.double() @ w.double()
        e = product_bound(dy.double(), w.double().t(), N)
        assert_within(dx, want, e + (want.abs() + e) * half_step(BF16) + tiny(BF16), "dx")
        want = i * (dy.double().t() @ x.double())
        e = i * product_bound(dy.double().t(), x.double().t(), T) + want.abs() * 2.0 ** -23
        assert_within(dw, want, e, "dw")


def test_offsets_past_32_bits():
    """2^20 rows of 4096 columns: more than 2^31 elements, more than 2^33 bytes."""
    T, N, K, rows = 1 << 20, 4096, 64, 1024
    x, w, b = randn(94, rows, K), randn(95, N, K, std=K ** -0.5), randn(96, N)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y = torch.zeros(T, N, dtype=BF16, device="cuda")
    moe.moe_linear(d, x.repeat(T // rows, 1), w, b, y, y, ws)
    status_ok(ws)
    _, want, bound = forward_bound(x.double(), w.double(), b.double(), None, "none", y, BF16)
    # the residual's zeros add a rounding to fp32 only
    assert_within(y[:rows], want, bound + want.abs() * 2.0 ** -24, "the first rows")
    for i in range(0, T, T // 16):
        part = y[i:i + T // 16].view(-1, rows, N)
        assert bool((part == y[:rows]).all()), f"rows from {i}"


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,N,K", [(1, 6336, 400), (16, 4104, 136), (17, 2056, 72), (64, 8200, 264), (33, 5000, 8)])
def test_backward_of_few_rows_and_many_terms(T, N, K, dtype):
    """dx of few rows and columns over many terms: the kernel for few rows, W as it lies."""
    x, w = randn(97, T, K, dtype=dtype), randn(98, N, K, std=K ** -0.5, dtype=dtype)
    dy = randn(99, T, N + 8, std=0.5, dtype=dtype)[:, :N]
    d = moe.linear_desc(T, N, K, moe.dtype_of(x), y_stride=N + 8, x_stride=K + 16)
    ws = moe.alloc_workspace(d)
    dxw = torch.full((T + 1, K + 16), 7.0, dtype=dtype, device="cuda")
    xw = torch.zeros(T, K + 16, dtype=dtype, device="cuda")
    xw[:, :K] = x
    dx, dw, db = dxw[:T, :K], torch.empty_like(w), torch.empty(N, device="cuda")
    want = dy.double() @ w.double()
    e = product_bound(dy.double(), w.double().t(), N)
    bound = e + (want.abs() + e) * half_step(dtype) + tiny(dtype)
    wdw = dy.double().t() @ x.double()
    e = product_bound(dy.double().t(), x.double().t(), T)
    for only in (False, True):
        dx.fill_(9.0)
        moe.moe_linear_backward(d, dy, xw[:, :K], w, None, dx, None if only else dw,
                                None if only else db, ws)
        status_ok(ws)
        assert_within(dx, want, bound, "dx")
        assert bool((dxw[T:] == 7).all()) and bool((dxw[:, K:] == 7).all())
    assert_within(dw, wdw, e + (wdw.abs() + e) * half_step(dtype) + tiny(dtype), "dw")
    assert_within(db, dy.double().sum(0), dy.double().abs().sum(0) * (T + 8) * 2.0 ** -24, "dbias")
