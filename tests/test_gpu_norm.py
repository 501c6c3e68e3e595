"""Residual addition with RMS norm (moe_add_rms_norm) and its gradient against
64-bit formulas (needs a GB300)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe
from dense_ref import EPS32, assert_within, dequantize, half_step, rms_norm, tiny

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_ffn_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def randn(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def code(dtype):
    return {BF16: moe.MOE_DTYPE_BF16, FP16: moe.MOE_DTYPE_FP16, FP32: moe.MOE_DTYPE_FP32}[dtype]


# rows: none, one, few (one chunk a thread), many; widths: one chunk, not a
# multiple of a 128 block, of a warp, the widest
SHAPES = [(0, 256), (1, 8), (1, 4096), (3, 16384), (5, 264), (17, 1160), (400, 136), (401, 4104),
          (330, 9000), (310, 16384)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("with_residual", [True, False])
def test_forward(T, H, dtype, with_residual):
    x, w = randn(1, T, H, dtype=dtype), randn(2, H, dtype=dtype)
    r = randn(3, T, H, std=2.0, dtype=dtype) if with_residual else None
    y, ro = torch.empty_like(x), torch.full_like(x, 7.0)
    q = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    e = torch.zeros(T, -(-H // 128), dtype=torch.int8, device="cuda")
    moe.moe_add_rms_norm(moe.norm_desc(T, H, code(dtype), 1e-5), x, r, w, ro, y, q, e)
    torch.cuda.synchronize()
    s, want = rms_norm(x, r, w, 1e-5)
    assert_within(ro, s, s.abs() * (half_step(dtype) + EPS32) + tiny(dtype), "residual_out")
    # fp32: the addition, a sum of H squares by a tree (its relative error is
    # below 2 log2 H steps), the root, the division and two products
    rel32 = 64 * EPS32
    assert_within(y, want, want.abs() * (half_step(dtype) + rel32) + tiny(dtype), "y")
    if T == 0:
        return
    # exponents: the least e with amax <= 448 * 2^e, where amax is not within
    # rounding of the border
    nb = e.shape[1]
    p = torch.zeros(T, nb * 128, dtype=torch.float64, device="cuda")
    p[:, :H] = want.abs()
    amax = p.view(T, nb, 128).amax(2)
    exact = torch.ceil(torch.log2(amax / 448.0)).clamp(min=-126)
    ratio = amax / 448.0 / torch.exp2(exact)
    clear = (ratio < 1 - 1e-5) & (ratio > 0.5 * (1 + 1e-5)) & (amax > 0)
    assert torch.equal(e.double()[clear], exact[clear])
    assert int((e.double() - exact).abs()[amax > 0].max()) <= 1
    scale = torch.exp2(e.double()).repeat_interleave(128, 1)[:, :H]
    got = dequantize(q, e)
    # E4M3: half a step of the value, or of its smallest numbers (2^-9) times the scale
    assert_within(got, want, want.abs() * (2.0 ** -4 + rel32) + scale * 2.0 ** -10, "y_q")


def test_zero_blocks_and_extremes():
    T, H = 4, 512
    x = torch.zeros(T, H, dtype=FP32, device="cuda")
    x[1, 128:256] = 1.0
    x[2] = 1e17
    x[3, 7] = float("inf")
    w = torch.ones(H, dtype=FP32, device="cuda")
    y, q = torch.empty_like(x), torch.full((T, H), 99, dtype=torch.uint8, device="cuda")
    e = torch.full((T, 4), 99, dtype=torch.int8, device="cuda")
    moe.moe_add_rms_norm(moe.norm_desc(T, H, moe.MOE_DTYPE_FP32, 1e-6), x, None, w, None, y, q, e)
    torch.cuda.synchronize()
    assert not q[0].any() and not e[0].any() and not y[0].any()
    assert e[1].tolist()[0] == 0 and not q[1, :128].any()
    assert_within(y[2], torch.ones(H), torch.full((H,), 64 * EPS32), "large rows")
    assert torch.isnan(y[3, 7]) and not y[3, :7].any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strides_and_in_place(dtype):
    T, H = 37, 520
    wide = randn(4, T, H + 24, dtype=dtype)
    r, w = randn(5, T, H + 8, dtype=dtype), randn(6, H, dtype=dtype)
    x, res = wide[:, 8:8 + H], r[:, :H]
    s, want = rms_norm(x, res, w, 1e-6)
    yw = torch.full((T, H + 16), 5.0, dtype=dtype, device="cuda")
    before = r[:, H:].clone()
    moe.moe_add_rms_norm(moe.norm_desc(T, H, code(dtype), 1e-6, H + 24, H + 8, H + 16), x, res, w,
                         res, yw[:, :H])
    torch.cuda.synchronize()
    assert_within(res, s, s.abs() * (half_step(dtype) + EPS32) + tiny(dtype), "in-place residual")
    assert_within(yw[:, :H], want, want.abs() * (half_step(dtype) + 64 * EPS32) + tiny(dtype), "y")
    assert bool((yw[:, H:] == 5.0).all()) and torch.equal(before, r[:, H:])


def backward_ref(dy, dres, s, w, eps):
    s = s.double().cpu().requires_grad_()
    w = w.double().cpu().requires_grad_()
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w
    dx, dw = torch.autograd.grad(y, (s, w), dy.double().cpu())
    return dx + (dres.double().cpu() if dres is not None else 0.0), dw


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H", [(0, 64), (1, 8), (1, 4096), (33, 264), (700, 1160), (513, 8192),
                                 (340, 8200), (311, 16384)])
@pytest.mark.parametrize("with_dres", [True, False])
def test_backward(T, H, dtype, with_dres):
    eps = 1e-5
    s, w = randn(11, T, H, dtype=dtype), randn(12, H, dtype=dtype)
    dy = randn(13, T, H, std=0.1, dtype=dtype)
    dres = randn(14, T, H, std=0.1, dtype=dtype) if with_dres else None
    dx, dw = torch.empty_like(s), torch.full((H,), 9.0, device="cuda")
    d = moe.norm_desc(T, H, code(dtype), eps)
    ws = moe.alloc_workspace(d)
    moe.moe_add_rms_norm_backward(d, dy, dres, s, w, dx, dw, ws)
    torch.cuda.synchronize()
    if T == 0:
        assert not dw.any()
        return
    want, want_w = backward_ref(dy, dres, s, w, eps)
    # the terms' magnitudes: r |w dy| + |n| mean|w dy n| r + |dres|
    sd, wd, dyd = s.double().cpu(), w.double().cpu(), dy.double().cpu()
    r = 1.0 / torch.sqrt(sd.square().mean(1, keepdim=True) + eps)
    n = sd * r
    mag = r * ((wd * dyd).abs() + n.abs() * (wd * dyd * n).abs().mean(1, keepdim=True))
    if dres is not None:
        mag = mag + dres.double().cpu().abs()
    assert_within(dx, want, want.abs() * half_step(dtype) + mag * 64 * EPS32 + tiny(dtype), "dx")
    # T products summed along at most T / CTAs rows and then the CTAs: each
    # addition is off by a step of the running sum, at most the magnitudes' sum
    magw = (dyd * n).abs().sum(0)
    assert_within(dw, want_w, magw * (64 + T) * EPS32 + 1e-30, "dweight")


def test_backward_same_bits_twice_and_in_place():
    T, H = 900, 1160
    s, w = randn(21, T, H), randn(22, H)
    dy, dres = randn(23, T, H), randn(24, T, H)
    d = moe.norm_desc(T, H, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    outs = []
    for _ in range(2):
        dx, dw = torch.empty_like(s), torch.empty(H, device="cuda")
        moe.moe_add_rms_norm_backward(d, dy, dres, s, w, dx, dw, ws)
        outs.append((dx, dw))
    g = dres.clone()
    moe.moe_add_rms_norm_backward(d, dy, g, s, w, g, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(g, outs[0][0])


def test_gradient_against_differences():
    """d/dh of L(s + h v) = <dx, v> for L = sum(dy * y), by central differences of the forward."""
    T, H, eps, h = 6, 264, 1e-5, 2.0 ** -7
    s, w = randn(31, T, H, dtype=FP32), randn(32, H, dtype=FP32)
    dy, v = randn(33, T, H, dtype=FP32), randn(34, T, H, dtype=FP32)
    d = moe.norm_desc(T, H, moe.MOE_DTYPE_FP32, eps)
    ws = moe.alloc_workspace(d)
    dx = torch.empty_like(s)
    moe.moe_add_rms_norm_backward(d, dy, None, s, w, dx, None, ws)

    def loss(x):
        y = torch.empty_like(x)
        moe.moe_add_rms_norm(d, x.contiguous(), None, w, None, y)
        return (y.double() * dy.double()).sum()

    diff = (loss(s + h * v) - loss(s - h * v)) / (2 * h)
    along = (dx.double() * v.double()).sum()
    # rounding: 64 fp32 steps of the terms over 2h; the cubic term of the
    # difference: h^2 / 6 times the third derivative, below 30 sum |dy w v| here
    mag = (dy.double() * w.double() * v.double()).abs().sum()
    assert abs(float(diff - along)) <= float(mag) * (64 * EPS32 / h + 5 * h * h)


def test_captured_in_a_graph_and_on_another_stream():
    T, H = 64, 4096
    x, w = randn(41, T, H), randn(42, H)
    d = moe.norm_desc(T, H, moe.MOE_DTYPE_BF16)
    want, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rms_norm(d, x, None, w, None, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_add_rms_norm(d, x, None, w, None, y, stream=st)
    st.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_add_rms_norm(d, x, None, w, None, y)
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """2^20 rows of 2056 elements: more than 2^31 of them, both directions and codes."""
    T, H, rows, eps = 1 << 20, 2056, 1024, 1e-5
    x, w, dy = randn(51, rows, H), randn(52, H), randn(53, rows, H, std=0.1)
    d = moe.norm_desc(T, H, code(BF16), eps)
    ws = moe.alloc_workspace(d)
    many = x.repeat(T // rows, 1)
    y = torch.empty_like(many)
    q = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    e = torch.empty(T, -(-H // 128), dtype=torch.int8, device="cuda")
    moe.moe_add_rms_norm(d, many, many, w, None, y, q, e)
    torch.cuda.synchronize()
    _, want = rms_norm(x, x, w, eps)
    assert_within(y[:rows], want, want.abs() * (half_step(BF16) + 64 * EPS32) + tiny(BF16), "y")
    for t in (y, q, e):
        for i in range(0, T, T // 16):
            assert bool((t[i:i + T // 16].view(-1, rows, t.shape[1]) == t[:rows]).all())
    del q, e
    grads = dy.repeat(T // rows, 1)
    dw = torch.empty(H, device="cuda")
    moe.moe_add_rms_norm_backward(d, grads, None, many, w, y, dw, ws)
    torch.cuda.synchronize()
    want, want_w = backward_ref(dy, None, x, w, eps)
    sd, wd, dyd = x.double().cpu(), w.double().cpu(), dy.double().cpu()
    r = 1.0 / torch.sqrt(sd.square().mean(1, keepdim=True) + eps)
    n = sd * r
    mag = r * ((wd * dyd).abs() + n.abs() * (wd * dyd * n).abs().mean(1, keepdim=True))
    assert_within(y[:rows], want, want.abs() * half_step(BF16) + mag * 64 * EPS32 + tiny(BF16), "dx")
    for i in range(0, T, T // 16):
        assert bool((y[i:i + T // 16].view(-1, rows, H) == y[:rows]).all())
    # a CTA adds at most T / 152 rows, then their sums are added
    magw = (dyd * n).abs().sum(0) * (T // rows)
    assert_within(dw, want_w * (T // rows), magw * (64 + T / 152 + 304) * EPS32, "dweight")
