"""Every path of the linear's kernels by name: the plan that a case runs by is read back, so that a
refit of the estimates cannot leave one without a test (needs a GB300)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe
from dense_ref import activation, assert_within, dequantize, half_step, product_bound, tiny

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
FEW, TILES = moe.MOE_LINEAR_FEW_ROWS, moe.MOE_LINEAR_TILES


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


def bound_of(x, w, bias, residual, act, out):
    """(z, result, bound) in 64 bits: fp32 sums, the activation to 2^-18 of z (slopes are below
    1.13), an fp32 step for each addition, one rounding to `out`."""
    z = x @ w.t()
    e = product_bound(x, w, x.shape[1])
    if bias is not None:
        z = z + bias
        e = e + (z.abs() + bias.abs()) * 2.0 ** -24
    y = activation(z, act)
    ez = e
    if act != "none":
        e = 1.13 * e + z.abs() * 2.0 ** -18
    if residual is not None:
        y = y + residual
        e = e + y.abs() * 2.0 ** -24
    return z, y, e + (y.abs() + e) * half_step(out) + tiny(out), ez


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP16), (BF16, FP32)])
@pytest.mark.parametrize("T,N,K", [(2000, 520, 8200), (1100, 1000, 4104), (1500, 264, 14344),
                                   (1030, 72, 7176)])
@pytest.mark.parametrize("keep", [False, True])
def test_split_between_pairs(T, N, K, dtype, out, keep):
    """K in two parts: bias, activation, residual and pre-activation behind the exchange."""
    x, w = randn(1, T, K, dtype=dtype), randn(2, N, K, std=K ** -0.5, dtype=dtype)
    b, r = randn(3, N, dtype=out), randn(4, T, N + 16, dtype=out)[:, :N]
    d = moe.linear_desc(T, N, K, moe.dtype_of(x), "silu", out_dtype=moe.dtype_of(b),
                        residual_stride=N + 16)
    plan = moe.moe_linear_plan(d, keep)
    assert (plan.kernel, plan.tile_rows, plan.split) == (TILES, 256, 2)
    ws = moe.alloc_workspace(d)
    y = torch.full((T, N), 3.0, dtype=out, device="cuda")
    z = torch.full((T, N), 3.0, device="cuda") if keep else None
    moe.moe_linear(d, x, w, b, r, y, ws, preact=z)
    status_ok(ws)
    wz, want, bound, ez = bound_of(x.double(), w.double(), b.double(), r.double(), "silu", out)
    assert_within(y, want, bound, "y")
    if keep:
        assert_within(z, wz, ez + wz.abs() * 2.0 ** -23, "preact")


def quantized(t, rows):
    """E4M3 codes and exponents of t in rows x 128 blocks."""
    R, C = t.shape
    nr, nc = -(-R // rows), -(-C // 128)
    p = torch.zeros(nr * rows, nc * 128, dtype=torch.float32, device=t.device)
    p[:R, :C] = t.float()
    p = p.view(nr, rows, nc, 128)
    e = torch.ceil(torch.log2((p.abs().amax(dim=(1, 3)) / 448).clamp(min=2.0 ** -15)))
    q = (p / torch.exp2(e)[:, None, :, None]).view(nr * rows, nc * 128)[:R, :C]
    return (q.clamp(-448, 448).to(torch.float8_e4m3fn).contiguous(),
            e.to(torch.int8).contiguous())


# stages of 128 of K: below one hand-over of scale factors (8), uneven blocks of four, unaligned
# rows of exponents, tails of K; tiles: one a cluster to more than three
@pytest.mark.parametrize("T,N,K,split", [
    (2047, 4104, 1040, 1), (2047, 4104, 2192, 1), (1025, 264, 16, 1), (1300, 520, 400, 1),
    (3100, 4104, 4112, 1), (2600, 4488, 1280, 1), (1030, 264, 7184, 2), (1100, 520, 9232, 2),
    (1500, 136, 4624, 2)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_e4m3_tiles(T, N, K, split, out):
    # exponents that differ along every axis: a wrong one shows
    x, w = randn(5, T, K, dtype=FP32), randn(6, N, K, std=K ** -0.5, dtype=FP32)
    blocks = torch.arange(K, device="cuda").div(128, rounding_mode="floor")
    x = x * torch.exp2(((torch.arange(T, device="cuda")[:, None] + 3 * blocks) % 7).float())
    w = w * torch.exp2(((torch.arange(N, device="cuda").div(128, rounding_mode="floor")[:, None]
                         + 2 * blocks) % 5).float())
    b, r = randn(7, N, dtype=out), randn(8, T, N, dtype=out)
    (xq, xe), (wq, we) = quantized(x, 1), quantized(w, 128)
    assert len(xe.unique()) > 4 and (K < 1000 or len(we.unique()) > 3)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_E4M3, "silu", out_dtype=moe.dtype_of(b))
    plan = moe.moe_linear_plan(d)
    assert (plan.kernel, plan.split) == (TILES, split)
    ws = moe.alloc_workspace(d)
    y = torch.full((T, N), 3.0, dtype=out, device="cuda")
    moe.moe_linear(d, xq, wq, b, r, y, ws, x_scale=xe, w_scale=we)
    status_ok(ws)
    _, want, bound, _ = bound_of(dequantize(xq, xe), dequantize(wq, we, 128), b.double(),
                                 r.double(), "silu", out)
    assert_within(y, want, bound, "y")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,N,K", [(300, 520, 264), (300, 4104, 136), (2047, 1032, 2056),
                                   (513, 14344, 264)])
def test_dx_alone(T, N, K, dtype):
    """More than 64 rows and no dw: one product with W as it lies, K (here N) split or not."""
    w = randn(10, N, K, std=K ** -0.5, dtype=dtype)
    dy = randn(11, T, N, std=0.5, dtype=dtype)
    d = moe.linear_desc(T, N, K, moe.dtype_of(w))
    ws = moe.alloc_workspace(d)
    dx = torch.full((T, K), 9.0, dtype=dtype, device="cuda")
    moe.moe_linear_backward(d, dy, None, w, None, dx, None, None, ws)
    status_ok(ws)
    want = dy.double() @ w.double()
    e = product_bound(dy.double(), w.double().t(), N)
    assert_within(dx, want, e + (want.abs() + e) * half_step(dtype) + tiny(dtype), "dx")


@pytest.mark.parametrize("T,N,K", [(300, 520, 264), (700, 2056, 136)])
def test_dw_alone(T, N, K):
    x, dy = randn(12, T, K), randn(13, T, N, std=0.5)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    dw = torch.full((N, K), 9.0, device="cuda")
    moe.moe_linear_backward(d, dy, x, None, None, None, dw, None, ws)
    status_ok(ws)
    want = dy.double().t() @ x.double()
    assert_within(dw, want, product_bound(dy.double().t(), x.double().t(), T), "dw")


@pytest.mark.parametrize("T,dtype,kernel", [(1, BF16, FEW), (40, BF16, FEW), (2000, BF16, TILES),
                                            (1, torch.float8_e4m3fn, FEW)])
def test_which_kernel(T, dtype, kernel):
    code = moe.MOE_DTYPE_BF16 if dtype is BF16 else moe.MOE_DTYPE_E4M3
    plan = moe.moe_linear_plan(moe.linear_desc(T, 4096, 4096, code))
    assert plan.kernel == kernel
    assert plan.tile_rows >= min(T, 16) and plan.split in (1, 2, 4, 8)
    # the pre-activation is stored by the tiled kernel only
    if code == moe.MOE_DTYPE_BF16:
        assert moe.moe_linear_plan(moe.linear_desc(T, 4096, 4096, code), True).kernel == TILES


def test_two_streams_with_a_workspace_each():
    """Products of both kernels and gradients, at the same time on two streams, give what they
    give alone."""
    def work(seed, T):
        x, w, dy = randn(seed, T, 1032), randn(seed + 1, 776, 1032, std=1 / 32), randn(seed + 2, T, 776)
        d = moe.linear_desc(T, 776, 1032, moe.MOE_DTYPE_BF16)
        ws = moe.alloc_workspace(d)
        y, dx = torch.empty(T, 776, dtype=BF16, device="cuda"), torch.empty_like(x)
        dw, db = torch.empty_like(w), torch.empty(776, device="cuda")

        def run(stream):
            moe.moe_linear(d, x, w, None, None, y, ws, stream=stream)
            moe.moe_linear_backward(d, dy, x, w, None, dx, dw, db, ws, stream=stream)
        return run, (y, dx, dw, db), ws
    jobs = [work(20, 40), work(30, 1500)]
    alone = []
    for run, outs, ws in jobs:
        run(None)
        torch.cuda.synchronize()
        alone.append([o.clone() for o in outs])
        for o in outs:
            o.fill_(9.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        for (run, _, _), s in zip(jobs, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, outs, ws), want in zip(jobs, alone):
        status_ok(ws)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_norm_in_place(dtype):
    """y in place of x, and dx in place of dy: the bits of the calls that are not in place."""
    T, H = 333, 1160
    x, r, w = randn(40, T, H, dtype=dtype), randn(41, T, H, dtype=dtype), randn(42, H, dtype=dtype)
    d = moe.norm_desc(T, H, moe.dtype_of(x))
    want, ro, rp = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rms_norm(d, x, r, w, ro, want)
    y = x.clone()
    moe.moe_add_rms_norm(d, y, r, w, rp, y)
    ws = moe.alloc_workspace(d)
    dy, dres = randn(43, T, H, dtype=dtype), randn(44, T, H, dtype=dtype)
    dx, dw, dw2 = torch.empty_like(x), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_add_rms_norm_backward(d, dy, dres, ro, w, dx, dw, ws)
    g = dy.clone()
    moe.moe_add_rms_norm_backward(d, g, dres, ro, w, g, dw2, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(rp, ro)
    assert torch.equal(g, dx) and torch.equal(dw, dw2)
