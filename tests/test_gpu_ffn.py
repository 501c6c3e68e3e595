"""The gated feed-forward block (moe_gated_ffn) and its gradients against
64-bit formulas (needs a GB300)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe
from dense_ref import assert_within, half_step, product_bound, rel_l2, tiny

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


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


def inputs(T, H, I, dtype):
    return dict(x=randn(1, T, H, dtype=dtype), w13=randn(2, 2 * I, H, std=H ** -0.5, dtype=dtype),
                w2=randn(3, H, I, std=I ** -0.5, dtype=dtype), r=randn(4, T, H, dtype=dtype),
                dy=randn(5, T, H, std=0.5, dtype=dtype))


def hidden(t, I):
    """g, u, h in 64 bits and what h may be off by before and after its rounding."""
    x, w13 = t["x"].double(), t["w13"].double()
    z = x @ w13.t()
    e = product_bound(x, w13, x.shape[1])
    g, u, eg, eu = z[:, :I], z[:, I:], e[:, :I], e[:, I:]
    a = torch.nn.functional.silu(g)
    h = a * u
    # SiLU's slope is below 1.1 and its value good to 2^-20 of itself
    eh = (1.1 * eg + a.abs() * 2.0 ** -20) * (u.abs() + eu) + a.abs() * eu
    return g, u, h, eg, eu, eh


SHAPES = [(0, 64, 64), (1, 8, 8), (1, 1024, 2048), (4, 264, 520), (16, 512, 1536), (33, 136, 1000),
          (130, 1032, 264), (256, 256, 512), (300, 520, 776), (1000, 264, 392)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_forward(T, H, I, dtype):
    t = inputs(T, H, I, dtype)
    d = moe.ffn_desc(T, H, I, moe.dtype_of(t["x"]))
    ws = moe.alloc_workspace(d)
    y, saved = torch.empty_like(t["x"]), torch.empty(T, 2 * I, device="cuda")
    g, u, h, eg, eu, eh = hidden(t, I)
    w2, r = t["w2"].double(), t["r"].double()
    er = eh + (h.abs() + eh) * half_step(dtype) + tiny(dtype)
    want = h @ w2.t() + r
    e = er @ w2.abs().t() + product_bound(h, w2, I) + want.abs() * 2.0 ** -24
    bound = e + (want.abs() + e) * half_step(dtype) + tiny(dtype)
    moe.moe_gated_ffn(d, t["x"], t["w13"], t["w2"], t["r"], saved, y, ws)
    status_ok(ws)
    assert_within(y, want, bound, "y with saved")
    assert_within(saved, torch.cat([g, u], 1), torch.cat([eg, eu], 1) + 1e-30, "saved")
    y.fill_(9.0)
    moe.moe_gated_ffn(d, t["x"], t["w13"], t["w2"], t["r"], None, y, ws)
    status_ok(ws)
    assert_within(y, want, bound, "y")
    if T > 1:
        assert rel_l2(y, want) <= 2 * half_step(dtype)
    moe.moe_gated_ffn(d, t["x"], t["w13"], t["w2"], None, None, y, ws)
    status_ok(ws)
    want = want - r
    e = er @ w2.abs().t() + product_bound(h, w2, I)
    assert_within(y, want, e + (want.abs() + e) * half_step(dtype) + tiny(dtype), "no residual")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,H,I", [(0, 64, 72), (1, 8, 8), (5, 264, 136), (64, 136, 264),
                                   (130, 512, 256), (300, 264, 1000), (520, 1032, 392)])
def test_backward(T, H, I, dtype):
    t = inputs(T, H, I, dtype)
    d = moe.ffn_desc(T, H, I, moe.dtype_of(t["x"]))
    ws = moe.alloc_workspace(d)
    saved = (t["x"].float() @ t["w13"].float().t()).contiguous()
    dx, dw13, dw2 = (torch.full_like(t[k], 5.0) for k in ("x", "w13", "w2"))
    moe.moe_gated_ffn_backward(d, t["dy"], t["x"], t["w13"], t["w2"], saved, dx, dw13, dw2, ws)
    status_ok(ws)
    x, w13, w2, dy = (t[k].double() for k in ("x", "w13", "w2", "dy"))
    sv = saved.double().requires_grad_()
    dh = dy @ w2
    h = torch.nn.functional.silu(sv[:, :I]) * sv[:, I:]
    dgu, = torch.autograd.grad(h, sv, dh)
    h = h.detach()
    hs = half_step(dtype)
    # dh's accumulation, the factors' fp32 evaluation (2^-16 of the terms' size), one rounding
    s = torch.sigmoid(sv.detach()[:, :I])
    fac = torch.cat([(sv.detach()[:, I:] * s * (1 + sv.detach()[:, :I].abs())).abs(),
                     (sv.detach()[:, :I] * s).abs()], 1)
    eh = product_bound(dy, w2.t(), H).repeat(1, 2) * fac + dh.abs().repeat(1, 2) * fac * 2.0 ** -16
    er = eh + (dgu.abs() + eh) * hs + tiny(dtype)
    checks = [
        ("dx", dx, dgu @ w13, er @ w13.abs() + product_bound(dgu, w13.t(), 2 * I)),
        ("dw13", dw13, dgu.t() @ x, er.t() @ x.abs() + product_bound(dgu.t(), x.t(), T)),
        ("dw2", dw2, dy.t() @ h,
         dy.abs().t() @ (h.abs() * (hs + 2.0 ** -16) + tiny(dtype)) + product_bound(dy.t(), h.t(), T))]
    for name, got, want, e in checks:
        assert_within(got, want, e + (want.abs() + e) * hs + tiny(dtype), name)
        if T > 1:
            # in the 2-norm each of the two roundings is off by at most half a step
            assert rel_l2(got, want) <= 2 * hs, name


def test_training_step_against_autograd():
    """Forward with saved, then backward, against the 64-bit gradient of the whole block."""
    T, H, I = 200, 264, 520
    t = inputs(T, H, I, BF16)
    d = moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y, saved = torch.empty_like(t["x"]), torch.empty(T, 2 * I, device="cuda")
    outs = [torch.empty_like(t[k]) for k in ("x", "w13", "w2")]
    moe.moe_gated_ffn(d, t["x"], t["w13"], t["w2"], t["r"], saved, y, ws)
    moe.moe_gated_ffn_backward(d, t["dy"], t["x"], t["w13"], t["w2"], saved, *outs, ws)
    status_ok(ws)
    leaves = [t[k].double().requires_grad_() for k in ("x", "w13", "w2")]
    g, u = (leaves[0] @ leaves[1].t()).chunk(2, 1)
    out = (torch.nn.functional.silu(g) * u) @ leaves[2].t()
    for got, want in zip(outs, torch.autograd.grad(out, leaves, t["dy"].double())):
        assert rel_l2(got, want) <= 2 * half_step(BF16)


def test_gradients_in_fp32_accumulate_and_may_be_left_out():
    T, H, I = 140, 136, 264
    t = inputs(T, H, I, BF16)
    d = moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    saved = (t["x"].float() @ t["w13"].float().t()).contiguous()
    a13, a2 = torch.empty(2 * I, H, device="cuda"), torch.empty(H, I, device="cuda")
    b13, b2, dx, dx2 = (torch.empty_like(v) for v in (a13, a2, t["x"], t["x"]))
    args = (d, t["dy"], t["x"], t["w13"], t["w2"], saved)
    moe.moe_gated_ffn_backward(*args, dx, a13, a2, ws)
    moe.moe_gated_ffn_backward(*args, None, b13, None, ws)
    moe.moe_gated_ffn_backward(*args, dx2, None, b2, ws)
    torch.cuda.synchronize()
    assert torch.equal(a13, b13) and torch.equal(a2, b2) and torch.equal(dx, dx2)
    moe.moe_gated_ffn_backward(*args, None, b13, b2, ws, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(b13, a13 + a13) and torch.equal(b2, a2 + a2)


def test_captured_training_step():
    """Forward and backward captured in one graph give the eager results."""
    T, H, I = 72, 256, 512
    t = inputs(T, H, I, BF16)
    d = moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y, saved = torch.empty_like(t["x"]), torch.empty(T, 2 * I, device="cuda")
    outs = [torch.empty_like(t[k]) for k in ("x", "w13", "w2")]

    def step():
        moe.moe_gated_ffn(d, t["x"], t["w13"], t["w2"], t["r"], saved, y, ws)
        moe.moe_gated_ffn_backward(d, t["dy"], t["x"], t["w13"], t["w2"], saved, *outs, ws)

    step()
    torch.cuda.synchronize()
    want = [v.clone() for v in (y, *outs)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for v in (y, saved, *outs):
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    for v, w in zip((y, *outs), want):
        assert torch.equal(v, w)
    status_ok(ws)


@pytest.mark.parametrize("T,H,I", [(200, 7176, 136), (300, 4104, 264), (513, 2056, 72)])
def test_deep_products(T, H, I):
    """Few tiles and many terms in the gated product and in its gradient: K is split between CTA
    pairs where that pays."""
    t = inputs(T, H, I, BF16)
    d = moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y, saved = torch.empty_like(t["x"]), torch.empty(T, 2 * I, device="cuda")
    g, u, h, eg, eu, eh = hidden(t, I)
    for keep in (saved, None):
        y.fill_(9.0)
        moe.moe_gated_ffn(d, t["x"], t["w13"], t["w2"], t["r"], keep, y, ws)
        status_ok(ws)
        w2 = t["w2"].double()
        want = h @ w2.t() + t["r"].double()
        er = eh + (h.abs() + eh) * half_step(BF16) + tiny(BF16)
        e = er @ w2.abs().t() + product_bound(h, w2, I) + want.abs() * 2.0 ** -24
        assert_within(y, want, e + (want.abs() + e) * half_step(BF16) + tiny(BF16), "y")
    assert_within(saved, torch.cat([g, u], 1), torch.cat([eg, eu], 1) + 1e-30, "saved")
    outs = [torch.empty_like(t[k]) for k in ("x", "w13", "w2")]
    moe.moe_gated_ffn_backward(d, t["dy"], t["x"], t["w13"], t["w2"], saved, *outs, ws)
    status_ok(ws)
    leaves = [t[k].double().requires_grad_() for k in ("x", "w13", "w2")]
    g, u = (leaves[0] @ leaves[1].t()).chunk(2, 1)
    out = (torch.nn.functional.silu(g) * u) @ leaves[2].t()
    for got, want in zip(outs, torch.autograd.grad(out, leaves, t["dy"].double())):
        assert rel_l2(got, want) <= 2 * half_step(BF16)


def test_offsets_past_32_bits():
    """2^20 rows of 2056 columns: more than 2^31 elements."""
    T, H, I, rows = 1 << 20, 2056, 8, 1024
    t = inputs(rows, H, I, BF16)
    d = moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    x, y = t["x"].repeat(T // rows, 1), torch.zeros(T, H, dtype=BF16, device="cuda")
    moe.moe_gated_ffn(d, x, t["w13"], t["w2"], x, None, y, ws)
    status_ok(ws)
    _, _, h, _, _, eh = hidden(t, I)
    w2 = t["w2"].double()
    want = h @ w2.t() + t["x"].double()
    er = eh + (h.abs() + eh) * half_step(BF16) + tiny(BF16)
    e = er @ w2.abs().t() + product_bound(h, w2, I) + want.abs() * 2.0 ** -24
    assert_within(y[:rows], want, e + (want.abs() + e) * half_step(BF16) + tiny(BF16), "first rows")
    for i in range(0, T, T // 16):
        assert bool((y[i:i + T // 16].view(-1, rows, H) == y[:rows]).all()), f"rows from {i}"
