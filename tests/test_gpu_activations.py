"""Activations to a few fp32 steps, also far from zero (needs a GB300)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe
from dense_ref import activation

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
STEP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_ffn_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def steps(z, act):
    """How many fp32 steps act(z) may be off by: four for the functions called (erfc 4, exp 1 and
    the division 2 by the library's own bounds) and three for the operations around them; and the
    rounding of an exponential's argument a, which moves the result by |a| steps: three roundings
    in 2 v of the tanh form, two in z^2 / 2."""
    c0, c1 = (2 / torch.pi) ** 0.5, 0.044715
    if act == "gelu_tanh":
        return 7 + 3 * (2 * c0 * (z + c1 * z ** 3)).abs()
    if act == "gelu":
        return 7 + 2 * z * z
    return torch.full_like(z, 7.0)


def exact(z, act):
    """In 64 bits, without the cancellation of 1 + erf and 1 + tanh far below zero."""
    c0, c1 = (2 / torch.pi) ** 0.5, 0.044715
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * 0.5 ** 0.5)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * c0 * (z + c1 * z ** 3))
    return activation(z, act)


def values(T, N):
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.rand(T, N, generator=g, device="cuda") * 18 - 9
    z[0, :8] = torch.tensor([0.0, -0.0, -1e-8, 1e-8, -30.0, 30.0, -80.0, 80.0])
    return z.to(BF16)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [3, 300, 1100])
@pytest.mark.parametrize("keep", [False, True])
def test_values(T, act, keep):
    """z = x I exactly, fp32 out: one row and many, with the pre-activation stored or not."""
    N = 256
    x, eye = values(T, N), torch.eye(N, dtype=BF16, device="cuda")
    d = moe.linear_desc(T, N, N, moe.MOE_DTYPE_BF16, act, out_dtype=moe.MOE_DTYPE_FP32)
    ws, y = moe.alloc_workspace(d), torch.empty(T, N, device="cuda")
    pre = torch.empty(T, N, device="cuda") if keep else None
    moe.moe_linear(d, x, eye, None, None, y, ws, preact=pre)
    torch.cuda.synchronize()
    z = x.double()
    want = exact(z, act)
    off = (y.double() - want).abs() - want.abs() * steps(z, act) * STEP
    assert float(off.max()) <= 1e-37, (float(off.max()), float(z.flatten()[int(off.argmax())]))


@pytest.mark.parametrize("act", moe.ACT_NAMES)
@pytest.mark.parametrize("T", [3, 300])
def test_infinities(T, act):
    """What the formulas give at infinities and NaN, element by element: act(+inf) = inf, and
    relu(-inf) = 0; where the formula is -inf times 0, NaN."""
    N = 256
    x = values(T, N)
    eye = torch.eye(N, dtype=BF16, device="cuda")
    b = torch.zeros(N, dtype=BF16, device="cuda")
    b[3], b[5], b[9] = float("inf"), float("-inf"), float("nan")
    d = moe.linear_desc(T, N, N, moe.MOE_DTYPE_BF16, act)
    ws, y = moe.alloc_workspace(d), torch.empty(T, N, dtype=BF16, device="cuda")
    moe.moe_linear(d, x, eye, b, None, y, ws)
    torch.cuda.synchronize()
    assert bool((y[:, 3] == float("inf")).all()) and bool(torch.isnan(y[:, 9]).all())
    if act == "none":
        assert bool((y[:, 5] == float("-inf")).all())
    elif act == "relu":
        assert bool((y[:, 5] == 0).all())
    else:
        assert bool(torch.isnan(y[:, 5]).all())
    rest = [j for j in range(N) if j not in (3, 5, 9)]
    assert bool(torch.isfinite(y[:, rest]).all())
