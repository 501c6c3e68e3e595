"""Plain 64-bit implementations of the dense operators and the error bounds their tests use.

The bounds count roundings: one rounding to a type is off by at most half a
step, ``finfo(t).eps / 2`` of the value; sums in fp32 add a few fp32 steps of
the sum of the terms' magnitudes.
"""

import torch

E4M3_MAX = 448.0
EPS32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the type's smallest numbers: what rounding near zero may cost."""
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def assert_within(got, want, bound, what):
    """|got - want| <= bound everywhere (bound: a tensor); NaN and infinities in the same places."""
    g, w = got.double().cpu(), want.double().cpu()
    b = bound.double().cpu() if torch.is_tensor(bound) else torch.full_like(w, float(bound))
    fin = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaN in other places"
    assert torch.equal(g[~fin & ~torch.isnan(w)], w[~fin & ~torch.isnan(w)]), f"{what}: infinities"
    over = ((g - w).abs() - b)[fin]
    if over.numel() and not bool((over <= 0).all()):
        i = int(over.argmax())
        raise AssertionError(f"{what}: off by {float((g - w).abs()[fin][i]):.4g}, allowed "
                             f"{float(b[fin][i]):.4g} at value {float(w[fin][i]):.4g} "
                             f"({int((over > 0).sum())} of {over.numel()} values)")


def dequantize(q, e, rows=1):
    """E4M3 codes [R,C] and int8 exponents of rows x 128 blocks -> float64."""
    v = q.view(torch.float8_e4m3fn).float().double()
    s = torch.exp2(e.double()).repeat_interleave(rows, 0).repeat_interleave(128, 1)
    return v * s[: v.shape[0], : v.shape[1]]


def rms_norm(x, residual, weight, eps):
    """(s, y) in 64 bits."""
    s = x.double() + (residual.double() if residual is not None else 0.0)
    return s, s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * weight.double()


def activation(z, act):
    f = torch.nn.functional
    return {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "silu": f.silu,
            "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[act](z)


def product_bound(a, b, K):
    """What fp32 accumulation of K exact products may be off by, for a [M,K] and b [N,K] in 64
    bits: every addition at most one step (2^-23) of the running sum, itself at most the sum of
    the products' magnitudes; the tensor cores add 16 products (or 32) at a time."""
    return (a.abs() @ b.abs().t()) * ((K / 8 + 8) * 2.0 ** -23)


def rel_l2(got, want):
    g, w = got.double(), want.double()
    n = float(w.norm())
    return float((g - w).norm()) / n if n else float((g - w).norm())
