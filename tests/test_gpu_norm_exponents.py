"""The row statistic of moe_add_rms_norm to its last bit, and the exponents of blocks whose
largest value lies at a step (needs a GB300)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_ffn_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def fp32_y(x, w):
    """y in fp32 from the mean rounded once: s r, then times w."""
    mean = x.double().square().mean(1, keepdim=True).float()
    return x * torch.rsqrt(mean + EPS) * w


def least_exponent(amax):
    """The least e with amax <= 448 2^e, in fp32 without a rounding (amax = m 2^e', 448 = 0.875 2^9)."""
    m, e = torch.frexp(amax)
    return e - 9 + (m > 0.875).int()


@pytest.mark.parametrize("T,H", [(4096, 1024), (2048, 7168), (8192, 256)])
def test_blocks_at_a_step(T, H):
    """The first block's largest value within 8 fp32 steps of 3.5 in every row.

    With the mean rounded once the kernel's y has the bits of the same fp32 operations wherever
    the threads' own sums do not turn that rounding: their error is some 2^-28 to 2^-27 of the
    mean against a spacing of 2^-24 to 2^-23, so in at most 1 of 8 rows.  Half of those move r,
    by one step, and a step meets the border in at most 2 of 17 rows: below 1 in 100."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, H, generator=g, device="cuda").clamp_(-3, 3)
    w = torch.randn(H, generator=g, device="cuda").mul_(0.1).clamp_(-0.15, 0.15).add_(1.0)
    w[0] = 1.0
    rest = x[:, 1:].double().square().sum(1)
    # x0 / sqrt((rest + x0^2) / H + eps) = 3.5, solved in 64 bits
    x0 = torch.sqrt(12.25 * (rest / H + EPS) / (1 - 12.25 / H)).float()
    step = torch.randint(-8, 9, (T,), generator=g, device="cuda", dtype=torch.int32)
    x[:, 0] = (x0.view(torch.int32) + step).view(torch.float32)
    y = torch.empty_like(x)
    q = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    e = torch.empty(T, H // 128, dtype=torch.int8, device="cuda")
    moe.moe_add_rms_norm(moe.norm_desc(T, H, moe.MOE_DTYPE_FP32, EPS), x, None, w, None, y, q, e)
    torch.cuda.synchronize()
    want = fp32_y(x, w)
    # the exponents are exactly those of the y that the call returns
    assert torch.equal(e.int(), least_exponent(y.view(T, -1, 128).abs().amax(2)))
    ew = least_exponent(want.view(T, -1, 128).abs().amax(2))
    assert 0.2 < float((ew[:, 0] == -7).float().mean()) < 0.8  # both sides of the step occur
    rows = float((y != want).any(1).float().mean())
    assert rows <= 1 / 8, f"{rows:.3f} of the rows have other bits"
    off = float((e[:, 0].int() != ew[:, 0]).float().mean())
    assert off <= 1 / 100, f"{off:.4f} of the exponents differ at the step"


@pytest.mark.parametrize("T,H", [(40, 1024), (40, 256), (40, 16384)])
def test_rows_of_any_magnitude(T, H):
    """Row i is of size 2^(3 i - 56), eps 0: sums of squares from below 2^-101 (where the integer
    units end) to near the end of fp32.  s r and its product with w round once each, the mean and
    r are good to 4 fp32 steps."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, H, generator=g, device="cuda")
    x = torch.ldexp(x, (3 * torch.arange(T, device="cuda") - 56)[:, None].clamp(max=54))
    w = torch.randn(H, generator=g, device="cuda")
    y = torch.empty_like(x)
    moe.moe_add_rms_norm(moe.norm_desc(T, H, moe.MOE_DTYPE_FP32, 0.0), x, None, w, None, y)
    torch.cuda.synchronize()
    want = x.double() / x.double().square().mean(1, keepdim=True).sqrt() * w.double()
    assert bool(((y.double() - want).abs() <= want.abs() * 8 * 2.0 ** -24).all())
