"""Outputs of the dense operators at the address of something that the same launch reads or
writes are refused on the host; what the call has read by then is not (no GPU)."""

import os

import pytest
import torch

import routed_expert_ffn_gb300 as moe

A = 1 << 20  # addresses A, 2A, ...: aligned, never dereferenced on the host


class Workspace(int):
    def numel(self):
        return 1 << 40

    def element_size(self):
        return 1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(moe.LIB_PATH):
        from routed_expert_ffn_gb300 import build
        build.build()


def refused(fn, d, **a):
    if fn is not moe.moe_add_rms_norm:
        a["ws"] = Workspace(1 << 30)
    try:
        fn(d, stream=0, **a)
    except moe.MoeError as e:
        return e.status == moe.MOE_ERR_INVALID_ARG
    return False


def placed(names, **at):
    """Each name at an address of its own; those in `at` where it says."""
    a = {n: A * (i + 1) for i, n in enumerate(names)}
    for k, v in at.items():
        a[k] = a[v] if isinstance(v, str) else v
    return a


# Without a GPU a call that is not refused ends at the device check; with one it would be launched.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")

NORM = ("x", "residual", "weight", "residual_out", "y", "y_q", "scale_exp")
LINEAR = ("x", "w", "bias", "residual", "preact", "y")
BACK = ("dy", "x", "w", "preact", "dx", "dw", "dbias")
FFN = ("x", "w13", "w2", "residual", "saved", "y")
FFN_BACK = ("dy", "x", "w13", "w2", "saved", "dx", "dw13", "dw2")


def test_norm():
    d = moe.norm_desc(4, 256, moe.MOE_DTYPE_BF16)
    f = moe.moe_add_rms_norm
    assert not refused(f, d, **placed(NORM))
    for other in ("x", "residual", "residual_out", "y"):
        assert refused(f, d, **placed(NORM, y_q=other))
    assert not refused(f, d, **placed(NORM, y="residual"))
    wide = moe.norm_desc(4, 256, moe.MOE_DTYPE_BF16, y_stride=512)
    assert refused(f, wide, **placed(NORM, y="residual"))  # other rows' residual
    assert not refused(f, d, **placed(NORM, residual_out="residual"))
    assert not refused(f, d, **placed(NORM, residual_out="x"))


def test_linear():
    d = moe.linear_desc(4, 256, 512, moe.MOE_DTYPE_BF16, "silu")
    f = moe.moe_linear
    assert not refused(f, d, **placed(LINEAR))
    for other in ("x", "w", "bias", "residual", "y"):
        assert refused(f, d, **placed(LINEAR, preact=other))
    assert not refused(f, d, **placed(LINEAR, y="residual"))
    wide = moe.linear_desc(4, 256, 512, moe.MOE_DTYPE_BF16, "silu", out_dtype=moe.MOE_DTYPE_FP32)
    assert not refused(f, wide, **placed(LINEAR, preact="residual"))  # element for element


def test_linear_backward():
    f = moe.moe_linear_backward
    d = moe.linear_desc(4, 256, 512, moe.MOE_DTYPE_BF16, "silu")
    plain = moe.linear_desc(4, 256, 512, moe.MOE_DTYPE_BF16)
    assert not refused(f, d, **placed(BACK))
    for other in ("x", "w", "dx"):
        assert refused(f, d, **placed(BACK, dw=other))
    for other in ("dy", "preact", "x", "w", "dx", "dw"):
        assert refused(f, d, **placed(BACK, dbias=other))
    assert not refused(f, d, **placed(BACK, dw="dy"))      # read by the launch before
    assert refused(f, plain, **placed(BACK, dw="dy"))
    assert not refused(f, d, **{**placed(BACK, dw="w"), "dx": None})  # w is not read


def test_gated_ffn():
    d = moe.ffn_desc(4, 256, 512, moe.MOE_DTYPE_BF16)
    f = moe.moe_gated_ffn
    assert not refused(f, d, **placed(FFN))
    for other in ("x", "w13", "w2", "residual", "y"):
        assert refused(f, d, **placed(FFN, saved=other))
    assert not refused(f, d, **placed(FFN, y="residual"))
    assert not refused(f, d, **placed(FFN, residual="x"))


def test_gated_ffn_backward():
    d = moe.ffn_desc(4, 256, 512, moe.MOE_DTYPE_BF16)
    f = moe.moe_gated_ffn_backward
    assert not refused(f, d, **placed(FFN_BACK))
    for other in ("x", "w13", "dy", "dx", "dw2"):
        assert refused(f, d, **placed(FFN_BACK, dw13=other))
    for other in ("dy", "w13", "x", "dx", "dw13"):
        assert refused(f, d, **placed(FFN_BACK, dw2=other))
    assert not refused(f, d, **placed(FFN_BACK, dw2="w2"))  # read by the launch before
    assert not refused(f, d, **{**placed(FFN_BACK, dw13="w13"), "dx": None})
