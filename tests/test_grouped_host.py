"""Refusals of the experts' ragged products on the host (no GPU): every bad argument is
rejected before anything is launched."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe
from test_dense_host import FAKE, INVALID, SHAPE, SMALL, lib, status, ws  # noqa: F401

BF16 = moe.MOE_DTYPE_BF16
X, W, Y, DY, DX, DW, OFF = (FAKE * i for i in range(1, 8))


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), SHAPE), (dict(R=(1 << 24) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE),
    (dict(N=4), SHAPE), (dict(N=260), SHAPE), (dict(N=(1 << 18) + 8), SHAPE), (dict(K=0), SHAPE),
    (dict(K=100), SHAPE), (dict(K=(1 << 18) + 8), SHAPE), (dict(x_stride=248), SHAPE),
    (dict(x_stride=260), SHAPE), (dict(y_stride=-512), SHAPE), (dict(y_stride=504), SHAPE),
    (dict(dtype=moe.MOE_DTYPE_FP32), INVALID), (dict(dtype=moe.MOE_DTYPE_E4M3), INVALID),
    (dict(out_dtype=moe.MOE_DTYPE_FP16), INVALID), (dict(out_dtype=7), INVALID)])
def test_descriptor(lib, kw, want):  # noqa: F811
    d = moe.grouped_desc(**{**dict(R=4, E=3, N=512, K=256, dtype=BF16), **kw})
    assert moe.moe_grouped_linear_workspace_size(d) == 0
    assert status(moe.moe_grouped_linear, d, X, OFF, W, Y, ws()) == want
    assert status(moe.moe_grouped_linear_backward, d, DY, X, OFF, W, DX, DW, ws()) == want
    with pytest.raises(moe.MoeError):
        moe.alloc_workspace(d, device="cpu")


def test_forward_pointers(lib):  # noqa: F811
    d = moe.grouped_desc(4, 3, 512, 256, BF16)
    f = moe.moe_grouped_linear
    need = moe.moe_grouped_linear_workspace_size(d)
    assert need > 0
    for bad in ((None, OFF, W, Y), (X, None, W, Y), (X, OFF, None, Y), (X, OFF, W, None),
                (X + 8, OFF, W, Y), (X, OFF + 2, W, Y), (X, OFF, W + 4, Y), (X, OFF, W, Y + 2),
                (X, OFF, W, X), (X, OFF, W, W), (X, OFF, W, OFF)):
        assert status(f, d, *bad, ws()) == INVALID
    assert status(f, d, X, OFF, W, Y, ws(need - 1)) == SMALL
    assert status(f, d, X, OFF, W, Y, ws(addr=FAKE + 128)) == INVALID
    none = moe.grouped_desc(0, 3, 512, 256, BF16)
    assert status(f, none, None, OFF, None, None, ws()) == moe.MOE_OK


def test_backward_pointers(lib):  # noqa: F811
    d = moe.grouped_desc(4, 3, 512, 256, BF16)
    f = moe.moe_grouped_linear_backward
    for bad in ((None, X, OFF, W, DX, DW), (DY, None, OFF, W, DX, DW), (DY, X, None, W, DX, DW),
                (DY, X, OFF, None, DX, DW), (DY, X, OFF, W, DX + 8, DW), (DY, X, OFF, W, DX, DW + 4),
                (DY, X, OFF, W, DY, DW), (DY, X, OFF, W, X, DW), (DY, X, OFF, W, W, DW),
                (DY, X, OFF, W, DX, DX), (DY, X, OFF, W, DX, W), (DY, X, OFF, W, DX, X),
                (DY, X, OFF, W, None, DY), (DY, X, OFF, W, OFF, DW)):
        assert status(f, d, *bad, ws()) == INVALID, bad
    assert status(f, d, DY, X, OFF, W, DX, DW, ws(1024)) == SMALL
    c = moe.library().moe_grouped_linear_backward
    import ctypes
    for dw_dtype, accumulate in ((moe.MOE_DTYPE_FP16, 0), (9, 0), (BF16, 2), (BF16, -1)):
        assert c(ctypes.byref(d), DY, X, OFF, W, DX, DW, dw_dtype, accumulate, FAKE, 1 << 40,
                 0) == INVALID


def test_tensors(lib):  # noqa: F811
    """The binding refuses tensors that are not on a GPU, of another type or too small."""
    d = moe.grouped_desc(4, 3, 512, 256, BF16)
    x, off = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_grouped_linear(d, x, OFF, W, Y, ws(), stream=0)
    with pytest.raises(ValueError):
        moe.moe_grouped_linear(d, X, off, W, Y, ws(), stream=0)
    with pytest.raises(ValueError):
        moe.moe_grouped_linear(d, X, off[:3], W, Y, ws(), stream=0)
    with pytest.raises(ValueError):
        moe.moe_grouped_linear(d, X, off.long(), W, Y, ws(), stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(group=16), INVALID), (dict(group=0), INVALID), (dict(group=256), INVALID),
    (dict(rows=-1), SHAPE), (dict(rows=(1 << 27) + 1), SHAPE), (dict(K=48), SHAPE),
    (dict(K=0), SHAPE), (dict(K=(1 << 18) + 32), SHAPE), (dict(dtype=moe.MOE_DTYPE_FP32), INVALID),
    (dict(w=None), INVALID), (dict(w=W + 8), INVALID), (dict(q=None), INVALID),
    (dict(q=W), INVALID), (dict(scale=None), INVALID), (dict(scale=W), INVALID),
    (dict(values=Y + 4), INVALID), (dict(values=X), INVALID), (dict(q=DX, scale=DX), INVALID)])
def test_quantize_int4(lib, kw, want):  # noqa: F811
    a = {**dict(w=W, rows=4, K=64, group=32, q=X, scale=Y, values=DW, dtype=BF16), **kw}
    assert status(moe.moe_quantize_int4, **a) == want


def test_linear_int4(lib):  # noqa: F811
    f, d = moe.moe_linear_int4, moe.linear_desc(4, 512, 256, BF16)
    q, s, b, r = DY, DX, DW, OFF
    for group in (0, 16, 96, 256, -32):
        assert status(f, d, group, X, q, s, b, r, Y, ws()) == INVALID
    for kw, want in ((dict(K=264), SHAPE), (dict(dtype=moe.MOE_DTYPE_E4M3), INVALID),
                     (dict(T=-1), SHAPE), (dict(N=260), SHAPE), (dict(act=9), INVALID)):
        e = moe.linear_desc(**{**dict(T=4, N=512, K=256, dtype=BF16), **kw})
        assert status(f, e, 32, X, q, s, b, r, Y, ws()) == want, kw
    for bad in ((None, q, s, b, r, Y), (X, None, s, b, r, Y), (X, q, None, b, r, Y),
                (X, q, s, b, r, None), (X + 2, q, s, b, r, Y), (X, q + 4, s, b, r, Y),
                (X, q, s + 2, b, r, Y), (X, q, s, b + 2, r, Y), (X, q, s, b, r + 8, Y),
                (X, q, s, b, r, X), (X, q, s, b, r, q), (X, q, s, b, r, s), (X, q, s, b, r, b)):
        assert status(f, d, 32, *bad, ws()) == INVALID, bad
    assert status(f, d, 32, X, q, s, b, r, Y, ws(64)) == SMALL
    t = moe.linear_desc(4, 512, 256, BF16, y_stride=520)
    assert status(f, t, 32, X, q, s, b, Y, Y, ws()) == INVALID  # in place, other rows


def test_grouped_linear_int4(lib):  # noqa: F811
    f, d = moe.moe_grouped_linear_int4, moe.grouped_desc(4, 3, 512, 256, BF16)
    for group in (0, 48, 512):
        assert status(f, d, group, X, OFF, W, DW, Y, ws()) == INVALID
    for kw, want in ((dict(K=264), SHAPE), (dict(R=(1 << 20) + 1), SHAPE), (dict(E=0), SHAPE)):
        e = moe.grouped_desc(**{**dict(R=4, E=3, N=512, K=256, dtype=BF16), **kw})
        assert status(f, e, 32, X, OFF, W, DW, Y, ws()) == want
    for bad in ((None, OFF, W, DW, Y), (X, None, W, DW, Y), (X, OFF, None, DW, Y),
                (X, OFF, W, None, Y), (X, OFF, W, DW, None), (X, OFF, W + 8, DW, Y),
                (X, OFF, W, DW, X), (X, OFF, W, DW, W), (X, OFF, W, DW, DW), (X, OFF, W, DW, OFF)):
        assert status(f, d, 64, *bad, ws()) == INVALID, bad
    assert status(f, d, 64, X, OFF, W, DW, Y, ws(512)) == SMALL
