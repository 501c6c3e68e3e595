"""Refusals of the dense operators on the host (no GPU): every bad argument is
rejected before anything is launched."""

import os

import pytest

import routed_expert_ffn_gb300 as moe

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from routed_expert_ffn_gb300 import build
        build.build()
    return moe.library()


class FakeWs(int):
    """An address with a size, in the place of a workspace tensor."""
    bytes = 1 << 40

    def numel(self):
        return self.bytes

    def element_size(self):
        return 1


def ws(n=1 << 40, addr=FAKE):
    w = FakeWs(addr)
    w.bytes = n
    return w


def status(fn, *a, **kw):
    kw.setdefault("stream", 0)
    try:
        fn(*a, **kw)
    except moe.MoeError as e:
        return e.status
    return moe.MOE_OK


BF16 = moe.MOE_DTYPE_BF16
INVALID, SHAPE, SMALL = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE,
                         moe.MOE_ERR_WORKSPACE_TOO_SMALL)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(H=0), SHAPE), (dict(H=4), SHAPE),
    (dict(H=4100), SHAPE), (dict(H=16392), SHAPE), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x_stride=4088), SHAPE), (dict(x_stride=4100), SHAPE), (dict(residual_stride=8), SHAPE),
    (dict(y_stride=-4096), SHAPE)])
def test_norm_descriptor(lib, kw, want):
    d = moe.norm_desc(**{**dict(T=4, H=4096, dtype=BF16), **kw})
    assert moe.moe_norm_workspace_size(d) == 0
    assert status(moe.moe_add_rms_norm, d, FAKE, FAKE, FAKE, FAKE, FAKE) == want
    assert status(moe.moe_add_rms_norm_backward, d, FAKE, FAKE, FAKE, FAKE, FAKE * 2, FAKE,
                  ws()) == want


def test_norm_pointers(lib):
    d = moe.norm_desc(4, 4096, BF16)
    f = moe.moe_add_rms_norm
    assert status(f, d, None, None, FAKE, None, FAKE) == INVALID
    assert status(f, d, FAKE, None, None, None, FAKE) == INVALID
    assert status(f, d, FAKE + 8, None, FAKE, None, FAKE) == INVALID
    assert status(f, d, FAKE, FAKE + 2, FAKE, None, FAKE) == INVALID
    assert status(f, d, FAKE, None, FAKE, None, None) == INVALID             # no output
    assert status(f, d, FAKE, None, FAKE, None, FAKE, FAKE, None) == INVALID  # codes without scales
    assert status(f, d, FAKE, None, FAKE, None, FAKE, None, FAKE) == INVALID
    s = moe.norm_desc(4, 4096, BF16, y_stride=8192)
    assert status(f, s, FAKE, None, FAKE, None, FAKE) == INVALID             # in place, other rows
    b = moe.moe_add_rms_norm_backward
    need = moe.moe_norm_workspace_size(d)
    assert need > 0
    assert status(b, d, FAKE, None, FAKE, FAKE, FAKE * 2, FAKE, ws(need - 1)) == SMALL
    assert status(b, d, FAKE, None, FAKE, FAKE, FAKE * 2, FAKE, ws(addr=FAKE + 16)) == INVALID
    assert status(b, d, FAKE, None, FAKE * 2, FAKE, FAKE * 2, FAKE, ws()) == INVALID  # dx is sum
    assert status(b, d, None, None, FAKE, FAKE, FAKE * 2, FAKE, ws()) == INVALID
    assert status(b, d, FAKE, None, FAKE, FAKE, None, FAKE, ws()) == INVALID


def test_strided_tensors_are_checked(lib):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        moe._rows(torch.zeros(4, 8), 0, 8)  # not on the GPU
