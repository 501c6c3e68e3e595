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


LINEAR = dict(T=4, N=256, K=512, dtype=BF16)


def linear(d, **kw):
    a = {**dict(x=FAKE, w=FAKE * 2, bias=None, residual=None, y=FAKE * 3, ws=ws()), **kw}
    return status(moe.moe_linear, d, **a)


def linear_back(d, **kw):
    a = {**dict(dy=FAKE, x=FAKE, w=FAKE, preact=None, dx=FAKE * 2, dw=FAKE * 3, dbias=None,
                ws=ws()), **kw}
    return status(moe.moe_linear_backward, d, **a)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(N=0), SHAPE), (dict(N=12), SHAPE),
    (dict(K=4), SHAPE), (dict(K=516), SHAPE), (dict(N=(1 << 18) + 8), SHAPE),
    (dict(dtype=2), INVALID), (dict(dtype=4), INVALID), (dict(act=5), INVALID),
    (dict(act=-1), INVALID), (dict(out_dtype=moe.MOE_DTYPE_FP16), INVALID),
    (dict(out_dtype=moe.MOE_DTYPE_E4M3), INVALID), (dict(x_stride=504), SHAPE),
    (dict(x_stride=516), SHAPE), (dict(y_stride=-256), SHAPE), (dict(residual_stride=260), SHAPE),
    (dict(dtype=3, K=520), SHAPE), (dict(dtype=3, x_stride=520), SHAPE),
    (dict(dtype=3, out_dtype=moe.MOE_DTYPE_FP16), INVALID)])
def test_linear_descriptor(lib, kw, want):
    d = moe.linear_desc(**{**LINEAR, **kw})
    assert moe.moe_linear_workspace_size(d) == 0
    assert linear(d) == want
    assert linear_back(d) == want


def test_linear_pointers(lib):
    d = moe.linear_desc(**LINEAR)
    need = moe.moe_linear_workspace_size(d)
    assert linear(d, x=None) == INVALID
    assert linear(d, w=FAKE + 2) == INVALID
    assert linear(d, y=None) == INVALID
    assert linear(d, bias=FAKE + 4) == INVALID
    assert linear(d, residual=FAKE + 8) == INVALID
    assert linear(d, x_scale=FAKE) == INVALID                   # scales of 16-bit operands
    assert linear(d, y=FAKE) == INVALID                         # y over x
    assert linear(d, ws=ws(need - 1)) == SMALL
    assert linear(d, ws=ws(addr=FAKE + 128)) == INVALID
    s = moe.linear_desc(**LINEAR, y_stride=512)
    assert linear(s, residual=FAKE * 3) == INVALID              # in place, other rows
    q = moe.linear_desc(**{**LINEAR, "dtype": moe.MOE_DTYPE_E4M3})
    assert linear(q) == INVALID                                 # no scales
    assert linear(q, x_scale=FAKE) == INVALID
    assert linear(q, x_scale=FAKE, w_scale=FAKE, preact=FAKE) == INVALID
    z = moe.linear_desc(**{**LINEAR, "T": 0})
    assert linear(z, x=None, y=None) == moe.MOE_OK              # nothing to do


def test_linear_backward_pointers(lib):
    d = moe.linear_desc(**LINEAR, act="silu")
    assert linear_back(d) == INVALID                            # no pre-activation
    assert linear_back(d, preact=FAKE, dy=None) == INVALID
    assert linear_back(d, preact=FAKE, x=None) == INVALID       # dw wants x
    assert linear_back(d, preact=FAKE, w=None) == INVALID       # dx wants w
    assert linear_back(d, preact=FAKE, dx=FAKE) == INVALID      # dx over dy
    assert linear_back(d, preact=FAKE, dbias=FAKE + 4) == INVALID
    assert linear_back(d, preact=FAKE, ws=ws(64)) == SMALL
    q = moe.linear_desc(**{**LINEAR, "dtype": moe.MOE_DTYPE_E4M3})
    assert linear_back(q) == INVALID


FFN = dict(T=4, H=256, I=512, dtype=BF16)


def ffn(d, **kw):
    a = {**dict(x=FAKE, w13=FAKE, w2=FAKE, residual=None, saved=None, y=FAKE * 2, ws=ws()), **kw}
    return status(moe.moe_gated_ffn, d, **a)


def ffn_back(d, **kw):
    a = {**dict(dy=FAKE, x=FAKE, w13=FAKE, w2=FAKE, saved=FAKE, dx=FAKE * 2, dw13=None, dw2=None,
                ws=ws()), **kw}
    return status(moe.moe_gated_ffn_backward, d, **a)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(H=4), SHAPE), (dict(H=260), SHAPE),
    (dict(I=0), SHAPE), (dict(I=(1 << 17) + 8), SHAPE), (dict(dtype=2), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID)])
def test_ffn_descriptor(lib, kw, want):
    d = moe.ffn_desc(**{**FFN, **kw})
    assert moe.moe_gated_ffn_workspace_size(d) == 0
    assert ffn(d) == want
    assert ffn_back(d) == want


def test_ffn_pointers(lib):
    d = moe.ffn_desc(**FFN)
    for k in ("x", "w13", "w2", "y"):
        assert ffn(d, **{k: None}) == INVALID
    assert ffn(d, residual=FAKE + 2) == INVALID
    assert ffn(d, saved=FAKE + 4) == INVALID
    assert ffn(d, y=FAKE) == INVALID
    assert ffn(d, ws=ws(moe.moe_gated_ffn_workspace_size(d) - 1)) == SMALL
    for k in ("dy", "w2", "saved", "w13"):
        assert ffn_back(d, **{k: None}) == INVALID
    assert ffn_back(d, x=None, dw13=FAKE) == INVALID
    assert ffn_back(d, dx=FAKE) == INVALID
    assert ffn_back(d, ws=ws(64)) == SMALL
    z = moe.ffn_desc(**{**FFN, "T": 0})
    assert ffn(z, x=None, y=None) == moe.MOE_OK
