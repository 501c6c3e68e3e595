"""The dense operators' binding refuses tensors that are smaller than the descriptor says or of
another type (no GPU: the library is a stand-in that records its calls)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe

BF16, FP16, FP32, INT8, U8 = (torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.uint8)


class Cuda(torch.Tensor):
    """A host tensor that says it is on the GPU."""
    is_cuda = True


def t(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Cuda)


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("moe_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, args))
            return moe.MOE_OK
        return call


@pytest.fixture()
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(moe, "_lib", lib)
    return lib


T, H, I, N, K = 6, 256, 136, 264, 384
WS = t(64, dtype=U8)

NORM = (moe.moe_add_rms_norm, lambda: moe.norm_desc(T, H, moe.MOE_DTYPE_BF16), dict(
    x=(T, H), residual=(T, H), weight=(H,), residual_out=(T, H), y=(T, H), y_q=((T, H), U8),
    scale_exp=((T, 2), INT8)))
NORM_BACK = (moe.moe_add_rms_norm_backward, lambda: moe.norm_desc(T, H, moe.MOE_DTYPE_BF16), dict(
    dy=(T, H), dresidual=(T, H), sum=(T, H), weight=(H,), dx=(T, H), dweight=((H,), FP32)))
LINEAR = (moe.moe_linear, lambda: moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, "silu"), dict(
    x=(T, K), w=(N, K), bias=(N,), residual=(T, N), y=(T, N), preact=((T, N), FP32)))
LINEAR32 = (moe.moe_linear, lambda: moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16,
                                                    out_dtype=moe.MOE_DTYPE_FP32), dict(
    x=(T, K), w=(N, K), bias=((N,), FP32), residual=((T, N), FP32), y=((T, N), FP32)))
LINEAR8 = (moe.moe_linear, lambda: moe.linear_desc(T, N, K, moe.MOE_DTYPE_E4M3), dict(
    x=((T, K), torch.float8_e4m3fn), w=((N, K), U8), bias=(N,), residual=(T, N), y=(T, N),
    x_scale=((T, 3), INT8), w_scale=((3, 3), INT8)))
LINEAR_BACK = (moe.moe_linear_backward,
               lambda: moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, "silu"), dict(
                   dy=(T, N), x=(T, K), w=(N, K), preact=((T, N), FP32), dx=(T, K), dw=(N, K),
                   dbias=((N,), FP32)))
FFN = (moe.moe_gated_ffn, lambda: moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16), dict(
    x=(T, H), w13=(2 * I, H), w2=(H, I), residual=(T, H), saved=((T, 2 * I), FP32), y=(T, H)))
FFN_BACK = (moe.moe_gated_ffn_backward, lambda: moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16), dict(
    dy=(T, H), x=(T, H), w13=(2 * I, H), w2=(H, I), saved=((T, 2 * I), FP32), dx=(T, H),
    dw13=((2 * I, H), FP32), dw2=((H, I), FP32)))
CALLS = dict(norm=NORM, norm_back=NORM_BACK, linear=LINEAR, linear_fp32=LINEAR32,
             linear_e4m3=LINEAR8, linear_back=LINEAR_BACK, ffn=FFN, ffn_back=FFN_BACK)


def shape_of(v):
    return v if isinstance(v[0], int) else v[0]


def type_of(v):
    return BF16 if isinstance(v[0], int) else v[1]


def args_of(spec):
    return {k: t(*shape_of(v), dtype=type_of(v)) for k, v in spec.items()}


def call(fn, d, a):
    a = dict(a)
    if fn is not moe.moe_add_rms_norm:
        a["ws"] = WS
    fn(d, stream=0, **a)


@pytest.mark.parametrize("name", CALLS)
def test_right_tensors_pass(lib, name):
    fn, desc, spec = CALLS[name]
    a = args_of(spec)
    call(fn, desc(), a)
    got = [p for p in lib.calls[0][1] if isinstance(p, int) and not isinstance(p, bool)]
    assert all(v.data_ptr() in got for v in a.values())
    # buffers for more rows serve fewer
    more = {k: t(*(2 * shape_of(v)[0],) + tuple(shape_of(v)[1:]), dtype=type_of(v))
            for k, v in spec.items()}
    call(fn, desc(), more)
    assert len(lib.calls) == 2


@pytest.mark.parametrize("name,arg", [(n, k) for n, (_, _, s) in CALLS.items() for k in s])
def test_a_row_less_or_another_type_is_refused(lib, name, arg):
    fn, desc, spec = CALLS[name]
    a = args_of(spec)
    full = a[arg]
    a[arg] = t(full.shape[0] - 1, *full.shape[1:], dtype=full.dtype)
    with pytest.raises(ValueError):
        call(fn, desc(), a)
    if (name, arg) == ("linear_back", "dw"):
        return  # its type goes to the library, which refuses what is neither x's nor fp32
    # of the same size, so that only its type is wrong
    other = {BF16: FP16, FP32: torch.int32, INT8: U8, U8: torch.bool,
             torch.float8_e4m3fn: torch.bool}[full.dtype]
    a[arg] = t(*full.shape, dtype=other)
    with pytest.raises(ValueError):
        call(fn, desc(), a)
    assert not lib.calls



def test_workspace_of_a_derived_descriptor():
    """A program's own class over a descriptor is one, as it was before the dense operators."""
    class Mine(moe.LayerDesc):
        pass
    with pytest.raises(moe.MoeError):  # a bad shape, not an unknown class
        moe.alloc_workspace(Mine(-1, 256, 8, 2, 128, moe.MOE_GATE_SOFTMAX_TOPK_RENORM, 0))
    with pytest.raises(TypeError):
        moe.alloc_workspace(object())
