"""The experts' products together with the stage calls around them, as examples/expert_layer.py
runs them, against the same layer in 64 bits (needs a GB300)."""

import importlib.util
import os

import pytest
import torch

import int4_ref
import routed_expert_ffn_gb300 as moe
from dense_ref import assert_within, half_step, product_bound

pytestmark = pytest.mark.gpu

F16 = half_step(torch.float16)
TINY = 2.0 ** -25  # half of fp16's smallest number


@pytest.fixture(scope="module")
def example():
    from routed_expert_ffn_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def matrices(layer):
    if layer.int4:
        return (int4_ref.values(layer.q1, layer.s1, 64), int4_ref.values(layer.q2, layer.s2, 64))
    return layer.w1.double(), layer.w2.double()


def times(x, e, w):
    """(x w^T, what it is off by where x is off by e and the result is rounded to fp16)."""
    y = x @ w.t()
    b = e @ w.abs().t() + 2 * product_bound(x, w, x.shape[1])
    return y, b + (y.abs() + b) * F16 + TINY


def reference(layer):
    """(y, bound) from the experts and gates that the layer chose; every rounding counted."""
    w1, w2 = matrices(layer)
    token = (layer.perm // layer.k).long()
    x = layer.x.double()[token]
    ends = layer.offsets.tolist()
    out, err = torch.zeros(x.shape[0], layer.H, dtype=torch.float64, device="cuda"), None
    err = torch.zeros_like(out)
    for e in range(layer.E):
        rows = slice(ends[e], ends[e + 1])
        if ends[e + 1] == ends[e]:
            continue
        # (x is bf16: as fp16 it is off by half a step, and by TINY near zero)
        h, eh = times(x[rows], x[rows].abs() * F16 + TINY, w1[e])
        r = h.clamp(min=0.0)
        a, ea = r.square(), 2 * r * eh + eh.square()
        ea = ea + (a + ea) * F16 + TINY
        out[rows], err[rows] = times(a, ea, w2[e])
    y, ey = torch.zeros(layer.T, layer.H, dtype=torch.float64, device="cuda"), None
    ey = torch.zeros_like(y)
    g = layer.gates_perm.double()[:, None]
    y.index_add_(0, token, g * out)
    ey.index_add_(0, token, g * err + (g * out).abs() * layer.k * 2.0 ** -23)
    return y, ey + (y.abs() + ey) * half_step(torch.bfloat16)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("T", [1, 7, 150])
def test_forward(example, T, int4):
    layer = example.ExpertLayer(T, 512, 320, 16, 4, int4, seed=T)
    layer.forward()
    layer.check()
    assert int(layer.offsets[-1]) == T * 4
    want, bound = reference(layer)
    assert_within(layer.y, want, bound, "y")


@pytest.mark.parametrize("int4", [False, True])
def test_replayed_on_new_tokens(example, int4):
    layer = example.ExpertLayer(9, 256, 192, 8, 2, int4)
    layer.step()
    layer.x.copy_(torch.randn(9, 256, device="cuda"))
    layer.step()
    layer.check()
    want, bound = reference(layer)
    assert_within(layer.y, want, bound, "y")


def test_gradients(example):
    """dw1, dw2 and the rows' gradient against the 64-bit formulas at the layer's own h and a."""
    layer = example.ExpertLayer(60, 256, 192, 8, 2)
    layer.forward()
    dy = torch.randn(60, 256, device="cuda") * 0.1
    dw1, dw2, drows = layer.backward(dy)
    layer.check()
    token, ends = (layer.perm // layer.k).long(), layer.offsets.tolist()
    dout = (dy[token] * layer.gates_perm[:, None]).half().double()
    h, a, rows = layer.h.double(), layer.a.double(), layer.rows.double()
    for e in range(layer.E):
        s = slice(ends[e], ends[e + 1])
        m = ends[e + 1] - ends[e]
        w1, w2 = layer.w1[e].double(), layer.w2[e].double()
        want = dout[s].t() @ a[s]
        assert_within(dw2[e], want, product_bound(dout[s].t(), a[s].t(), m) + want.abs() * 2.0 ** -24,
                      f"dw2 of expert {e}")
        if m == 0:
            assert not bool(dw1[e].any())
            continue
        da, ea = times(dout[s], torch.zeros_like(dout[s]), w2.t())
        # da is rounded, and two products in fp16 after it
        dh = da * 2 * h[s].clamp(min=0.0)
        eh = ea * 2 * h[s].clamp(min=0.0)
        eh = eh + 2 * (dh.abs() + eh) * F16 + 4 * TINY * (1 + h[s].abs())
        want = dh.t() @ rows[s]
        bound = eh.t() @ rows[s].abs() + product_bound(dh.t(), rows[s].t(), m)
        assert_within(dw1[e], want, bound + want.abs() * 2.0 ** -24, f"dw1 of expert {e}")
        want, bound = times(dh, eh, w1.t())
        assert_within(drows[s], want, bound, f"rows of expert {e}")


@pytest.mark.parametrize("args", [["--T", "5", "--steps", "3"], ["--T", "5", "--steps", "3", "--int4"],
                                  ["--train", "--T", "128", "--steps", "2"]])
def test_runs(example, args, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["expert_layer.py"] + args)
    example.main()
    assert capsys.readouterr().out
