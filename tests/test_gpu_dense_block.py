"""The dense operators together, as examples/dense_block.py runs them, against the same block in
64 bits (needs a GB300).

Tolerances are relative L2 errors: each rounding to bf16 moves a tensor by at most 2^-8 of its
norm, each quantisation to E4M3 by at most 2^-4 of its own; the blocks pass an error on with a
factor near one (unit-variance rows, weights of variance 1/K), so they add up.
"""

import importlib.util
import os

import pytest
import torch

from dense_ref import dequantize, rel_l2, rms_norm

pytestmark = pytest.mark.gpu

EPS16, EPS8 = 2.0 ** -8, 2.0 ** -4


@pytest.fixture(scope="module")
def example():
    from routed_expert_ffn_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "dense_block.py")
    spec = importlib.util.spec_from_file_location("dense_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def ffn(h, w13, w2):
    g, u = (h @ w13.t()).chunk(2, 1)
    return (torch.nn.functional.silu(g) * u) @ w2.t()


def norm(x, w):
    return rms_norm(x, None, w, 1e-6)[1]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_decode(example, T, e4m3):
    H, I, layers = 320, 520, 2
    b = example.DecodeBlocks(T, H, I, layers, e4m3)
    y = b.step().clone()
    b.forward()
    assert torch.equal(y, b.y), "replayed and eager calls differ"
    s = b.x.double()
    for w, attn in zip(b.weights, b.attn):
        wp = dequantize(w["proj_q"], w["proj_e"], 128) if e4m3 else w["proj"].double()
        a = norm(attn.double(), torch.ones(H, dtype=torch.float64, device="cuda")) if e4m3 else attn.double()
        s = s + a @ wp.t()
        s = s + ffn(norm(s, w["norm"].double()), w["w13"].double(), w["w2"].double())
    want = norm(s, b.last.double())
    # a layer: s, h, the product of the gate, s again; at the end y
    tol = (4 * layers + 1) * EPS16 + (layers * EPS8 if e4m3 else 0.0)
    assert rel_l2(y, want) <= tol
    # the graph reads what the inputs hold when it runs
    b.x.mul_(-1)
    z = b.step().clone()
    b.forward()
    assert torch.equal(z, b.y) and not torch.equal(z, y)
    example.check(b.ws)


def test_gradients(example):
    T, H, I = 300, 264, 520
    b = example.TrainBlock(T, H, I)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = example.randn(g, T, H), example.randn(g, T, H, std=0.5)
    y = b.forward(x).clone()
    dx = b.backward(x, dy).clone()
    w = {k: v.double().requires_grad_() for k, v in b.w.items()}
    x64 = x.double().requires_grad_()
    z = norm(x64, w["norm1"]) @ w["wp"].t() + w["b"]
    s = x64 + torch.nn.functional.gelu(z, approximate="tanh")
    want = s + ffn(norm(s, w["norm2"]), w["w13"], w["w2"])
    want.backward(dy.double())
    assert rel_l2(y, want.detach()) <= 5 * EPS16  # h1, s, h2, the product of the gate, y
    # forward's four, and dg, du and h, the norm's input gradient, ds, dz, dh1, dx
    for k, v in b.grad.items():
        assert rel_l2(v, w[k].grad) <= 11 * EPS16, k
    assert rel_l2(dx, x64.grad) <= 11 * EPS16
    example.check(b.ws)


def test_training_lowers_the_loss(example):
    losses = example.main(["--train", "--T", "256", "--H", "128", "--I", "256", "--steps", "30"])
    assert losses[-1] < 0.8 * losses[0]


def test_decode_command(example):
    y = example.main(["--T", "2", "--H", "256", "--I", "512", "--layers", "2", "--steps", "3"])
    assert torch.isfinite(y.float()).all()
