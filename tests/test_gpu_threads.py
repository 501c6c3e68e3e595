"""Calls from other host threads than the first (needs a GB300)."""

import os
import subprocess
import sys
import threading

import pytest
import torch

import routed_expert_ffn_gb300 as moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_ffn_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def randn(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def in_a_new_thread(call):
    """The exception that `call` raises in a thread which has made no CUDA call before, or None."""
    got = []

    def run():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            got.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return got[0] if got else None


@pytest.mark.parametrize("T", [4, 1100])
def test_the_first_cuda_call_of_a_thread(T):
    x, w = randn(1, T, 520), randn(2, 264, 520, std=1 / 23)
    d = moe.linear_desc(T, 264, 520, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    want, y = torch.empty(T, 264, dtype=BF16, device="cuda"), randn(3, T, 264)
    stream = torch.cuda.current_stream().cuda_stream
    moe.moe_linear(d, x, w, None, None, want, ws)  # what is set up once is set up
    assert in_a_new_thread(lambda: moe.moe_linear(d, x, w, None, None, y, ws, stream=stream)) is None
    assert torch.equal(y, want)
    dy, dx, dw = randn(4, T, 264), torch.empty_like(x), torch.empty_like(w)
    moe.moe_linear_backward(d, dy, x, w, None, dx, dw, None, ws)
    a, b = torch.empty_like(x), torch.empty_like(w)
    assert in_a_new_thread(lambda: moe.moe_linear_backward(d, dy, x, w, None, a, b, None, ws,
                                                           stream=stream)) is None
    assert torch.equal(a, dx) and torch.equal(b, dw)
    f = moe.ffn_desc(T, 520, 264, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(f)
    w13, w2 = randn(5, 528, 520, std=1 / 23), randn(6, 520, 264, std=1 / 16)
    moe.moe_gated_ffn(f, x, w13, w2, None, None, dx, ws)
    assert in_a_new_thread(lambda: moe.moe_gated_ffn(f, x, w13, w2, None, None, a, ws,
                                                     stream=stream)) is None
    assert torch.equal(a, dx)


def test_a_layer_from_a_new_thread():
    """The layer keeps its tensor maps; with other buffers a new thread makes them."""
    T, H, E, k, I = 300, 256, 8, 2, 128
    d = moe.desc(T, H, E, k, I, moe.MOE_GATE_SOFTMAX_TOPK_RENORM, shared=False)
    stream = torch.cuda.current_stream().cuda_stream
    out = []
    for thread in (False, True):
        ws = moe.alloc_workspace(d)
        tensors = (randn(1, E, H, dtype=torch.float32), randn(2, E, 2 * I, H, std=1 / 16),
                   randn(3, E, H, I, std=1 / 11))
        w = moe.layer_weights(*tensors)
        x, y = randn(4, T, H), torch.empty(T, H, dtype=BF16, device="cuda")
        call = lambda: moe.moe_layer_forward(d, w, x, y, ws, stream=stream)  # noqa: E731
        if thread:
            assert in_a_new_thread(call) is None
        else:
            call()
        torch.cuda.synchronize()
        out.append((y, ws, tensors, x))  # (kept: the second round has buffers of its own)
    assert torch.equal(out[0][0], out[1][0])


def test_first_calls_of_every_kernel_from_many_threads():
    """With sizes that take different amounts of shared memory; in a process of its own, because
    only a kernel's first calls set how much it may have."""
    worker = os.path.join(os.path.dirname(os.path.abspath(__file__)), "threads_worker.py")
    p = subprocess.run([sys.executable, worker], capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, (p.stdout + p.stderr)[-3000:]
    assert p.stdout.strip().endswith("ok")
