"""A layer of experts whose activation is not SwiGLU, from the framework's stage calls and the
experts' products: router, dispatch, up projection, squared ReLU, down projection, combine.

    serve    fp16 experts, or experts in 4 bits (--int4), captured once in a CUDA graph
    train    forward, backward and an SGD step of the experts' matrices on a regression target

    python examples/expert_layer.py [--T 16] [--H 4096] [--I 1536] [--E 32] [--k 8] [--int4]
    python examples/expert_layer.py --train [--T 2048] [--H 1024] [--I 768] [--E 8] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_expert_ffn_gb300 as moe  # noqa: E402

GROUP = 64


class ExpertLayer:
    """y = sum over a token's k experts of g * W2 relu(W1 x)^2; x [T,H] bf16 in ``self.x``, y in
    ``self.y``; the experts' rows and matrices are fp16, or 4-bit codes with scales."""

    def __init__(self, T, H, I, E, k, int4=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.T, self.H, self.I, self.E, self.k, self.int4 = T, H, I, E, k, int4
        R = T * k
        self.d = moe.desc(T, H, E, k, I, moe.MOE_GATE_SOFTMAX_TOPK_RENORM)
        self.ws = moe.alloc_workspace(self.d)
        self.w_router = rn(E, H) * H ** -0.5
        self.w1, self.w2 = (rn(E, I, H) * H ** -0.5).half(), (rn(E, H, I) * I ** -0.5).half()
        self.up = moe.grouped_desc(R, E, I, H, moe.MOE_DTYPE_FP16)
        self.down = moe.grouped_desc(R, E, H, I, moe.MOE_DTYPE_FP16)
        # one buffer for both: calls on one stream follow each other
        n = max(moe.moe_grouped_linear_workspace_size(d) for d in (self.up, self.down))
        self.products = torch.empty(n, dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(self.products)
        if int4:
            self.q1, self.s1 = self.quantized(self.w1)
            self.q2, self.s2 = self.quantized(self.w2)
        new = lambda *s, dt=torch.float16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        i32 = torch.int32
        self.x, self.y = rn(T, H).bfloat16(), new(T, H, dt=torch.bfloat16)
        self.logits, self.ids = new(T, E, dt=torch.float32), new(T, k, dt=i32)
        self.gates, self.gates_perm = new(T, k, dt=torch.float32), new(R, dt=torch.float32)
        self.counts, self.offsets = new(E, dt=i32), new(E + 1, dt=i32)
        self.perm, self.inverse = new(R, dt=i32), new(R, dt=i32)
        self.h, self.out = new(R, I), new(R, H)
        self.graph = None

    def quantized(self, w):
        E, N, K = w.shape
        q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(E, N, -(-K // GROUP), dtype=w.dtype, device="cuda")
        moe.moe_quantize_int4(w, E * N, K, GROUP, q, s)
        return q, s

    def route(self):
        moe.moe_route(self.d, self.x, self.w_router, None, self.logits, self.ids, self.gates, None,
                      self.ws)
        moe.moe_build_dispatch(self.d, self.ids, self.gates, self.counts, self.offsets, self.perm,
                               self.inverse, self.gates_perm, self.ws)
        return self.x.half()[torch.div(self.perm, self.k, rounding_mode="floor")]

    def forward(self):
        self.rows = self.route()
        if self.int4:
            moe.moe_grouped_linear_int4(self.up, GROUP, self.rows, self.offsets, self.q1, self.s1,
                                        self.h, self.products)
        else:
            moe.moe_grouped_linear(self.up, self.rows, self.offsets, self.w1, self.h, self.products)
        self.a = torch.relu(self.h).square()
        if self.int4:
            moe.moe_grouped_linear_int4(self.down, GROUP, self.a, self.offsets, self.q2, self.s2,
                                        self.out, self.products)
        else:
            moe.moe_grouped_linear(self.down, self.a, self.offsets, self.w2, self.out, self.products)
        moe.moe_combine(self.d, self.out, self.inverse, self.gates, self.y)

    def step(self):
        """One pass; captured at the first."""
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.forward()
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.forward()
        self.graph.replay()

    def backward(self, dy):
        """(dw1, dw2) in fp32 and the rows' gradient of the experts' part, from dy [T,H] fp32."""
        token = torch.div(self.perm, self.k, rounding_mode="floor")
        dout = (dy[token] * self.gates_perm[:, None]).half()
        da, dw2 = torch.empty_like(self.a), torch.empty(self.w2.shape, device="cuda")
        moe.moe_grouped_linear_backward(self.down, dout, self.a, self.offsets, self.w2, da, dw2,
                                        self.products)
        dh = da * 2 * torch.relu(self.h)
        drows, dw1 = torch.empty_like(self.rows), torch.empty(self.w1.shape, device="cuda")
        moe.moe_grouped_linear_backward(self.up, dh, self.rows, self.offsets, self.w1, drows, dw1,
                                        self.products)
        return dw1, dw2, drows

    def check(self):
        for ws in (self.ws, self.products):
            status, raw = moe.moe_get_device_status(ws)
            if status != moe.MOE_OK:
                raise RuntimeError(f"device status {status} ({raw:#x})")


def train(a):
    layer = ExpertLayer(a.T, a.H, a.I, a.E, a.k)
    target = torch.randn(a.T, a.H, device="cuda") * 0.5
    for step in range(a.steps):
        layer.forward()
        diff = layer.y.float() - target
        dw1, dw2, _ = layer.backward(diff / a.T)
        layer.w1 -= (a.lr * dw1).half()
        layer.w2 -= (a.lr * dw2).half()
        if step % 5 == 0 or step == a.steps - 1:
            print(f"step {step}: loss {float(diff.square().mean()):.4f}")
    layer.check()


def serve(a):
    layer = ExpertLayer(a.T, a.H, a.I, a.E, a.k, a.int4)
    layer.step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        layer.step()
    end.record()
    torch.cuda.synchronize()
    layer.check()
    print(f"{'4-bit' if a.int4 else 'fp16'} experts, {a.T} tokens: "
          f"{start.elapsed_time(end) / a.steps * 1e3:.1f} us a pass")


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--train", action="store_true")
    p.add_argument("--int4", action="store_true")
    p.add_argument("--T", type=int)
    p.add_argument("--H", type=int)
    p.add_argument("--I", type=int)
    p.add_argument("--E", type=int)
    p.add_argument("--k", type=int)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--lr", type=float, default=0.02)
    a = p.parse_args()
    sizes = dict(T=2048, H=1024, I=768, E=8, k=2) if a.train else dict(T=16, H=4096, I=1536, E=32, k=8)
    for name, value in sizes.items():
        if getattr(a, name) is None:
            setattr(a, name, value)
    train(a) if a.train else serve(a)


if __name__ == "__main__":
    main()
