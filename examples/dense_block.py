"""The dense half of a transformer block, as a serving and as a training program would run it.

A block here is what surrounds attention: its output projection onto the residual stream, the
norm, and the gated feed-forward block; between blocks the norm that adds the residual.

    decode   the blocks over a few rows, with bf16 or E4M3 projections, captured once in a CUDA
             graph and replayed
    train    forward, backward and an SGD step of one block on a regression target

    python examples/dense_block.py [--T 4] [--H 4096] [--I 14336] [--layers 4] [--e4m3]
    python examples/dense_block.py --train [--T 2048] [--H 1024] [--I 2816] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_expert_ffn_gb300 as moe  # noqa: E402

EPS = 1e-6


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


class DecodeBlocks:
    """`layers` blocks over T rows: one graph launch a step.

    The attention output of a step goes into ``self.attn[layer]``, the block's input into
    ``self.x``; ``step()`` leaves the last block's output, normalised, in ``self.y``.
    """

    def __init__(self, T, H, I, layers, e4m3=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.e4m3 = T, H, e4m3
        self.weights = []
        for _ in range(layers):
            w = dict(proj=randn(g, H, H, std=H ** -0.5), norm=randn(g, H, std=0.1) + 1,
                     w13=randn(g, 2 * I, H, std=H ** -0.5), w2=randn(g, H, I, std=I ** -0.5))
            if e4m3:  # 128 x 128 blocks of codes, one exponent each
                w["proj_q"] = torch.empty(H, H, dtype=torch.uint8, device="cuda")
                w["proj_e"] = torch.empty(-(-H // 128), -(-H // 128), dtype=torch.int8, device="cuda")
                moe.moe_quantize_fp8(w["proj"], 1, H, H, w["proj_q"], w["proj_e"])
            self.weights.append(w)
        self.last = randn(g, H, std=0.1) + 1
        self.attn = [randn(g, T, H) for _ in range(layers)]
        self.x = randn(g, T, H)
        self.stream = torch.empty_like(self.x)  # the residual stream
        self.h, self.y = torch.empty_like(self.x), torch.empty_like(self.x)
        self.codes = torch.empty(T, H, dtype=torch.uint8, device="cuda")
        self.exps = torch.empty(T, -(-H // 128), dtype=torch.int8, device="cuda")
        self.ones = torch.ones(H, dtype=torch.bfloat16, device="cuda")

        self.norm = moe.norm_desc(T, H, moe.MOE_DTYPE_BF16, EPS)
        self.proj = moe.linear_desc(T, H, H, moe.MOE_DTYPE_E4M3 if e4m3 else moe.MOE_DTYPE_BF16)
        self.ffn = moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16)
        # one buffer for both: calls on one stream follow each other
        sizes = (moe.moe_linear_workspace_size(self.proj), moe.moe_gated_ffn_workspace_size(self.ffn))
        self.ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(self.ws)
        self.graph = None

    def forward(self):
        x = self.x
        for w, attn in zip(self.weights, self.attn):
            # the residual stream goes on through the projection's epilogue
            if self.e4m3:
                moe.moe_add_rms_norm(self.norm, attn, None, self.ones, None, None, self.codes, self.exps)
                moe.moe_linear(self.proj, self.codes, w["proj_q"], None, x, self.stream, self.ws,
                               x_scale=self.exps, w_scale=w["proj_e"])
            else:
                moe.moe_linear(self.proj, attn, w["proj"], None, x, self.stream, self.ws)
            moe.moe_add_rms_norm(self.norm, self.stream, None, w["norm"], None, self.h)
            moe.moe_gated_ffn(self.ffn, self.h, w["w13"], w["w2"], self.stream, None, self.stream,
                              self.ws)
            x = self.stream
        moe.moe_add_rms_norm(self.norm, x, None, self.last, None, self.y)

    def step(self):
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.forward()  # the first call sets the kernels up
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.forward()
        self.graph.replay()
        return self.y

    def bytes_read(self):
        per = sum(t.numel() * t.element_size() for k, t in self.weights[0].items()
                  if k not in (("proj",) if self.e4m3 else ()))
        return per * len(self.weights)


class TrainBlock:
    """One block with its gradients: x -> x + act(norm(x) Wp^T + b) = s -> s + FFN(norm(s)).

    Weights in bf16 beside fp32 masters; gradients in fp32.
    """

    NAMES = ("norm1", "wp", "b", "norm2", "w13", "w2")

    def __init__(self, T, H, I, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        f = lambda *s, std: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
        self.master = dict(norm1=1 + f(H, std=0.1), wp=f(H, H, std=H ** -0.5), b=f(H, std=0.1),
                           norm2=1 + f(H, std=0.1), w13=f(2 * I, H, std=H ** -0.5),
                           w2=f(H, I, std=I ** -0.5))
        self.w = {k: v.bfloat16() for k, v in self.master.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.norm = moe.norm_desc(T, H, moe.MOE_DTYPE_BF16, EPS)
        self.proj = moe.linear_desc(T, H, H, moe.MOE_DTYPE_BF16, act="gelu_tanh")
        self.ffn = moe.ffn_desc(T, H, I, moe.MOE_DTYPE_BF16)
        sizes = (moe.moe_norm_workspace_size(self.norm), moe.moe_linear_workspace_size(self.proj),
                 moe.moe_gated_ffn_workspace_size(self.ffn))
        self.ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(self.ws)
        row = lambda n=H, t=torch.bfloat16: torch.empty(T, n, dtype=t, device="cuda")  # noqa: E731
        self.h1, self.s, self.h2, self.y, self.dx = row(), row(), row(), row(), row()
        self.t1, self.t2 = row(), row()
        self.preact, self.saved = row(t=torch.float32), row(2 * I, torch.float32)

    def forward(self, x):
        w, ws = self.w, self.ws
        moe.moe_add_rms_norm(self.norm, x, None, w["norm1"], None, self.h1)
        moe.moe_linear(self.proj, self.h1, w["wp"], w["b"], x, self.s, ws, preact=self.preact)
        moe.moe_add_rms_norm(self.norm, self.s, None, w["norm2"], None, self.h2)
        moe.moe_gated_ffn(self.ffn, self.h2, w["w13"], w["w2"], self.s, self.saved, self.y, ws)
        return self.y

    def backward(self, x, dy):
        """Gradients of every weight into self.grad, of x returned."""
        w, g, ws = self.w, self.grad, self.ws
        moe.moe_gated_ffn_backward(self.ffn, dy, self.h2, w["w13"], w["w2"], self.saved, self.t1,
                                   g["w13"], g["w2"], ws)
        # s feeds the norm and the residual: dy goes on as dresidual
        moe.moe_add_rms_norm_backward(self.norm, self.t1, dy, self.s, w["norm2"], self.t2,
                                      g["norm2"], ws)
        moe.moe_linear_backward(self.proj, self.t2, self.h1, w["wp"], self.preact, self.t1, g["wp"],
                                g["b"], ws)
        moe.moe_add_rms_norm_backward(self.norm, self.t1, self.t2, x, w["norm1"], self.dx,
                                      g["norm1"], ws)
        return self.dx

    def sgd(self, lr):
        for k in self.NAMES:
            self.master[k].add_(self.grad[k], alpha=-lr)
            self.w[k].copy_(self.master[k])

    def train_step(self, x, target, lr):
        d = self.forward(x).float() - target
        loss = d.square().mean()
        self.backward(x, (d * (2.0 / d.shape[0])).bfloat16())
        self.sgd(lr)
        return loss


def check(ws):
    st, bits = moe.moe_get_device_status(ws)
    if st != moe.MOE_OK:
        raise RuntimeError(f"{moe.moe_status_string(st)} (status bits {bits:#x})")


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--train", action="store_true")
    p.add_argument("--T", type=int)
    p.add_argument("--H", type=int)
    p.add_argument("--I", type=int)
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--e4m3", action="store_true")
    a = p.parse_args(argv)
    if a.train:
        T, H, I = a.T or 2048, a.H or 1024, a.I or 2816
        block = TrainBlock(T, H, I)
        g = torch.Generator(device="cuda").manual_seed(1)
        x = randn(g, T, H)
        target = x.float() + randn(g, T, H, std=0.5).float()
        losses = [float(block.train_step(x, target, 0.02)) for _ in range(a.steps)]
        check(block.ws)
        print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
        return losses
    blocks = DecodeBlocks(a.T or 4, a.H or 4096, a.I or 14336, a.layers, a.e4m3)
    blocks.step()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        y = blocks.step()
    end.record()
    check(blocks.ws)
    us = start.elapsed_time(end) / a.steps * 1e3
    print(f"{us:.1f} us a step of {a.layers} blocks, "
          f"{blocks.bytes_read() / us / 1e6:.2f} TB/s of weights")
    return y


if __name__ == "__main__":
    main()
