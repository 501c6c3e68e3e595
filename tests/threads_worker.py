"""First calls of the dense operators from several host threads at once, each on a stream and a
workspace of its own; then every call again, alone.  Prints what failed, and "ok"."""

import os
import sys
import threading

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_expert_ffn_gb300 as moe  # noqa: E402

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def randn(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def linear(T):
    x, w = randn(T, T, 1024), randn(1, 512, 1024, std=1 / 32)
    d = moe.linear_desc(T, 512, 1024, moe.MOE_DTYPE_BF16, "silu")
    ws, y = moe.alloc_workspace(d), torch.empty(T, 512, dtype=BF16, device="cuda")

    def call(stream):
        moe.moe_linear(d, x, w, None, None, y, ws, stream=stream)
        return y
    return call


def linear_e4m3(T):
    x = randn(T, T, 1024).to(torch.float8_e4m3fn)
    w = randn(1, 512, 1024, std=1 / 32).to(torch.float8_e4m3fn)
    xe = torch.zeros(T, 8, dtype=torch.int8, device="cuda")
    we = torch.zeros(4, 8, dtype=torch.int8, device="cuda")
    d = moe.linear_desc(T, 512, 1024, moe.MOE_DTYPE_E4M3)
    ws, y = moe.alloc_workspace(d), torch.empty(T, 512, dtype=BF16, device="cuda")

    def call(stream):
        moe.moe_linear(d, x, w, None, None, y, ws, x_scale=xe, w_scale=we, stream=stream)
        return y
    return call


def ffn(T):
    x, w13, w2 = randn(T, T, 512), randn(1, 2048, 512, std=1 / 23), randn(2, 512, 1024, std=1 / 32)
    d = moe.ffn_desc(T, 512, 1024, moe.MOE_DTYPE_BF16)
    ws, y = moe.alloc_workspace(d), torch.empty_like(x)

    def call(stream):
        moe.moe_gated_ffn(d, x, w13, w2, None, None, y, ws, stream=stream)
        return y
    return call


def linear_dx(T):
    dy, w = randn(T, T, 6336, std=0.5), randn(1, 6336, 400, std=1 / 20)
    d = moe.linear_desc(T, 6336, 400, moe.MOE_DTYPE_BF16)
    ws, dx = moe.alloc_workspace(d), torch.empty(T, 400, dtype=BF16, device="cuda")

    def call(stream):
        moe.moe_linear_backward(d, dy, dx.new_empty(T, 400), w, None, dx, None, None, ws,
                                stream=stream)
        return dx
    return call


def norm_back(dtype, H):
    T = 300
    s, w, dy = randn(1, T, H, dtype=dtype), randn(2, H, dtype=dtype), randn(3, T, H, dtype=dtype)
    d = moe.norm_desc(T, H, moe.dtype_of(s))
    ws, dx = moe.alloc_workspace(d), torch.empty_like(s)

    def call(stream):
        moe.moe_add_rms_norm_backward(d, dy, None, s, w, dx, None, ws, stream=stream)
        return dx
    return call


def groups():
    rows = (60, 1, 40, 20, 64, 9, 33, 17)  # 16, 32, 48 and 64 to a tile
    for make in (linear, linear_e4m3, ffn, linear_dx):
        yield make.__name__, [make(T) for T in rows]
    for dtype in (BF16, FP16, FP32):
        widths = (8192, 256, 4096, 1024, 6144, 512, 2048, 136)
        yield f"norm_back {dtype}", [norm_back(dtype, H) for H in widths]
        widths = (16384, 8200, 12288, 9000, 16000, 8704, 10240, 14336)
        yield f"norm_back {dtype} wide", [norm_back(dtype, H) for H in widths]


def main():
    bad = []
    for name, calls in groups():
        first, streams = [None] * len(calls), [torch.cuda.Stream() for _ in calls]
        torch.cuda.synchronize()
        gate = threading.Barrier(len(calls))

        def run(i):
            try:
                gate.wait()
                first[i] = calls[i](streams[i])
            except Exception as e:  # noqa: BLE001
                bad.append(f"{name} {i}: {e}")

        threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for i, call in enumerate(calls):
            before = None if first[i] is None else first[i].clone()
            try:
                again = call(None)
                torch.cuda.synchronize()
                if before is not None and not torch.equal(before, again):
                    bad.append(f"{name} {i}: another result")
            except Exception as e:  # noqa: BLE001
                bad.append(f"{name} {i} alone: {e}")
    print("\n".join(bad) or "ok")
    return 1 if bad else 0


if __name__ == "__main__":
    sys.exit(main())
