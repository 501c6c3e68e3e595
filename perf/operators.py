"""The cases by which the dense half of a transformer block is measured: the
residual addition with root-mean-square norm, the matrix product with an
epilogue, and the gated feed-forward block.

Every case is a dict of plain values.  ``prepare`` makes its inputs from a
seed, ``run`` is one pass as a user's program makes it -- in plain torch
operations in 32 bits, or through the package's entry points where ``own`` is
true -- and ``exact`` is the same from the definitions in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-6
_BLOCK = 128            # 8-bit values share a power-of-two scale by 128
_E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoding step of one sequence, between two layers: latency only
        dict(name="norm_decode", op="norm", T=1, H=4096, dtype="bf16", out="same", pad=0),
        # the norm before an FP8 layer over a prefill batch: 8-bit rows with
        # scales, and the residual stream carried on
        dict(name="norm_prefill_e4m3", op="norm", T=8192, H=7168, dtype="bf16", out="e4m3", pad=0),
        # an odd batch of a half-precision model, its rows a slice of a wider
        # tensor (a fused projection's output)
        dict(name="norm_odd_fp16", op="norm", T=1021, H=4104, dtype="fp16", out="same", pad=72),
        # its gradient in a training step
        dict(name="norm_backward", op="norm_backward", T=8192, H=4096, dtype="bf16"),
        # attention's output projection for one token, onto the residual stream
        dict(name="linear_decode", op="linear", T=1, N=4096, K=4096, dtype="bf16", act="none",
             bias=True, residual=True),
        # the first projection of a plain feed-forward layer over a prefill batch
        dict(name="linear_prefill", op="linear", T=4096, N=14336, K=4096, dtype="bf16",
             act="gelu_tanh", bias=True, residual=False),
        # a ragged batch on sizes that no tile divides
        dict(name="linear_odd_fp16", op="linear", T=333, N=4104, K=2056, dtype="fp16", act="silu",
             bias=True, residual=True),
        # an output projection on 8-bit rows and 8-bit weights (prefill)
        dict(name="linear_prefill_e4m3", op="linear", T=4096, N=4096, K=7168, dtype="e4m3",
             act="none", bias=False, residual=True),
        # gradients of a projection with its activation in a training step
        dict(name="linear_backward", op="linear_backward", T=2047, N=4096, K=4096, dtype="bf16",
             act="gelu_tanh", bias=True),
        # a dense feed-forward block while four sequences decode: the weights' bytes
        dict(name="ffn_decode", op="ffn", T=4, H=4096, I=14336, dtype="bf16"),
        # a shared expert's shape over one chunk of a prefill
        dict(name="ffn_chunk", op="ffn", T=509, H=7168, I=2048, dtype="bf16"),
        # a training step's forward and backward of the block
        dict(name="ffn_train", op="ffn_train", T=4096, H=4096, I=14336, dtype="bf16"),
    ]


def _size(rng, lo, hi, step=1):
    """A size spread over its logarithm; a multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    v = max(lo, min(hi, v // step * step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "linear", "linear", "linear_e4m3",
                     "linear_backward", "ffn", "ffn", "ffn_train"])
    if op in ("norm", "norm_backward"):
        H = _size(rng, 256, 8192, 8)
        T = _size(rng, 1, 8192)
        c = dict(op=op, T=T, H=H, dtype=rng.choice(["bf16", "fp16", "fp32"]))
        while c["T"] * c["H"] > 8192 * 7168:
            c["T"] //= 2
        if op == "norm":
            c["out"] = rng.choice(["same", "e4m3"])
            c["pad"] = rng.choice([0, 0, 8 * rng.randint(1, 32)])
        return c
    if op in ("linear", "linear_e4m3", "linear_backward"):
        step = 16 if op == "linear_e4m3" else 8
        c = dict(op=op.replace("_e4m3", ""), T=_size(rng, 1, 8192), N=_size(rng, 256, 14336, 8),
                 K=_size(rng, 256, 7168, step),
                 dtype="e4m3" if op == "linear_e4m3" else rng.choice(["bf16", "fp16"]),
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                 bias=rng.random() < 0.5)
        if op != "linear_backward":
            c["residual"] = rng.random() < 0.5
        return c
    H, I = _size(rng, 256, 7168, 8), _size(rng, 256, 14336, 8)
    T = _size(rng, 1, 4096)
    while T * H * I > 4096 * 4096 * 14336:
        T //= 2
    return dict(op=op, T=T, H=H, I=I, dtype=rng.choice(["bf16", "bf16", "fp16"]))


# ----------------------------------------------------------------- inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1 + int(seed) * 7919)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    return t.mul_(std).to(dtype)


def _hidden(g, T, H, dtype):
    """Hidden states: unit rows of each token's own size, one channel in 128 some times as large."""
    t = torch.randn(T, H, generator=g, device="cuda")
    t *= 0.5 + torch.rand(T, 1, generator=g, device="cuda")
    t[:, torch.randperm(H, generator=g, device="cuda")[: max(1, H // 128)]] *= 6.0
    return t.to(dtype)


def _quantized(t, rows):
    """(E4M3 values, int8 exponents) of t, one power-of-two scale for each `rows` x 128 block: the
    least with every |value| / 2^s <= 448."""
    R, C = t.shape
    nr, nc = -(-R // rows), -(-C // _BLOCK)
    p = torch.zeros(nr * rows, nc * _BLOCK, device=t.device)
    p[:R, :C] = t.float()
    p = p.view(nr, rows, nc, _BLOCK)
    m, e = torch.frexp(p.abs().amax(dim=(1, 3)) / _E4M3_MAX)       # amax / 448 = m 2^e, m in [0.5, 1)
    s = torch.where(m == 0.5, e - 1, e).clamp(-15, 7)
    q = torch.ldexp(p, -s[:, None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
    q = q.view(nr * rows, nc * _BLOCK)[:R, :C].to(torch.float8_e4m3fn).contiguous()
    return q, s.to(torch.int8).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    op, T = case["op"], case["T"]
    dt = _TYPES.get(case["dtype"])
    s = dict(case=dict(case), kept={})
    if op == "norm":
        H, pad = case["H"], case["pad"]
        s["x"] = _hidden(g, T, H + pad, dt)[:, :H]
        s["residual"] = _randn(g, T, H, std=2.0, dtype=dt)
        s["weight"] = _randn(g, H, std=0.1, dtype=torch.float32).add_(1.0).to(dt)
    elif op == "norm_backward":
        H = case["H"]
        s["sum"] = _hidden(g, T, H, dt)
        s["weight"] = _randn(g, H, std=0.1, dtype=torch.float32).add_(1.0).to(dt)
        s["dy"] = _randn(g, T, H, std=0.1, dtype=dt)
        s["dresidual"] = _randn(g, T, H, std=0.1, dtype=dt)
    elif op in ("linear", "linear_backward"):
        N, K = case["N"], case["K"]
        x = _hidden(g, T, K, dt or torch.float32)
        w = _randn(g, N, K, std=K ** -0.5, dtype=dt or torch.bfloat16)
        od = dt or torch.bfloat16
        if dt is None:
            s["x"], s["x_scale"] = _quantized(x, 1)
            s["w"], s["w_scale"] = _quantized(w, _BLOCK)
        else:
            s["x"], s["w"] = x, w
        s["bias"] = _randn(g, N, std=0.5, dtype=od) if case["bias"] else None
        if op == "linear":
            s["residual"] = _randn(g, T, N, std=2.0, dtype=od) if case["residual"] else None
        else:
            z = x.float() @ w.float().t()
            s["preact"] = z.add_(s["bias"].float()) if case["bias"] else z
            s["dy"] = _randn(g, T, N, std=0.1, dtype=dt)
    else:
        H, I = case["H"], case["I"]
        s["x"] = _hidden(g, T, H, dt)
        s["w13"] = _randn(g, 2 * I, H, std=H ** -0.5, dtype=dt)
        s["w2"] = _randn(g, H, I, std=I ** -0.5, dtype=dt)
        s["residual"] = _randn(g, T, H, std=2.0, dtype=dt)
        if op == "ffn_train":
            s["dy"] = _randn(g, T, H, std=0.1, dtype=dt)
    return s


# ------------------------------------------------------------- plain forms --

def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_C0 * (z + _C1 * z * z * z)))
    if act == "silu":
        return z * _sigmoid(z)
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (z + _C1 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * z * z)
    if act == "silu":
        p = _sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _widen(q, scale, rows):
    """8-bit values times their block scales."""
    e = scale.float().repeat_interleave(rows, 0).repeat_interleave(_BLOCK, 1)
    return q.float() * torch.exp2(e[: q.shape[0], : q.shape[1]])


def _plain_norm(s):
    x = s["x"].float() + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS) * s["weight"].float()
    out = {"residual": x.to(s["x"].dtype)}
    if s["case"]["out"] == "e4m3":
        q, e = _quantized_rows(y)
        out["q"], out["scale"] = q, torch.exp2(e.float())
    else:
        out["y"] = y.to(s["x"].dtype)
    return out


def _quantized_rows(y):
    T, H = y.shape
    nb = -(-H // _BLOCK)
    p = torch.nn.functional.pad(y, (0, nb * _BLOCK - H)).view(T, nb, _BLOCK)
    m, e = torch.frexp(p.abs().amax(2) / _E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e).clamp(-126, 127)
    q = torch.ldexp(p, -e[:, :, None]).view(T, nb * _BLOCK)[:, :H]
    return q.to(torch.float8_e4m3fn), e


def _plain_norm_backward(s):
    x, w = s["sum"].float(), s["weight"].float()
    dy = s["dy"].float()
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS)
    n = x * r
    wdy = w * dy
    dx = r * (wdy - n * (wdy * n).mean(1, keepdim=True)) + s["dresidual"].float()
    return {"dx": dx.to(s["sum"].dtype), "dweight": (dy * n).sum(0)}


def _plain_linear(s):
    c = s["case"]
    if c["dtype"] == "e4m3":
        x, w = _widen(s["x"], s["x_scale"], 1), _widen(s["w"], s["w_scale"], _BLOCK)
        od = torch.bfloat16
    else:
        x, w, od = s["x"].float(), s["w"].float(), s["x"].dtype
    z = x @ w.t()
    if c["bias"]:
        z = z + s["bias"].float()
    z = _act(z, c["act"])
    if c["residual"]:
        z = z + s["residual"].float()
    return {"y": z.to(od)}


def _plain_linear_backward(s):
    c = s["case"]
    dz = s["dy"].float() * _act_slope(s["preact"], c["act"])
    dt = s["x"].dtype
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    return out


def _plain_ffn(s):
    dt, I = s["x"].dtype, s["case"]["I"]
    x, w13, w2 = s["x"].float(), s["w13"].float(), s["w2"].float()
    g, u = x @ w13[:I].t(), x @ w13[I:].t()
    p = _sigmoid(g)
    h = g * p * u
    out = {"y": (h @ w2.t() + s["residual"].float()).to(dt)}
    if s["case"]["op"] == "ffn_train":
        dy = s["dy"].float()
        dh = dy @ w2
        dg, du = dh * u * p * (1.0 + g * (1.0 - p)), dh * g * p
        out["dx"] = (dg @ w13[:I] + du @ w13[I:]).to(dt)
        out["dw13"] = torch.cat([dg.t() @ x, du.t() @ x]).to(dt)
        out["dw2"] = (dy.t() @ h).to(dt)
    return out


# -------------------------------------------------------- the entry points --

def _keep(s, make):
    """What a program allocates once for its calls: descriptor, workspace, outputs."""
    if not s["kept"]:
        s["kept"].update(make())
    return s["kept"]


def _own_norm(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]
    T, H, x = c["T"], c["H"], s["x"]

    def make():
        k = dict(d=moe.norm_desc(T, H, moe.dtype_of(x), eps=_EPS, x_stride=H + c["pad"]),
                 res=torch.empty(T, H, dtype=x.dtype, device="cuda"), y=None, q=None, e=None)
        if c["out"] == "e4m3":
            k["q"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
            k["e"] = torch.empty(T, -(-H // _BLOCK), dtype=torch.int8, device="cuda")
        else:
            k["y"] = torch.empty(T, H, dtype=x.dtype, device="cuda")
        return k

    k = _keep(s, make)
    moe.moe_add_rms_norm(k["d"], x, s["residual"], s["weight"], k["res"], k["y"], k["q"], k["e"])
    if c["out"] == "e4m3":
        return {"residual": k["res"], "q": k["q"], "scale": torch.exp2(k["e"].float())}
    return {"residual": k["res"], "y": k["y"]}


def _own_norm_backward(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]

    def make():
        d = moe.norm_desc(c["T"], c["H"], moe.dtype_of(s["sum"]), eps=_EPS)
        return dict(d=d, ws=moe.alloc_workspace(d), dx=torch.empty_like(s["sum"]),
                    dw=torch.empty(c["H"], device="cuda"))

    k = _keep(s, make)
    moe.moe_add_rms_norm_backward(k["d"], s["dy"], s["dresidual"], s["sum"], s["weight"], k["dx"],
                                  k["dw"], k["ws"])
    return {"dx": k["dx"], "dweight": k["dw"]}


def _own_linear(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]

    def make():
        d = moe.linear_desc(c["T"], c["N"], c["K"], moe.dtype_of(s["x"]), act=c["act"])
        od = torch.bfloat16 if c["dtype"] == "e4m3" else s["x"].dtype
        return dict(d=d, ws=moe.alloc_workspace(d),
                    y=torch.empty(c["T"], c["N"], dtype=od, device="cuda"))

    k = _keep(s, make)
    moe.moe_linear(k["d"], s["x"], s["w"], s["bias"], s["residual"], k["y"], k["ws"],
                   x_scale=s.get("x_scale"), w_scale=s.get("w_scale"))
    return {"y": k["y"]}


def _own_linear_backward(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]

    def make():
        d = moe.linear_desc(c["T"], c["N"], c["K"], moe.dtype_of(s["x"]), act=c["act"])
        return dict(d=d, ws=moe.alloc_workspace(d), dx=torch.empty_like(s["x"]),
                    dw=torch.empty_like(s["w"]),
                    db=torch.empty(c["N"], device="cuda") if c["bias"] else None)

    k = _keep(s, make)
    moe.moe_linear_backward(k["d"], s["dy"], s["x"], s["w"], s["preact"], k["dx"], k["dw"],
                            k["db"], k["ws"])
    out = {"dx": k["dx"], "dw": k["dw"]}
    if c["bias"]:
        out["dbias"] = k["db"]
    return out


def _own_ffn(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]
    T, H, I = c["T"], c["H"], c["I"]
    train = c["op"] == "ffn_train"

    def make():
        d = moe.ffn_desc(T, H, I, moe.dtype_of(s["x"]))
        k = dict(d=d, ws=moe.alloc_workspace(d), y=torch.empty_like(s["x"]), saved=None)
        if train:
            k.update(saved=torch.empty(T, 2 * I, device="cuda"), dx=torch.empty_like(s["x"]),
                     dw13=torch.empty_like(s["w13"]), dw2=torch.empty_like(s["w2"]))
        return k

    k = _keep(s, make)
    moe.moe_gated_ffn(k["d"], s["x"], s["w13"], s["w2"], s["residual"], k["saved"], k["y"], k["ws"])
    if not train:
        return {"y": k["y"]}
    moe.moe_gated_ffn_backward(k["d"], s["dy"], s["x"], s["w13"], s["w2"], k["saved"], k["dx"],
                               k["dw13"], k["dw2"], k["ws"])
    return {"y": k["y"], "dx": k["dx"], "dw13": k["dw13"], "dw2": k["dw2"]}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "linear": _plain_linear,
          "linear_backward": _plain_linear_backward, "ffn": _plain_ffn, "ffn_train": _plain_ffn}
_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "linear": _own_linear,
        "linear_backward": _own_linear_backward, "ffn": _own_ffn, "ffn_train": _own_ffn}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    op, T = case["op"], case["T"]
    b = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}[case["dtype"]]
    if op == "norm":
        H = case["H"]
        y = T * H + T * -(-H // _BLOCK) if case["out"] == "e4m3" else T * H * b
        return {"bytes": 3 * T * H * b + y + H * b, "flops": 5 * T * H}
    if op == "norm_backward":
        H = case["H"]
        return {"bytes": 4 * T * H * b + H * (b + 4), "flops": 11 * T * H}
    if op in ("linear", "linear_backward"):
        N, K = case["N"], case["K"]
        ob = 2
        if op == "linear":
            n = (T * K + N * K) * b + T * N * ob * (2 if case["residual"] else 1)
            n += N * ob if case["bias"] else 0
            if case["dtype"] == "e4m3":
                n += (T + -(-N // _BLOCK)) * -(-K // _BLOCK)
            return {"bytes": n, "flops": 2 * T * N * K}
        z = 0 if case["act"] == "none" else T * N * 4
        n = 2 * (T * K + N * K) * b + T * N * b + z + (N * 4 if case["bias"] else 0)
        return {"bytes": n, "flops": 4 * T * N * K}
    H, I = case["H"], case["I"]
    n = 3 * H * I * b + 3 * T * H * b
    if op == "ffn":
        return {"bytes": n, "flops": 6 * T * H * I}
    return {"bytes": 2 * 3 * H * I * b + 5 * T * H * b, "flops": 18 * T * H * I}


# -------------------------------------------------- the definitions, 64 bits --

def _exact_act(z, act):
    f = torch.nn.functional
    return {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "silu": f.silu,
            "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[act](z)


def _exact_values(q, e, rows):
    q = q.to(torch.float32).double()
    i = torch.arange(q.shape[0], device=q.device) // rows
    j = torch.arange(q.shape[1], device=q.device) // _BLOCK
    return q * torch.pow(2.0, e.double())[i][:, j]


def _exact_rms(x, w):
    return x / (x.square().sum(1, keepdim=True) / x.shape[1] + _EPS).sqrt() * w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.dtype in (torch.bfloat16, torch.float16, torch.float32)}
    if op == "norm":
        r = d["x"] + d["residual"]
        y = _exact_rms(r, d["weight"])
        if case["out"] != "e4m3":
            return {"residual": r, "y": y}
        q, scale = torch.empty_like(y), []
        for j in range(0, case["H"], _BLOCK):
            block = y[:, j:j + _BLOCK]
            p = torch.pow(2.0, torch.ceil(torch.log2(block.abs().amax(1) / _E4M3_MAX)))
            q[:, j:j + _BLOCK] = block / p[:, None]
            scale.append(p)
        return {"residual": r, "q": q, "scale": torch.stack(scale, 1)}
    if op == "norm_backward":
        x, w = d["sum"].requires_grad_(), d["weight"].requires_grad_()
        dx, dw = torch.autograd.grad(_exact_rms(x, w), (x, w), d["dy"])
        return {"dx": dx + d["dresidual"], "dweight": dw}
    if op == "linear":
        if case["dtype"] == "e4m3":
            x, w = (_exact_values(s["x"], s["x_scale"], 1),
                    _exact_values(s["w"], s["w_scale"], _BLOCK))
        else:
            x, w = d["x"], d["w"]
        y = torch.nn.functional.linear(x, w, d.get("bias"))
        y = _exact_act(y, case["act"])
        return {"y": y + d["residual"] if case["residual"] else y}
    if op == "linear_backward":
        z = d["preact"].requires_grad_()
        dz, = torch.autograd.grad(_exact_act(z, case["act"]), z, d["dy"])
        out = {"dx": torch.einsum("tn,nk->tk", dz, d["w"]),
               "dw": torch.einsum("tn,tk->nk", dz, d["x"])}
        if case["bias"]:
            out["dbias"] = torch.einsum("tn->n", dz)
        return out
    leaves = [d["x"], d["w13"], d["w2"]]
    if op == "ffn_train":
        leaves = [t.requires_grad_() for t in leaves]
    x, w13, w2 = leaves
    gate, up = torch.nn.functional.linear(x, w13).chunk(2, dim=1)
    ffn = torch.nn.functional.linear(torch.nn.functional.silu(gate) * up, w2)
    if op == "ffn":
        return {"y": ffn + d["residual"]}
    dx, dw13, dw2 = torch.autograd.grad(ffn, leaves, d["dy"])
    return {"y": (ffn + d["residual"]).detach(), "dx": dx, "dw13": dw13, "dw2": dw2}
