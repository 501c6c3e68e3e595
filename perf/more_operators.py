"""The cases by which the experts' matrix products are measured: products of ragged
groups of rows with each group's own matrix and their gradients, and products with
weights held in 4 bits with group scales, of one matrix and of one for each expert.

Every case is a dict of plain values.  ``prepare`` makes its inputs from a seed, ``run``
is one pass as a user's program makes it -- in plain torch operations in 32 bits, or
through the package's entry points where ``own`` is true -- and ``exact`` is the same
from the definitions in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's eight experts of the 32 that a GPU holds, by the down projection:
        # the weights' bytes and latency
        dict(name="grouped_decode", op="grouped", R=8, used=8, E=32, active=8, N=4096, K=1536,
             dtype="bf16", out="same", pad=0),
        # a prefill batch of 1024 tokens with 8 experts each, gate and up projection
        dict(name="grouped_prefill", op="grouped", R=8192, used=8192, E=32, active=32, N=4096,
             K=7168, dtype="bf16", out="same", pad=0),
        # a half-precision layer on sizes that no tile divides, most experts without rows or
        # with few, rows left over behind the last expert's, x a slice of a wider tensor
        dict(name="grouped_odd_fp16", op="grouped", R=1021, used=977, E=13, active=9, N=1864,
             K=2056, dtype="fp16", out="fp32", pad=72),
        # gradients of the gate projections of a layer of few large experts (training)
        dict(name="grouped_train", op="grouped_backward", R=8192, used=8192, E=8, active=8,
             N=14336, K=4096, dtype="bf16", dw="same"),
        # gradients of many small experts, kept in 32 bits for the optimizer
        dict(name="grouped_train_small", op="grouped_backward", R=4099, used=4001, E=64, active=59,
             N=1536, K=2048, dtype="bf16", dw="fp32"),
        # one token through an output projection whose weights are held in 4 bits
        dict(name="int4_decode", op="int4", T=1, N=4096, K=4096, group=128, dtype="bf16",
             act="none", bias=False, residual=True),
        # eight sequences through the first projection of a plain feed-forward layer
        dict(name="int4_batch", op="int4", T=8, N=14336, K=4096, group=128, dtype="bf16",
             act="gelu_tanh", bias=True, residual=False),
        # a ragged chunk of a prompt, fine groups, sizes that no tile divides
        dict(name="int4_chunk_fp16", op="int4", T=203, N=7176, K=2080, group=32, dtype="fp16",
             act="silu", bias=True, residual=True),
        # four tokens' eight experts of 128, weights in 4 bits
        dict(name="grouped_int4_decode", op="grouped_int4", R=32, used=32, E=128, active=29,
             N=4096, K=1536, group=128, dtype="bf16", out="same"),
        # 64 tokens with 8 experts each: few rows for each of the experts
        dict(name="grouped_int4_batch", op="grouped_int4", R=512, used=512, E=32, active=32,
             N=4096, K=7168, group=64, dtype="bf16", out="same"),
        # a checkpoint's expert matrices to 4 bits, with the values that the codes stand for
        # (training with the rounding in the forward)
        dict(name="quantize_experts", op="quantize", rows=32768, K=4096, group=128, dtype="bf16"),
        # one odd matrix
        dict(name="quantize_odd_fp16", op="quantize", rows=1000, K=2080, group=32, dtype="fp16"),
    ]


def _size(rng, lo, hi, step=1):
    """A size spread over its logarithm; a multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(-(-lo // step) * step, min(hi, v) // step * step)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_backward", "grouped_backward", "int4", "int4",
                     "grouped_int4", "grouped_int4", "quantize"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    group = rng.choice([32, 64, 128])
    if op == "quantize":
        c = dict(op=op, rows=_size(rng, 64, 131072), K=_size(rng, 256, 14336, 32), group=group,
                 dtype=dtype)
        while c["rows"] * c["K"] > 32768 * 4096:
            c["rows"] //= 2
        return c
    if op == "int4":
        return dict(op=op, T=_size(rng, 1, 256), N=_size(rng, 256, 14336, 8),
                    K=_size(rng, 256, 8192, 32), group=group, dtype=dtype,
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    E = _size(rng, 4, 128)
    N, K = _size(rng, 256, 7168, 8), _size(rng, 256, 7168, 32 if op == "grouped_int4" else 8)
    while E * N * K > 32 * 4096 * 7168 // (4 if op == "grouped_backward" else 1):
        E -= 1
    used = _size(rng, 1, 1024 if op == "grouped_int4" else 8192)
    active = rng.choice([min(E, used), rng.randint(1, min(E, used))])
    c = dict(op=op, R=used + rng.choice([0, 0, rng.randint(1, 100)]), used=used, E=E,
             active=active, N=N, K=K, dtype=dtype)
    if op == "grouped_backward":
        c["dw"] = rng.choice(["same", "fp32"])
    else:
        c["out"] = rng.choice(["same", "same", "fp32"])
    if op == "grouped":
        c["pad"] = rng.choice([0, 0, 8 * rng.randint(1, 32)])
    if op == "grouped_int4":
        c["group"] = group
    return c


# ----------------------------------------------------------------- inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1 + int(seed) * 7919)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    t = torch.empty(*shape, device="cuda", dtype=dtype)
    return t.normal_(0.0, std, generator=g)


def _hidden(g, T, H, dtype):
    """Hidden states: unit rows of each token's own size, one channel in 128 some times as large."""
    t = torch.randn(T, H, generator=g, device="cuda")
    t *= 0.5 + torch.rand(T, 1, generator=g, device="cuda")
    t[:, torch.randperm(H, generator=g, device="cuda")[: max(1, H // 128)]] *= 6.0
    return t.to(dtype)


def _segments(seed, c):
    """Rows of each expert as a router leaves them: some experts more popular than others, those
    that are not active without any."""
    r = torch.Generator()
    r.manual_seed(3 + int(seed))
    E, active = c["E"], c["active"]
    ids = torch.randperm(E, generator=r)[:active]
    p = torch.softmax(0.5 * torch.randn(active, generator=r), 0)
    more = torch.multinomial(p, max(1, c["used"] - active), replacement=True, generator=r)
    counts = torch.zeros(E, dtype=torch.int64)
    counts[ids] = 1 + torch.bincount(more, minlength=active)
    if c["used"] == active:
        counts.clamp_(max=1)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets.cuda(), int(counts.max())


def _groups(n, group):
    return -(-n // group)


def _packed(w, group):
    """(4-bit codes, two to a byte, the even column's in the low half; scales) of w [rows, K]:
    scale = largest magnitude of `group` columns / 7, code = value / scale rounded, plus 8."""
    rows, K = w.shape
    G = _groups(K, group)
    p = torch.nn.functional.pad(w.float(), (0, G * group - K)).view(rows, G, group)
    s = (p.abs().amax(2) / 7.0).to(w.dtype)
    c = torch.round(p / s.float()[:, :, None]).nan_to_num_().clamp_(-8, 7).add_(8)
    c = c.view(rows, G * group)[:, :K].to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def prepare(case, seed):
    g = _generator(seed)
    op, dt = case["op"], _TYPES[case["dtype"]]
    s = dict(case=dict(case), kept={})
    K = case["K"]
    if op == "quantize":
        s["w"] = _randn(g, case["rows"], K, std=K ** -0.5, dtype=dt)
        return s
    N = case["N"]
    if op == "int4":
        T = case["T"]
        s["x"] = _hidden(g, T, K, dt)
        s["q"], s["scale"] = _packed(_randn(g, N, K, std=K ** -0.5, dtype=dt), case["group"])
        s["bias"] = _randn(g, N, std=0.5, dtype=dt) if case["bias"] else None
        s["residual"] = _randn(g, T, N, std=2.0, dtype=dt) if case["residual"] else None
        return s
    R, E, pad = case["R"], case["E"], case.get("pad", 0)
    s["offsets"], s["most"] = _segments(seed, case)
    s["x"] = _hidden(g, R, K + pad, dt)[:, :K]
    if op == "grouped_int4":
        s["q"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty(E, N, _groups(K, case["group"]), dtype=dt, device="cuda")
        for e in range(E):
            s["q"][e], s["scale"][e] = _packed(_randn(g, N, K, std=K ** -0.5, dtype=dt),
                                               case["group"])
    else:
        s["w"] = _randn(g, E, N, K, std=K ** -0.5, dtype=dt)
    if op == "grouped_backward":
        s["dy"] = _randn(g, R, N, std=0.1, dtype=dt)
        s["dx"] = torch.zeros(R, K, dtype=dt, device="cuda")
        s["dw"] = torch.empty(E, N, K, dtype=dt if case["dw"] == "same" else torch.float32,
                              device="cuda")
    else:
        # a buffer that the program made once; rows that belong to no expert stay as they are
        s["y"] = torch.zeros(R, N, dtype=dt if case["out"] == "same" else torch.float32,
                             device="cuda")
    return s


# ------------------------------------------------------------- plain forms --
# The experts that have rows, each padded to the most rows of any: one batched product.

def _plain_places(s):
    """(experts with rows, each row's place among them and in its expert's rows)."""
    c, o = s["case"], s["offsets"].long()
    ids = (o[1:] - o[:-1]).topk(c["active"]).indices
    row = torch.arange(c["used"], device="cuda")
    e = torch.searchsorted(o[1:].contiguous(), row, right=True)
    at = torch.zeros(c["E"], dtype=torch.int64, device="cuda")
    at[ids] = torch.arange(c["active"], device="cuda")
    return ids, at[e], row - o[e]


def _plain_padded(s, t, a, i):
    p = torch.zeros(s["case"]["active"], s["most"], t.shape[1], device="cuda")
    p[a, i] = t[: s["case"]["used"]].float()
    return p


def _plain_values(q, scale, group):
    """The values [..., K] of 4-bit codes in 32 bits."""
    c = torch.stack([q & 15, q >> 4], -1).flatten(-2).float() - 8.0
    return c * scale.float().repeat_interleave(group, -1)[..., : c.shape[-1]]


def _plain_grouped(s):
    c = s["case"]
    ids, a, i = _plain_places(s)
    if c["op"] == "grouped_int4":
        w = _plain_values(s["q"][ids], s["scale"][ids], c["group"])
    else:
        w = s["w"][ids].float()
    y = torch.bmm(_plain_padded(s, s["x"], a, i), w.transpose(1, 2))
    s["y"][: c["used"]] = y[a, i].to(s["y"].dtype)
    return {"y": s["y"]}


def _plain_grouped_backward(s):
    c = s["case"]
    ids, a, i = _plain_places(s)
    dy = _plain_padded(s, s["dy"], a, i)
    dx = torch.bmm(dy, s["w"][ids].float())
    s["dx"][: c["used"]] = dx[a, i].to(s["dx"].dtype)
    dw = torch.bmm(dy.transpose(1, 2), _plain_padded(s, s["x"], a, i))
    s["dw"].zero_()
    s["dw"][ids] = dw.to(s["dw"].dtype)
    return {"dx": s["dx"], "dw": s["dw"]}


def _plain_act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_int4(s):
    c = s["case"]
    z = s["x"].float() @ _plain_values(s["q"], s["scale"], c["group"]).t()
    if c["bias"]:
        z = z + s["bias"].float()
    z = _plain_act(z, c["act"])
    if c["residual"]:
        z = z + s["residual"].float()
    return {"y": z.to(s["x"].dtype)}


def _plain_quantize(s):
    c, w = s["case"], s["w"]
    G = _groups(c["K"], c["group"])
    p = torch.nn.functional.pad(w.float(), (0, G * c["group"] - c["K"]))
    p = p.view(c["rows"], G, c["group"])
    scale = (p.abs().amax(2) / 7.0).to(w.dtype)
    t = scale.float()[:, :, None]
    v = torch.where(t > 0, torch.round(p / t), torch.zeros_like(p)).clamp(-8, 7) * t
    return {"values": v.view(c["rows"], -1)[:, : c["K"]].to(w.dtype), "scale": scale}


# -------------------------------------------------------- the entry points --

def _keep(s, make):
    """What a program allocates once for its calls: descriptor, workspace, outputs."""
    if not s["kept"]:
        s["kept"].update(make())
    return s["kept"]


def _own_grouped(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]

    def make():
        d = moe.grouped_desc(c["R"], c["E"], c["N"], c["K"], moe.dtype_of(s["x"]),
                             out_dtype=moe.dtype_of(s["y"]), x_stride=c["K"] + c.get("pad", 0))
        return dict(d=d, ws=moe.alloc_workspace(d))

    k = _keep(s, make)
    if c["op"] == "grouped_int4":
        moe.moe_grouped_linear_int4(k["d"], c["group"], s["x"], s["offsets"], s["q"], s["scale"],
                                    s["y"], k["ws"])
    else:
        moe.moe_grouped_linear(k["d"], s["x"], s["offsets"], s["w"], s["y"], k["ws"])
    return {"y": s["y"]}


def _own_grouped_backward(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]

    def make():
        d = moe.grouped_desc(c["R"], c["E"], c["N"], c["K"], moe.dtype_of(s["x"]))
        return dict(d=d, ws=moe.alloc_workspace(d))

    k = _keep(s, make)
    moe.moe_grouped_linear_backward(k["d"], s["dy"], s["x"], s["offsets"], s["w"], s["dx"], s["dw"],
                                    k["ws"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _own_int4(s):
    import routed_expert_ffn_gb300 as moe
    c = s["case"]

    def make():
        d = moe.linear_desc(c["T"], c["N"], c["K"], moe.dtype_of(s["x"]), act=c["act"])
        return dict(d=d, ws=moe.alloc_workspace(d),
                    y=torch.empty(c["T"], c["N"], dtype=s["x"].dtype, device="cuda"))

    k = _keep(s, make)
    moe.moe_linear_int4(k["d"], c["group"], s["x"], s["q"], s["scale"], s["bias"], s["residual"],
                        k["y"], k["ws"])
    return {"y": k["y"]}


def _own_quantize(s):
    import routed_expert_ffn_gb300 as moe
    c, w = s["case"], s["w"]

    def make():
        return dict(q=torch.empty(c["rows"], c["K"] // 2, dtype=torch.uint8, device="cuda"),
                    scale=torch.empty(c["rows"], _groups(c["K"], c["group"]), dtype=w.dtype,
                                      device="cuda"), values=torch.empty_like(w))

    k = _keep(s, make)
    moe.moe_quantize_int4(w, c["rows"], c["K"], c["group"], k["q"], k["scale"], k["values"])
    return {"values": k["values"], "scale": k["scale"]}


_PLAIN = {"grouped": _plain_grouped, "grouped_backward": _plain_grouped_backward,
          "grouped_int4": _plain_grouped, "int4": _plain_int4, "quantize": _plain_quantize}
_OWN = {"grouped": _own_grouped, "grouped_backward": _own_grouped_backward,
        "grouped_int4": _own_grouped, "int4": _own_int4, "quantize": _own_quantize}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    op, K = case["op"], case["K"]
    if op == "quantize":
        n = case["rows"] * K
        scales = case["rows"] * _groups(K, case["group"])
        return {"bytes": 2 * n + n // 2 + 2 * n + 2 * scales, "flops": 4 * n}
    N = case["N"]
    if op == "int4":
        T = case["T"]
        n = N * K // 2 + 2 * N * _groups(K, case["group"]) + 2 * T * (K + N)
        n += 2 * N if case["bias"] else 0
        n += 2 * T * N if case["residual"] else 0
        return {"bytes": n, "flops": 2 * T * N * K}
    used, E, active = case["used"], case["E"], case["active"]
    if op == "grouped_backward":
        dw = 2 if case["dw"] == "same" else 4
        return {"bytes": 2 * active * N * K + dw * E * N * K + 2 * used * (N + 2 * K),
                "flops": 4 * used * N * K}
    out = 2 if case["out"] == "same" else 4
    w = 2 * N * K if op == "grouped" else N * K // 2 + 2 * N * _groups(K, case["group"])
    return {"bytes": active * w + used * (2 * K + out * N), "flops": 2 * used * N * K}


# -------------------------------------------------- the definitions, 64 bits --

def _exact_int4(q, scale, group):
    k = torch.arange(2 * q.shape[1], device=q.device)
    code = (q.long()[:, k // 2] >> (4 * (k % 2))) & 15
    return (code - 8).double() * scale.double()[:, k // group]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        w, K, scale = s["w"].double(), case["K"], []
        values = torch.zeros_like(w)
        for j in range(0, K, case["group"]):
            block = w[:, j:j + case["group"]]
            t = (block.abs().max(1, keepdim=True).values / 7).to(s["w"].dtype).double()
            c = (block / torch.where(t == 0, torch.ones_like(t), t)).round().clamp(-8, 7)
            values[:, j:j + case["group"]] = torch.where(t == 0, torch.zeros_like(c), c) * t
            scale.append(t)
        return {"values": values, "scale": torch.cat(scale, 1)}
    if op == "int4":
        f = torch.nn.functional
        y = f.linear(s["x"].double(), _exact_int4(s["q"], s["scale"], case["group"]),
                     s["bias"].double() if case["bias"] else None)
        y = {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "silu": f.silu,
             "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[case["act"]](y)
        return {"y": y + s["residual"].double() if case["residual"] else y}
    ends = s["offsets"].tolist()
    x = s["x"].double()
    if op == "grouped_backward":
        dy = s["dy"].double()
        dx, dw = torch.zeros_like(x), torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    else:
        y = torch.zeros(case["R"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        rows = slice(ends[e], ends[e + 1])
        if op == "grouped_backward":
            dx[rows] = torch.einsum("tn,nk->tk", dy[rows], s["w"][e].double())
            dw[e] = torch.einsum("tn,tk->nk", dy[rows], x[rows])
        elif op == "grouped":
            y[rows] = torch.nn.functional.linear(x[rows], s["w"][e].double())
        elif ends[e + 1] > ends[e]:
            w = _exact_int4(s["q"][e], s["scale"][e], case["group"])
            y[rows] = torch.nn.functional.linear(x[rows], w)
    return {"dx": dx, "dw": dw} if op == "grouped_backward" else {"y": y}
