"""Products with 4-bit weights (moe_linear_int4, moe_grouped_linear_int4) and the quantiser
against 64-bit formulas (needs a GB300)."""

import pytest
import torch

import int4_ref
import routed_expert_ffn_gb300 as moe
from dense_ref import activation, assert_within, half_step, product_bound, tiny

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_ffn_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def randn(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float32) * std).to(dtype).cuda()


def weights(seed, *shape, group, dtype):
    """Any codes, 0 among them, and scales of their own size for each group."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, shape, generator=g)
    scale = torch.rand(*shape[:-1], -(-shape[-1] // group), generator=g) + 0.25
    return int4_ref.pack(codes).cuda(), (scale * 0.25 * shape[-1] ** -0.5).to(dtype).cuda()


def status_ok(ws):
    st, raw = moe.moe_get_device_status(ws)
    assert st == moe.MOE_OK, (st, raw)


def forward_bound(x, w, bias, residual, act, dtype):
    """(result, bound) in 64 bits: fp32 sums (product_bound counts a step for each addition; the
    scales' multiplications, one for a group, add at most as many), rounded once."""
    e = 2 * product_bound(x, w, x.shape[1])
    z = x @ w.t()
    if bias is not None:
        z = z + bias
        e = e + z.abs() * 2.0 ** -23
    y = activation(z, act)
    e = 1.13 * e + (0 if act == "none" else 1) * z.abs() * 2.0 ** -16
    if residual is not None:
        y = y + residual
        e = e + y.abs() * 2.0 ** -24
    return y, e + (y.abs() + e) * half_step(dtype) + tiny(dtype)


SHAPES = [(0, 64, 64), (1, 8, 32), (1, 1000, 4096), (2, 136, 2080), (7, 264, 96), (8, 4096, 256),
          (9, 40, 1504), (16, 512, 7168), (17, 1000, 544), (33, 264, 160), (64, 776, 1024),
          (130, 520, 288), (257, 136, 2048)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_linear(T, N, K, group, dtype):
    x = randn(1, T, K, dtype=dtype)
    q, s = weights(2, N, K, group=group, dtype=dtype)
    b, r = randn(3, N, dtype=dtype), randn(4, T, N, dtype=dtype)
    d = moe.linear_desc(T, N, K, moe.dtype_of(x))
    ws = moe.alloc_workspace(d)
    y = torch.full((T, N), 3.0, dtype=dtype, device="cuda")
    moe.moe_linear_int4(d, group, x, q, s, b, r, y, ws)
    status_ok(ws)
    w = int4_ref.values(q, s, group)
    want, bound = forward_bound(x.double(), w, b.double(), r.double(), "none", dtype)
    assert_within(y, want, bound, "y")
    d = moe.linear_desc(T, N, K, moe.dtype_of(x), out_dtype=moe.MOE_DTYPE_FP32)
    y32 = torch.full((T, N), 3.0, device="cuda")
    moe.moe_linear_int4(d, group, x, q, s, None, None, y32, ws)
    want, bound = forward_bound(x.double(), w, None, None, "none", FP32)
    assert_within(y32, want, bound, "y in fp32")


@pytest.mark.parametrize("act", moe.ACT_NAMES)
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_activations(T, act, out):
    N, K, group = 264, 544, 64
    x = randn(11, T, K, std=2.0)
    q, s = weights(12, N, K, group=group, dtype=BF16)
    b, r = randn(13, N, dtype=out), randn(14, T, N, dtype=out)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, act=act, out_dtype=moe.dtype_of(b))
    ws = moe.alloc_workspace(d)
    y = torch.empty(T, N, dtype=out, device="cuda")
    moe.moe_linear_int4(d, group, x, q, s, b, r, y, ws)
    status_ok(ws)
    want, bound = forward_bound(x.double(), int4_ref.values(q, s, group), b.double(), r.double(),
                                act, out)
    assert_within(y, want, bound, "y")


@pytest.mark.parametrize("T", [5, 100])
def test_strides_in_place_and_neighbours(T):
    N, K, group = 520, 288, 128
    xw = torch.full((T + 3, K + 40), NAN, dtype=BF16, device="cuda")
    xw[:T, 8:8 + K] = randn(21, T, K)
    yw = torch.full((T + 3, N + 24), NAN, dtype=BF16, device="cuda")
    yw[:T, :N] = randn(22, T, N)
    q, s = weights(23, N, K, group=group, dtype=BF16)
    x, y = xw[:T, 8:8 + K], yw[:T, :N]
    want, bound = forward_bound(x.double(), int4_ref.values(q, s, group), None, y.double(), "silu",
                                BF16)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, "silu", x_stride=K + 40,
                        residual_stride=N + 24, y_stride=N + 24)
    ws = moe.alloc_workspace(d)
    moe.moe_linear_int4(d, group, x, q, s, None, y, y, ws)
    status_ok(ws)
    assert_within(y, want, bound, "y in place")
    assert bool(torch.isnan(yw[T:]).all()) and bool(torch.isnan(yw[:T, N:]).all())


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_infinities_stay_where_they_belong(T, group):
    """A NaN or infinity of x reaches its row, one of a scale its column."""
    N, K = 264, 544
    x = randn(31, T, K)
    q, s = weights(32, N, K, group=group, dtype=BF16)
    x[1, 3], x[2, K - 1] = float("inf"), NAN
    s[5, -1] = float("inf")
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    moe.moe_linear_int4(d, group, x, q, s, None, None, y, ws)
    status_ok(ws)
    fine = torch.isfinite(y)
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[1:3] = False
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[5] = False
    assert bool(fine[rows][:, cols].all())
    assert not bool(fine[1:3].any()) and not bool(fine[:, 5].any())
    assert bool(torch.isnan(y[2]).all())


def row_error(x, w):
    """What rows of x as fp16, each times a power of two, add to the bound: numbers below 2^-28 of
    the row's largest are off by half a step of fp16's smallest, 2^-25 where that is 2^14 or more."""
    most = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(1, keepdim=True)
    return most * 2.0 ** -39 * w.abs().sum(1)


@pytest.mark.parametrize("T,N,K", [(8, 264, 16384), (1, 40, 65536), (2500, 136, 160)])
def test_deep_and_long(T, N, K):
    """Rows that do not fit beside the codes, and more than are multiplied at a time."""
    x = randn(91, T, K)
    q, s = weights(92, N, K, group=64, dtype=BF16)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    y = torch.empty(T, N, device="cuda")
    moe.moe_linear_int4(d, 64, x, q, s, None, None, y, ws)
    status_ok(ws)
    w = int4_ref.values(q, s, 64)
    want, bound = forward_bound(x.double(), w, None, None, "none", FP32)
    assert_within(y, want, bound + row_error(x.double(), w), "y")


@pytest.mark.parametrize("T", [3, 40])
def test_rows_of_any_size(T):
    """Rows from the smallest numbers to the largest, and rows with both."""
    N, K, group = 136, 544, 128
    x = randn(93, T, K).float()
    x[0] *= 2.0 ** -126
    x[1] *= 2.0 ** 110
    x[2, ::2] *= 2.0 ** -60
    x[2, 1::2] *= 2.0 ** 20
    x = x.to(BF16)
    if T > 3:
        x[3] = 0.0
        x[4] = 2.0 ** -133
        x[5] = torch.finfo(BF16).max
        x[5, ::2] = -torch.finfo(BF16).max
    q, s = weights(94, N, K, group=group, dtype=BF16)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    y = torch.empty(T, N, device="cuda")
    moe.moe_linear_int4(d, group, x, q, s, None, None, y, ws)
    status_ok(ws)
    w = int4_ref.values(q, s, group)
    want, bound = forward_bound(x.double(), w, None, None, "none", FP32)
    # (sums of the smallest numbers are subnormal: one step of those more for each group)
    bound = bound + row_error(x.double(), w) + 2.0 ** -148
    # the largest rows' sums reach 8 x 544 x 2^128 / 4 sqrt(544): what fp32 cannot hold (2^128 less
    # half a step, and more) rounds to infinity
    beyond = want.abs() - bound > torch.finfo(FP32).max
    assert torch.equal(y[beyond], torch.sign(want[beyond]).float() * float("inf"))
    near = (want.abs() + bound > torch.finfo(FP32).max) & ~beyond
    y[beyond | near], want[beyond | near] = 0.0, 0.0
    assert_within(y, want, bound, "y")


def test_two_streams():
    """Two calls at once, each with a workspace of its own."""
    N, K, group = 1000, 2080, 32
    q, s = weights(95, N, K, group=group, dtype=FP16)
    w = int4_ref.values(q, s, group)
    runs = []
    for i, T in enumerate((5, 70)):
        d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_FP16)
        runs.append((d, randn(96 + i, T, K, dtype=FP16), torch.empty(T, N, dtype=FP16, device="cuda"),
                     moe.alloc_workspace(d), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for d, x, y, ws, stream in runs:
            moe.moe_linear_int4(d, group, x, q, s, None, None, y, ws, stream=stream)
    torch.cuda.synchronize()
    for d, x, y, ws, _ in runs:
        status_ok(ws)
        want, bound = forward_bound(x.double(), w, None, None, "none", FP16)
        assert_within(y, want, bound, "y")


@pytest.mark.parametrize("T", [6, 33])
def test_runs_give_the_same_bits(T):
    N, K, group = 4096, 4096, 128
    x = randn(97, T, K)
    q, s = weights(98, N, K, group=group, dtype=BF16)
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    y, again = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    moe.moe_linear_int4(d, group, x, q, s, None, None, y, ws)
    for _ in range(5):
        moe.moe_linear_int4(d, group, x, q, s, None, None, again, ws)
        assert torch.equal(y, again)
    status_ok(ws)


SEGMENTS = [[700, 3, 0, 1500, 40], [1], [0, 0, 3], [7, 0, 8, 9, 1], [0] * 40 + [1] * 8 + [0, 5] * 16, [40, 17, 0, 64, 130],
            [0, 0, 0]]


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP32)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(8, 32), (264, 544), (1000, 2080)])
@pytest.mark.parametrize("counts", SEGMENTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_grouped(counts, N, K, group, dtype, out):
    E, first = len(counts), 3
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    R = o[-1] + 5
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    x = randn(41, R, K, dtype=dtype)
    x[:first] = NAN
    x[o[-1]:] = NAN
    q, s = weights(42, E, N, K, group=group, dtype=dtype)
    y = torch.full((R, N), 3.0, dtype=out, device="cuda")
    d = moe.grouped_desc(R, E, N, K, moe.dtype_of(x), out_dtype=moe.dtype_of(y))
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear_int4(d, group, x, off, q, s, y, ws)
    status_ok(ws)
    for e in range(E):
        if counts[e]:
            rows = slice(o[e], o[e + 1])
            want, bound = forward_bound(x[rows].double(), int4_ref.values(q[e], s[e], group), None,
                                        None, "none", out)
            assert_within(y[rows], want, bound, f"expert {e}")
    assert bool((y[:first] == 3.0).all()) and bool((y[o[-1]:] == 3.0).all())


def test_bad_offsets():
    R, E, N, K = 10, 2, 64, 64
    q, s = weights(51, E, N, K, group=64, dtype=BF16)
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y = torch.full((R, N), 3.0, dtype=BF16, device="cuda")
    for bad in ([-1, 4, 8], [0, 9, 8], [0, 4, 11]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        moe.moe_grouped_linear_int4(d, 64, randn(52, R, K), off, q, s, y, ws)
        assert moe.moe_get_device_status(ws)[0] == moe.MOE_ERR_DEVICE_CHECK
    assert bool((y == 3.0).all())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (1000, 2080), (64, 256), (513, 4096), (2, 40960)])
def test_quantize(rows, K, group, dtype):
    """Codes and scales are the definition's, bit for bit: ties, zeros and large values among them."""
    w = randn(61, rows, K, std=K ** -0.5, dtype=dtype)
    w[0, :32] = 0.0
    if rows > 2:
        # sevenths of the maximum in halves: ties
        w[1, :32] = torch.arange(-16, 16, device="cuda").to(dtype) * 0.5 * 2.0 ** -4
        w[1, 0] = 7 * 2.0 ** -4
        w[2, :] *= 2.0 ** 12
        w[2, 32:64] *= 2.0 ** -20
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, -(-K // group), dtype=dtype, device="cuda")
    v = torch.empty_like(w)
    moe.moe_quantize_int4(w, rows, K, group, q, s, v)
    codes, scale = int4_ref.quantize(w, group)
    assert torch.equal(s, scale)
    assert torch.equal(q, int4_ref.pack(codes))
    assert torch.equal(v.double(), int4_ref.values(q, s, group).to(dtype).double())
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    moe.moe_quantize_int4(w, rows, K, group, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_quantize_what_is_no_number():
    w = randn(71, 8, 64)
    w[1, 3], w[2, 40], w[3, 5], w[4, :] = NAN, float("inf"), float("-inf"), 1e-40
    q = torch.empty(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.empty(8, 2, dtype=BF16, device="cuda")
    moe.moe_quantize_int4(w, 8, 64, 32, q, s)
    codes, scale = int4_ref.quantize(w, 32)
    assert torch.equal(torch.isnan(s), torch.isnan(scale)) and bool(torch.isnan(s[1, 0]))
    assert torch.equal(s.nan_to_num(), scale.nan_to_num())
    assert torch.equal(q, int4_ref.pack(codes))


def test_quantized_and_multiplied_in_a_graph():
    """The operators together, captured: an expert layer's down projection in 4 bits against the
    same with the values that the codes stand for."""
    E, N, K, group = 6, 264, 544, 32
    o = [0, 3, 3, 20, 21, 30, 64]
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    x, w = randn(81, o[-1], K, dtype=FP16), randn(82, E, N, K, std=K ** -0.5, dtype=FP16)
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // group, dtype=FP16, device="cuda")
    v = torch.empty_like(w)
    d = moe.grouped_desc(o[-1], E, N, K, moe.MOE_DTYPE_FP16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    y, z = torch.zeros(o[-1], N, device="cuda"), torch.zeros(o[-1], N, device="cuda")

    def step():
        moe.moe_quantize_int4(w, E * N, K, group, q, s, v)
        moe.moe_grouped_linear_int4(d, group, x, off, q, s, y, ws)
        moe.moe_grouped_linear(d, x, off, v, z, ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    w.copy_(randn(83, E, N, K, std=K ** -0.5, dtype=FP16))
    graph.replay()
    torch.cuda.synchronize()
    status_ok(ws)
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        a, b = x[rows].double(), int4_ref.values(q[e], s[e], group)
        want, bound = forward_bound(a, b, None, None, "none", FP32)
        assert_within(y[rows], want, bound, f"expert {e}")
        # values of fp16 are off by half a step each
        assert_within(z[rows], want, bound + (a.abs() @ b.abs().t()) * half_step(FP16) +
                      a.abs().sum(1, keepdim=True) * tiny(FP16), f"expert {e}, values")
