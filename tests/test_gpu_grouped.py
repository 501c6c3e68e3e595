"""The experts' ragged products (moe_grouped_linear) and their gradients against 64-bit
formulas (needs a GB300)."""

import pytest
import torch

import routed_expert_ffn_gb300 as moe
from dense_ref import assert_within, half_step, product_bound, tiny

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


def status_ok(ws):
    st, raw = moe.moe_get_device_status(ws)
    assert st == moe.MOE_OK, (st, raw)


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


def rounded(want, e, dtype):
    """The bound of a result `want`, off by `e` before it is rounded to `dtype`."""
    return e + (want.abs() + e) * half_step(dtype) + tiny(dtype)


def check_forward(x, w, o, y, before, what=""):
    """y against W_e x_p; rows of no expert as they were."""
    E, N, K = w.shape
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        if o[e + 1] > o[e]:
            a, b = x[rows].double(), w[e].double()
            want = a @ b.t()
            assert_within(y[rows], want, rounded(want, product_bound(a, b, K), y.dtype),
                          f"{what}expert {e}")
    outside = torch.ones(y.shape[0], dtype=torch.bool, device="cuda")
    outside[o[0]:o[-1]] = False
    same = (y == before) | (torch.isnan(y) & torch.isnan(before))
    assert bool(same[outside].all()), f"{what}rows of no expert changed"


# counts of each expert's rows
SEGMENTS = [[1], [0, 0, 3], [31, 0, 33, 1, 0], [256, 257, 0, 1], [300, 17, 0, 64, 511, 2],
            [0] * 40 + [1] * 8 + [0, 5] * 16, [2305, 7], [0, 0, 0]]


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP32)])
@pytest.mark.parametrize("N,K", [(8, 8), (264, 72), (1000, 520)])
@pytest.mark.parametrize("counts", SEGMENTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_forward(counts, N, K, dtype, out):
    E, first = len(counts), 3
    off, o = offsets_of(counts, first)
    R = o[-1] + 5
    x, w = randn(1, R, K, dtype=dtype), randn(2, E, N, K, std=K ** -0.5, dtype=dtype)
    x[:first] = NAN
    x[o[-1]:] = NAN
    y = torch.full((R, N), 3.0, dtype=out, device="cuda")
    before = y.clone()
    d = moe.grouped_desc(R, E, N, K, moe.dtype_of(x), out_dtype=moe.dtype_of(y))
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    status_ok(ws)
    check_forward(x, w, o, y, before)


@pytest.mark.parametrize("counts", [[2, 0, 1, 1, 3, 0, 1, 8], [150, 90, 200, 30, 8, 61, 300, 12]])
@pytest.mark.parametrize("N,K", [(4096, 1536), (512, 7168)])
def test_split_tiles(counts, N, K):
    """Fewer tiles than clusters: their depth is split, and runs give the same bits."""
    E = len(counts)
    off, o = offsets_of(counts)
    x, w = randn(5, o[-1], K), randn(6, E, N, K, std=K ** -0.5)
    y = torch.zeros(o[-1], N, dtype=FP32, device="cuda")
    d = moe.grouped_desc(o[-1], E, N, K, moe.MOE_DTYPE_BF16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    status_ok(ws)
    check_forward(x, w, o, y, y)
    for _ in range(4):
        again = torch.zeros_like(y)
        moe.moe_grouped_linear(d, x, off, w, again, ws)
        assert torch.equal(again, y)
    status_ok(ws)


@pytest.mark.parametrize("counts", [[40, 0, 300, 1]])
def test_strides(counts):
    """Rows inside wider buffers: what lies past a row's end is neither read nor written."""
    E, N, K = len(counts), 520, 264
    off, o = offsets_of(counts)
    R = o[-1]
    wide = torch.full((R, K + 40), NAN, dtype=BF16, device="cuda")
    wide[:, 8:8 + K] = randn(11, R, K)
    x, w = wide[:, 8:8 + K], randn(12, E, N, K, std=K ** -0.5)
    yw = torch.full((R, N + 24), NAN, dtype=BF16, device="cuda")
    y = yw[:, 16:16 + N]
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16, x_stride=K + 40, y_stride=N + 24)
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    status_ok(ws)
    check_forward(x, w, o, y, y)
    assert bool(torch.isnan(yw[:, :16]).all()) and bool(torch.isnan(yw[:, 16 + N:]).all())
    dx = torch.full_like(wide, NAN)
    dw = torch.empty(E, N, K, device="cuda")
    moe.moe_grouped_linear_backward(d, y, x, off, w, dx[:, 8:8 + K], dw, ws)
    status_ok(ws)
    check_backward(y, x, w, o, dx[:, 8:8 + K], dw, None, dx[:, 8:8 + K])
    assert bool(torch.isnan(dx[:, :8]).all()) and bool(torch.isnan(dx[:, 8 + K:]).all())


def check_backward(dy, x, w, o, dx, dw, held, before):
    E, N, K = w.shape
    for e in range(E):
        rows, m = slice(o[e], o[e + 1]), o[e + 1] - o[e]
        a, b = dy[rows].double(), x[rows].double()
        if dx is not None and m:
            want = a @ w[e].double()
            bound = product_bound(a, w[e].double().t(), N)
            assert_within(dx[rows], want, rounded(want, bound, dx.dtype), f"dx of expert {e}")
        if dw is not None:
            want, bound = a.t() @ b, product_bound(a.t(), b.t(), m)
            if held is not None:
                want = want + held[e].double()
                bound = bound + want.abs() * 2.0 ** -24
            assert_within(dw[e], want, rounded(want, bound, dw.dtype), f"dw of expert {e}")
    if dx is not None:
        outside = torch.ones(dx.shape[0], dtype=torch.bool, device="cuda")
        outside[o[0]:o[-1]] = False
        assert bool((dx == before)[outside].all()), "rows of no expert changed"


@pytest.mark.parametrize("dtype,kind", [(BF16, BF16), (FP16, FP32)])
@pytest.mark.parametrize("N,K", [(8, 8), (264, 72), (520, 1000)])
@pytest.mark.parametrize("counts", SEGMENTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_backward(counts, N, K, dtype, kind):
    """Rows of no expert are NaN: they reach no gradient."""
    E, first = len(counts), 3
    off, o = offsets_of(counts, first)
    R = o[-1] + 5
    x, dy = randn(21, R, K, dtype=dtype), randn(22, R, N, std=0.1, dtype=dtype)
    w = randn(23, E, N, K, std=K ** -0.5, dtype=dtype)
    for t in (x, dy):
        t[:first] = NAN
        t[o[-1]:] = NAN
    d = moe.grouped_desc(R, E, N, K, moe.dtype_of(x))
    ws = moe.alloc_workspace(d)
    dx = torch.full((R, K), 3.0, dtype=dtype, device="cuda")
    dw = torch.full((E, N, K), NAN, dtype=kind, device="cuda")
    before = dx.clone()
    moe.moe_grouped_linear_backward(d, dy, x, off, w, dx, dw, ws)
    status_ok(ws)
    check_backward(dy, x, w, o, dx, dw, None, before)
    held = randn(24, E, N, K, dtype=kind)
    dw.copy_(held)
    moe.moe_grouped_linear_backward(d, dy, x, off, w, None, dw, ws, accumulate=True)
    status_ok(ws)
    check_backward(dy, x, w, o, None, dw, held, None)


def test_an_experts_infinities_stay_its_own():
    """NaN and infinities in the rows of one expert, right behind the last rows of another."""
    counts, N, K = [70, 3, 65, 0, 1], 264, 136
    off, o = offsets_of(counts)
    R, E = o[-1], len(counts)
    x, dy, w = randn(31, R, K), randn(32, R, N, std=0.1), randn(33, E, N, K, std=K ** -0.5)
    x[o[1]:o[2]] = NAN
    dy[o[1]:o[2]] = float("inf")
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y, dx = torch.zeros(R, N, dtype=BF16, device="cuda"), torch.zeros_like(x)
    dw = torch.empty_like(w)
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    moe.moe_grouped_linear_backward(d, dy, x, off, w, dx, dw, ws)
    status_ok(ws)
    clean = [e for e in range(E) if e != 1]
    for e in clean:
        rows = slice(o[e], o[e + 1])
        assert bool(torch.isfinite(y[rows]).all()) and bool(torch.isfinite(dx[rows]).all())
        assert bool(torch.isfinite(dw[e]).all())
    assert bool(torch.isnan(y[o[1]:o[2]]).all()) and bool(torch.isnan(dw[1]).all())


@pytest.mark.parametrize("bad", [[-1, 4, 8], [0, 9, 8], [0, 4, 11]])
def test_bad_offsets(bad):
    """A status and no output; the workspace serves the next call."""
    R, E, N, K = 10, 2, 64, 64
    x, w = randn(41, R, K), randn(42, E, N, K)
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y = torch.full((R, N), 3.0, dtype=BF16, device="cuda")
    dw = torch.full((E, N, K), 3.0, dtype=BF16, device="cuda")
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    assert moe.moe_get_device_status(ws)[0] == moe.MOE_ERR_DEVICE_CHECK
    moe.moe_grouped_linear_backward(d, y, x, off, w, None, dw, ws)
    assert moe.moe_get_device_status(ws)[0] == moe.MOE_ERR_DEVICE_CHECK
    assert bool((y == 3.0).all()) and bool((dw == 3.0).all())
    off, o = offsets_of([4, 4])
    before = y.clone()
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    status_ok(ws)
    check_forward(x, w, o, y, before)


def test_no_rows():
    E, N, K = 3, 64, 72
    d = moe.grouped_desc(0, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    none = torch.empty(0, K, dtype=BF16, device="cuda")
    dy = torch.empty(0, N, dtype=BF16, device="cuda")
    w, dw = randn(51, E, N, K), randn(52, E, N, K)
    moe.moe_grouped_linear(d, none, off, w, dy, ws)
    held = dw.clone()
    moe.moe_grouped_linear_backward(d, dy, none, off, w, none, dw, ws, accumulate=True)
    assert torch.equal(dw, held)
    moe.moe_grouped_linear_backward(d, dy, none, off, w, none, dw, ws)
    status_ok(ws)
    assert not bool(dw.any())


def test_gradients_against_differences():
    """The gradients of sum(y g) by differences of the fp32 result along random directions: the
    sum is linear in x and in w, so differences are exact but for roundings."""
    counts, N, K = [5, 0, 70], 72, 40
    off, o = offsets_of(counts)
    R, E = o[-1], len(counts)
    x, w, g = randn(61, R, K), randn(62, E, N, K, std=0.2), randn(63, R, N)
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    d32 = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    dx, dw = torch.zeros_like(x), torch.empty(E, N, K, device="cuda")
    moe.moe_grouped_linear_backward(d, g, x, off, w, dx, dw, ws)

    def loss(x, w):
        y = torch.zeros(R, N, device="cuda")
        moe.moe_grouped_linear(d32, x, off, w, y, ws)
        return float((y.double() * g.double()).sum())

    # steps that x + v and w + v hold exactly: multiples of a step of the larger values
    def step(t, seed):
        n = torch.randint(-3, 4, t.shape, generator=torch.Generator().manual_seed(seed)).cuda()
        v = n * 2.0 ** -3
        return ((t.double() + v).to(BF16).double() - t.double()), (t.double() + v).to(BF16)

    vx, x1 = step(x, 64)
    vw, w1 = step(w, 65)
    # fp32 results: 2^-19 of the sum of the terms' magnitudes covers K = 40 additions of each
    terms = g.double().abs()
    for got, grad, v, want, a, b in ((dx.double(), dx, vx, loss(x1, w) - loss(x, w), x1, w),
                                     (dw.double(), dw, vw, loss(x, w1) - loss(x, w), x, w1)):
        size = sum(float((terms[o[e]:o[e + 1]] *
                          (a[o[e]:o[e + 1]].double().abs() @ b[e].double().abs().t())).sum())
                   for e in range(E))
        allowed = float((got.abs() * v.abs()).sum()) * half_step(grad.dtype) + 2 * size * 2.0 ** -19
        assert abs(float((got * v).sum()) - want) <= allowed


def test_captured_and_replayed():
    """One workspace for a captured forward and backward and for eager calls in between, on
    another stream than the tensors'."""
    counts, N, K = [33, 0, 190, 4], 328, 200
    off, o = offsets_of(counts)
    R, E = o[-1], len(counts)
    x, w, dy = randn(71, R, K), randn(72, E, N, K, std=K ** -0.5), randn(73, R, N, std=0.1)
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    y, dx, dw = torch.zeros(R, N, dtype=BF16, device="cuda"), torch.zeros_like(x), torch.zeros_like(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_grouped_linear(d, x, off, w, y, ws)
        moe.moe_grouped_linear_backward(d, dy, x, off, w, dx, dw, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            moe.moe_grouped_linear(d, x, off, w, y, ws)
            moe.moe_grouped_linear_backward(d, dy, x, off, w, dx, dw, ws)
        # other inputs and other segments: the offsets are read at each replay
        x.copy_(randn(74, R, K))
        off2, o2 = offsets_of([0, 100, 7, 120])
        off.copy_(off2)
        for t in (y, dx, dw):
            t.zero_()
        graph.replay()
        moe.moe_grouped_linear(d, x, off, w, y, ws)
        graph.replay()
    torch.cuda.synchronize()
    status_ok(ws)
    check_forward(x, w, o2, y, y)
    check_backward(dy, x, w, o2, dx, dw, None, dx)
