"""The experts' products at the ends of what they take: 512 experts, offsets past 32 bits, weights
and offsets written by the launch before, one workspace for calls of every kind (needs a GB300)."""

import pytest
import torch

import int4_ref
import routed_expert_ffn_gb300 as moe
from dense_ref import assert_within, product_bound
from test_gpu_grouped import check_backward, check_forward, offsets_of, randn, rounded, status_ok
from test_gpu_int4 import forward_bound, weights

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_ffn_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("R", [7, 400, 1500])
def test_512_experts(R):
    E, N, K, group = 512, 264, 160, 64
    counts = [R // E + (1 if (e * 37) % E < R % E else 0) for e in range(E)]
    off, o = offsets_of(counts)
    x, w = randn(1, R, K, dtype=FP16), randn(2, E, N, K, std=K ** -0.5, dtype=FP16)
    y = torch.zeros(R, N, device="cuda")
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_FP16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    status_ok(ws)
    check_forward(x, w, o, y, y)
    dy, dx, dw = randn(3, R, N, dtype=FP16), torch.zeros_like(x), torch.full_like(w, float("nan"))
    moe.moe_grouped_linear_backward(d, dy, x, off, w, dx, dw, ws)
    status_ok(ws)
    check_backward(dy, x, w, o, dx, dw, None, dx)
    q, s = weights(4, E, N, K, group=group, dtype=FP16)
    moe.moe_grouped_linear_int4(d, group, x, off, q, s, y, ws)
    status_ok(ws)
    for e in range(E):
        if counts[e]:
            rows = slice(o[e], o[e + 1])
            want, bound = forward_bound(x[rows].double(), int4_ref.values(q[e], s[e], group), None, None,
                                        "none", FP32)
            assert_within(y[rows], want, bound, f"expert {e}")


def test_rows_past_32_bits():
    """dy and y of more than 2^31 numbers."""
    E, N, K, group = 3, 32768, 64, 32
    off, o = offsets_of([65536, 0, 4465])
    R = o[-1]
    assert R * N > 1 << 31
    x, w = randn(11, R, K), randn(12, E, N, K, std=K ** -0.5)
    y = torch.zeros(R, N, dtype=BF16, device="cuda")
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    status_ok(ws)
    places = [(0, slice(0, 70)), (0, slice(65500, 65536)), (2, slice(65536, 65600)), (2, slice(R - 70, R))]
    for e, rows in places:
        a, b = x[rows].double(), w[e].double()
        want = a @ b.t()
        assert_within(y[rows], want, rounded(want, product_bound(a, b, K), BF16), f"rows {rows}")
    dx, dw = torch.zeros_like(x), torch.zeros(E, N, K, device="cuda")
    moe.moe_grouped_linear_backward(d, y, x, off, w, dx, dw, ws)
    status_ok(ws)
    for e, rows in places:
        a, b = y[rows].double(), w[e].double()
        want = a @ b
        assert_within(dx[rows], want, rounded(want, product_bound(a, b.t(), N), BF16), f"dx {rows}")
    rows = slice(65536, R)
    for n in (slice(0, 40), slice(N - 40, N)):
        a, b = y[rows, n].double(), x[rows].double()
        want = a.t() @ b
        assert_within(dw[2, n], want, rounded(want, product_bound(a.t(), b.t(), R - 65536), FP32), "dw")
    assert bool((dw[1] == 0).all())
    q, s = weights(13, E, N, K, group=group, dtype=BF16)
    moe.moe_grouped_linear_int4(d, group, x, off, q, s, y, ws)
    status_ok(ws)
    for e, rows in places:
        want, bound = forward_bound(x[rows].double(), int4_ref.values(q[e], s[e], group), None, None, "none",
                                    BF16)
        assert_within(y[rows], want, bound, f"4 bits, rows {rows}")


def test_matrices_past_32_bits():
    E, N, K = 512, 4096, 1032
    assert E * N * K > 1 << 31
    counts = [0] * E
    counts[0], counts[300], counts[511] = 3, 5, 9
    off, o = offsets_of(counts)
    R = o[-1]
    w = torch.zeros(E, N, K, dtype=BF16, device="cuda")
    for e in (0, 300, 511):
        w[e] = randn(20 + e, N, K, std=K ** -0.5)
    x, dy = randn(21, R, K), randn(22, R, N)
    y, dx, dw = torch.zeros(R, N, dtype=BF16, device="cuda"), torch.zeros_like(x), torch.full_like(w, 3.0)
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear(d, x, off, w, y, ws)
    moe.moe_grouped_linear_backward(d, dy, x, off, w, dx, dw, ws)
    status_ok(ws)
    pick = [0, 300, 511]
    o3 = [o[0], o[300], o[511], o[512]]
    check_forward(x, w[pick], o3, y, y)
    check_backward(dy, x, w[pick], o3, dx, dw[pick], None, dx)
    for e in (1, 299, 301, 510):
        assert bool((dw[e] == 0).all()), f"dw of expert {e}, which has no rows"


def test_codes_past_32_bits():
    E, N, K, group = 512, 8192, 1024, 128
    w = torch.zeros(E, N, K, dtype=BF16, device="cuda")
    for e in (0, 511):
        w[e] = randn(30 + e, N, K, std=K ** -0.5)
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // group, dtype=BF16, device="cuda")
    assert w.numel() > 1 << 31 and q.numel() >= 1 << 31
    moe.moe_quantize_int4(w, E * N, K, group, q, s)
    for e in (0, 511):
        codes, scale = int4_ref.quantize(w[e], group)
        assert torch.equal(s[e], scale) and torch.equal(q[e], int4_ref.pack(codes))
    assert bool((q[255] == 0x88).all()) and bool((s[255] == 0).all())
    counts = [0] * E
    counts[0], counts[511] = 20, 3
    off, o = offsets_of(counts)
    x, y = randn(33, 23, K), torch.zeros(23, N, device="cuda")
    d = moe.grouped_desc(23, E, N, K, moe.MOE_DTYPE_BF16, out_dtype=moe.MOE_DTYPE_FP32)
    ws = moe.alloc_workspace(d)
    moe.moe_grouped_linear_int4(d, group, x, off, q, s, y, ws)
    status_ok(ws)
    for e, rows in ((0, slice(0, 20)), (511, slice(20, 23))):
        want, bound = forward_bound(x[rows].double(), int4_ref.values(q[e], s[e], group), None, None, "none", FP32)
        assert_within(y[rows], want, bound, f"expert {e}")


@pytest.mark.parametrize("T,K", [(1, 2048), (8, 16384), (40, 2048)])
def test_weights_of_the_launch_before(T, K):
    """Codes and scales that the launch before wrote: never those before them."""
    N, group = 4096, 64
    x = randn(41, T, K, dtype=FP16)
    ws_of = [randn(42 + i, N, K, std=K ** -0.5, dtype=FP16) for i in range(2)]
    q = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(N, K // group, dtype=FP16, device="cuda")
    d = moe.linear_desc(T, N, K, moe.MOE_DTYPE_FP16)
    ws = moe.alloc_workspace(d)
    ys = [torch.empty(T, N, dtype=FP16, device="cuda") for _ in range(12)]
    for i, y in enumerate(ys):
        moe.moe_quantize_int4(ws_of[i % 2], N, K, group, q, s)
        moe.moe_linear_int4(d, group, x, q, s, None, None, y, ws)
    status_ok(ws)
    assert not torch.equal(ys[0], ys[1])
    for i, y in enumerate(ys):
        assert torch.equal(y, ys[i % 2]), f"call {i}"


def test_offsets_of_the_launch_before():
    """Offsets and rows that a kernel wrote just before."""
    E, N, K, R, group = 16, 512, 1024, 64, 32
    x, w = randn(51, R, K), randn(52, E, N, K, std=K ** -0.5)
    q, s = weights(53, E, N, K, group=group, dtype=BF16)
    kinds = [torch.arange(E + 1, device="cuda", dtype=torch.int32) * 4,
             torch.tensor([0] * 9 + [R] * 8, device="cuda", dtype=torch.int32)]
    d = moe.grouped_desc(R, E, N, K, moe.MOE_DTYPE_BF16)
    ws = moe.alloc_workspace(d)
    off = kinds[0].clone()
    out = [[torch.empty(R, N, dtype=BF16, device="cuda") for _ in range(2)] + [torch.empty_like(w)]
           for _ in range(8)]
    for i, (y, y4, dw) in enumerate(out):
        off.copy_(kinds[i % 2])
        moe.moe_grouped_linear(d, x, off, w, y, ws)
        off.copy_(kinds[i % 2])
        moe.moe_grouped_linear_int4(d, group, x, off, q, s, y4, ws)
        moe.moe_grouped_linear_backward(d, y, x, off, w, None, dw, ws)
    status_ok(ws)
    for i, got in enumerate(out):
        for a, b in zip(got, out[i % 2]):
            assert torch.equal(a, b), f"call {i}"
    for i in range(2):
        check_forward(x, w, kinds[i].tolist(), out[i][0], out[i][0])
        check_backward(out[i][0], x, w, kinds[i].tolist(), None, out[i][2], None, None)


def test_one_workspace_for_all():
    """Dense, 4-bit and grouped calls take turns in one workspace, captured and replayed: each leaves
    it as the next one needs it."""
    T, N, K, E, group = 37, 776, 1024, 5, 128
    x, w = randn(61, T, K), randn(62, E, N, K, std=K ** -0.5)
    q, s = weights(63, E, N, K, group=group, dtype=BF16)
    off, o = offsets_of([7, 0, 1, 20, 9])
    d, g = moe.linear_desc(T, N, K, moe.MOE_DTYPE_BF16), moe.grouped_desc(T, E, N, K, moe.MOE_DTYPE_BF16)
    one, two = moe.alloc_workspace(d), moe.alloc_workspace(g)
    ws = one if one.numel() * one.element_size() >= two.numel() * two.element_size() else two
    ys = [torch.zeros(T, N, dtype=BF16, device="cuda") for _ in range(4)]

    def step():
        moe.moe_linear(d, x, w[3], None, None, ys[0], ws)
        moe.moe_grouped_linear(g, x, off, w, ys[1], ws)
        moe.moe_linear_int4(d, group, x, q[3], s[3], None, None, ys[2], ws)
        moe.moe_grouped_linear_int4(g, group, x, off, q, s, ys[3], ws)

    step()
    first = [y.clone() for y in ys]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for _ in range(3):
        for y in ys:
            y.zero_()
        graph.replay()
    torch.cuda.synchronize()
    status_ok(ws)
    for a, b in zip(ys, first):
        assert torch.equal(a, b)
    check_forward(x, w, o, ys[1], ys[1])
    check_forward(x, w[3:4], [0, T], ys[0], ys[0])
    want, bound = forward_bound(x.double(), int4_ref.values(q[3], s[3], group), None, None, "none", BF16)
    assert_within(ys[2], want, bound, "4 bits")
    assert_within(ys[3][o[3]:o[4]], want[o[3]:o[4]], bound[o[3]:o[4]], "4 bits, expert 3")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,K", [(3, 96), (1000, 2080), (20000, 4096)])
def test_values_in_place(rows, K, group, dtype):
    """The values written over the weights: as beside them."""
    w = randn(71, rows, K, std=K ** -0.5, dtype=dtype)
    q = [torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.empty(rows, -(-K // group), dtype=dtype, device="cuda") for _ in range(2)]
    v = torch.empty_like(w)
    moe.moe_quantize_int4(w, rows, K, group, q[0], s[0], v)
    moe.moe_quantize_int4(w, rows, K, group, q[1], s[1], w)
    assert torch.equal(q[0], q[1]) and torch.equal(s[0], s[1]) and torch.equal(v, w)


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP32)])
@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("E,N,K", [(64, 264, 544), (40, 1000, 7168), (64, 136, 17952), (512, 40, 32)])
def test_few_rows_and_all_of_one(E, N, K, group, dtype, out):
    """Few rows on average, all of them or most with one expert: several passes over its matrix."""
    wide = torch.full((E + 9, K + 8), float("nan"), dtype=dtype, device="cuda")
    wide[3:3 + E, :K] = randn(81, E, K, dtype=dtype)
    x = wide[:, :K]
    q, s = weights(82, E, N, K, group=group, dtype=dtype)
    d = moe.grouped_desc(E + 9, E, N, K, moe.dtype_of(wide), out_dtype=moe.MOE_DTYPE_FP32 if out == FP32 else None,
                         x_stride=K + 8, y_stride=N + 16)
    ws = moe.alloc_workspace(d)
    for counts in ([0] * (E // 2) + [E] + [0] * (E - E // 2 - 1), [1] + [0] * (E - 2) + [E - 1],
                   [E - 12] + [11, 1] + [0] * (E - 3), [1] * E):
        off, o = offsets_of(counts, 3)
        yw = torch.full((E + 9, N + 16), 3.0, dtype=out, device="cuda")
        y = yw[:, :N]
        moe.moe_grouped_linear_int4(d, group, x, off, q, s, y, ws)
        status_ok(ws)
        for e in [e for e in range(E) if counts[e]][:6]:
            rows = slice(o[e], o[e + 1])
            want, bound = forward_bound(x[rows].double(), int4_ref.values(q[e], s[e], group), None, None,
                                        "none", out)
            assert_within(y[rows], want, bound, f"expert {e}")
        assert bool((yw[:3] == 3).all()) and bool((yw[3 + E:] == 3).all()) and bool((yw[:, N:] == 3).all())
    y0 = y.clone()
    for bad in ([-1] + [4] * E, [0, 9] + [8] * (E - 1), [0] * E + [E + 10]):
        y.fill_(5.0)
        moe.moe_workspace_init(ws)
        moe.moe_grouped_linear_int4(d, group, x, torch.tensor(bad, dtype=torch.int32, device="cuda"), q, s, y, ws)
        st, _ = moe.moe_get_device_status(ws)
        assert st != moe.MOE_OK and bool((y == 5).all())
    moe.moe_workspace_init(ws)
    moe.moe_grouped_linear_int4(d, group, x, off, q, s, y, ws)
    status_ok(ws)
    assert torch.equal(y[3:3 + E], y0[3:3 + E])
