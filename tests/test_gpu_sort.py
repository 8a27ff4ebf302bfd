"""moe_sort, moe_sort_i8, moe_unsort and moe_unsort_backward against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_stable_b200 as moe
from sparse_mixture_experts_stable_b200 import binding as B
from tests.gpu_util import DEV, cpu, cpu64
from tests.sorted_util import HALF, U, ref_quantize, ref_sort, ref_unsort, routing, within

pytestmark = pytest.mark.gpu

# tokens, choices, experts: one token, a block's edge, the one-launch form's last size and the next ones, many experts,
# many choices, more choices than experts
SIZES = [(1, 1, 1), (1, 8, 256), (3, 2, 8), (37, 3, 5), (512, 8, 64), (513, 8, 64), (4096, 1, 16), (4097, 1, 16),
         (300, 64, 2048), (2500, 5, 2048), (20000, 2, 7), (70, 64, 1000), (9000, 8, 256)]


def _check_order(r, sel, E):
    off, row, src = ref_sort(sel, E)
    np.testing.assert_array_equal(cpu(r["offsets"]), off)
    np.testing.assert_array_equal(cpu(r["row"]), row)
    np.testing.assert_array_equal(cpu(r["source"]), src)
    return off, row, src


@pytest.mark.parametrize("T,k,E", SIZES)
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_order(T, k, E, dropped):
    sel = routing(np.random.default_rng(T + k), T, k, E, dropped=dropped)
    status = moe.new_status(DEV)
    r = moe.moe_sort(torch.from_numpy(sel).to(DEV), E, dev_status=status)
    _check_order(r, sel, E)
    assert moe.moe_read_status(status) == 0


@pytest.mark.parametrize("sel", [np.zeros((700, 8), np.int64), np.full((700, 8), -1, np.int64),
                                 np.full((2, 3), -1, np.int64), np.tile(np.int64(63), (5, 2))])
def test_order_of_one_expert_and_of_none(sel):
    x = torch.randn(sel.shape[0], 40, device=DEV)
    r = moe.moe_sort(torch.from_numpy(sel).to(DEV), 64, x)
    off, _, src = _check_order(r, sel, 64)
    n = off[-1]
    assert torch.equal(r["xs"][:n], x[torch.from_numpy(src[:n] // sel.shape[1]).to(DEV)])


@pytest.mark.parametrize("T,k", [(20, 2), (5000, 2)])
def test_bad_indices_are_reported_and_take_no_part(T, k):
    sel = routing(np.random.default_rng(3), T, k, 8)
    for bad in (8, -2, 2 ** 40, -2 ** 62):
        s = sel.copy()
        s[T // 2, 1] = bad
        status = moe.new_status(DEV)
        r = moe.moe_sort(torch.from_numpy(s).to(DEV), 8, dev_status=status)
        _check_order(r, s, 8)
        assert moe.moe_read_status(status) == B.MOE_ERR_BAD_INDEX


def test_no_tokens():
    sel = torch.empty(0, 4, dtype=torch.int64, device=DEV)
    x = torch.empty(0, 32, device=DEV, dtype=torch.bfloat16)
    for r in (moe.moe_sort(sel, 9, x), moe.moe_sort_i8(sel, 9, x)):
        assert cpu(r["offsets"]).tolist() == [0] * 10 and r["row"].shape == (0, 4)
    assert moe.moe_unsort(torch.empty(0, 32, device=DEV), torch.empty(0, 4, dtype=torch.int32, device=DEV)).shape == (0, 32)
    # tokens without rows
    row = torch.full((5, 4), -1, dtype=torch.int32, device=DEV)
    assert torch.equal(moe.moe_unsort(torch.empty(0, 32, device=DEV), row), torch.zeros(5, 32, device=DEV))
    dys, dg = moe.moe_unsort_backward(torch.ones(5, 32, device=DEV), torch.empty(0, 32, device=DEV), row)
    assert dys.shape == (0, 32) and torch.equal(dg, torch.zeros(5, 4, device=DEV))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,E,D", [(1, 1, 4, 1), (5, 3, 4, 7), (600, 8, 64, 129), (33, 2, 8, 2048), (5000, 2, 64, 264),
                                     (2000, 4, 16, 1001), (64, 64, 100, 8192), (17, 2, 8, 20000)])
def test_rows(dtype, T, k, E, D):
    rng = np.random.default_rng(D)
    sel = routing(rng, T, k, E, dropped=0.2)
    x = torch.randn(T, D, device=DEV).to(dtype)
    xs = torch.full((T * k, D), 7.0, device=DEV, dtype=dtype)
    r = moe.moe_sort(torch.from_numpy(sel).to(DEV), E, x, out=dict(xs=xs))
    off, _, src = _check_order(r, sel, E)
    n = off[-1]
    assert torch.equal(xs[:n], x[torch.from_numpy(src[:n] // k).to(DEV)])
    assert (xs[n:] == 7.0).all()  # rows behind the last one stay


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("skip,width", [(0, 96), (1, 97), (2, 100), (8, 112), (3, 131)])
def test_rows_in_wider_matrices(dtype, skip, width):
    rng = np.random.default_rng(width)
    T, k, E, D = 700, 8, 16, 80
    sel = routing(rng, T, k, E)
    x = torch.randn(T, width, device=DEV).to(dtype)[:, skip:skip + D]
    big = torch.full((T * k, width + 1), 7.0, device=DEV, dtype=dtype)
    r = moe.moe_sort(torch.from_numpy(sel).to(DEV), E, x, out=dict(xs=big[:, skip:skip + D]))
    src = torch.from_numpy(ref_sort(sel, E)[2] // k).to(DEV)
    assert torch.equal(r["xs"], x[src])
    assert (big[:, :skip] == 7.0).all() and (big[:, skip + D:] == 7.0).all()


def _awkward_rows(T, D, dtype, seed):
    """Rows with exact ties (127 x / m half-way), zeros, one value, large and denormal values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g)
    x[0] = 0
    if T > 5 and D > 4:
        x[1] = torch.arange(D) % 128 - 63.5
        x[1, 0] = 127.0
        x[2] = 1e-38 * torch.randn(D, generator=g)
        x[3] = 3e38 * (2 * torch.rand(D, generator=g) - 1)
        x[4] = 0
        x[4, D // 2] = -2.5
        x[5] = 1e-41 * torch.arange(D)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (7, 5), (100, 64), (33, 1000), (9, 2048), (70, 131), (8, 9001)])
def test_quantize(dtype, M, K):
    x = _awkward_rows(M, K, dtype, K)
    q, scale = moe.moe_quantize_i8(x.to(DEV))
    want, s = ref_quantize(cpu64(x))
    np.testing.assert_array_equal(cpu64(q), want)
    np.testing.assert_array_equal(cpu64(scale), s)
    if M > 1:
        assert q.stride(0) % 16 == 0


def test_quantize_near_ties_in_fp32():
    # x next to every tie of its row, one fp32 step below, on and above it where fp32 holds it
    m = np.float32(1.7)
    t = (np.arange(-127, 127) + 0.5) * (np.float64(m) / 127)
    c = t.astype(np.float32)
    x = np.concatenate([[m], c, np.nextafter(c, np.float32(9)), np.nextafter(c, np.float32(-9))])[None]
    q, _ = moe.moe_quantize_i8(torch.from_numpy(x).to(DEV))
    np.testing.assert_array_equal(cpu64(q), ref_quantize(x.astype(np.float64))[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_reports_rows_that_are_not_finite(dtype):
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = torch.randn(5, 40).to(dtype)
        x[2, 17] = bad
        status = moe.new_status(DEV)
        q, scale = moe.moe_quantize_i8(x.to(DEV), dev_status=status)
        assert moe.moe_read_status(status) == B.MOE_ERR_NONFINITE
        assert torch.isnan(scale[2]) and (q[2] == 0).all()
        keep = [0, 1, 3, 4]
        want, s = ref_quantize(cpu64(x[keep]))
        np.testing.assert_array_equal(cpu64(q)[keep], want)
        np.testing.assert_array_equal(cpu64(scale)[keep], s)


def test_quantize_views():
    x = torch.randn(40, 75, device=DEV)
    want, s = ref_quantize(cpu64(x[:, 3:60]))
    buf = torch.full((40, 80), 99, dtype=torch.int8, device=DEV)
    q, scale = moe.moe_quantize_i8(x[:, 3:60], q=buf[:, 5:62])
    np.testing.assert_array_equal(cpu64(q), want)
    np.testing.assert_array_equal(cpu64(scale), s)
    assert (buf[:, :5] == 99).all() and (buf[:, 62:] == 99).all()
    w = torch.randn(3, 5, 37, device=DEV)
    q, scale = moe.moe_quantize_i8(w)
    want, s = ref_quantize(cpu64(w))
    np.testing.assert_array_equal(cpu64(q), want)
    np.testing.assert_array_equal(cpu64(scale), s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,E,D", [(1, 1, 4, 1), (16, 8, 256, 2048), (700, 8, 64, 131), (5000, 2, 64, 264), (40, 3, 8, 72)])
def test_sort_i8(dtype, T, k, E, D):
    sel = routing(np.random.default_rng(T), T, k, E, dropped=0.1)
    x = _awkward_rows(T, D, dtype, D)
    r = moe.moe_sort_i8(torch.from_numpy(sel).to(DEV), E, x.to(DEV))
    off, _, src = _check_order(r, sel, E)
    n = off[-1]
    want, s = ref_quantize(cpu64(x))
    np.testing.assert_array_equal(cpu64(r["xq"])[:n], want[src[:n] // k])
    np.testing.assert_array_equal(cpu64(r["xscale"])[:n], s[src[:n] // k])


def _back(T, k, E, dropped, seed):
    rng = np.random.default_rng(seed)
    sel = routing(rng, T, k, E, dropped=dropped)
    if T > 2:
        sel[T // 2] = -1  # a token without rows
        sel[-1] = -1      # a padding token
    off, row, _ = ref_sort(sel, E)
    return rng, off[-1], row


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gates", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,E,N", [(1, 1, 4, 1), (5, 3, 4, 7), (600, 8, 64, 129), (33, 2, 8, 2048), (300, 17, 64, 264),
                                     (40, 64, 100, 1001)])
@pytest.mark.parametrize("base", [False, True])
def test_unsort(dtype, gates, T, k, E, N, base):
    rng, R, row = _back(T, k, E, 0.2, N)
    ys = torch.randn(max(R, 1), N).to(dtype)
    g = None if gates is None else torch.from_numpy(rng.uniform(0, 1, (T, k)).astype(np.float32)).to(gates)
    b = torch.randn(T, N).to(dtype) if base else None
    status = moe.new_status(DEV)
    y = moe.moe_unsort(ys.to(DEV), torch.from_numpy(row.astype(np.int32)).to(DEV), None if g is None else g.to(DEV),
                       base=None if b is None else b.to(DEV), dev_status=status)
    want, mag = ref_unsort(cpu64(ys), row, None if g is None else cpu64(g), None if b is None else cpu64(b), N)
    # k fused multiply-adds in fp32, each off by U of a partial sum that is at most mag, then one rounding to the type
    sums = k * U * mag * 1.001
    within(cpu64(y), want, sums + HALF[dtype] * (np.abs(want) + sums), "y")
    assert moe.moe_read_status(status) == 0
    empty = (row < 0).all(1)
    np.testing.assert_array_equal(cpu64(y)[empty], 0.0 if b is None else cpu64(b)[empty])


def test_unsort_does_not_read_rows_that_no_token_has():
    ys = torch.full((6, 64), float("nan"), device=DEV)
    ys[2], ys[5] = 1.0, 2.0
    row = torch.tensor([[2, -1], [-1, 5], [-1, -1]], dtype=torch.int32, device=DEV)
    gates = torch.tensor([[0.5, float("nan")], [float("inf"), 0.25], [float("nan"), 1.0]], device=DEV)
    y = moe.moe_unsort(ys, row, gates)
    assert torch.equal(y, torch.tensor([0.5, 0.5, 0.0], device=DEV)[:, None].expand(3, 64))
    dys, dg = moe.moe_unsort_backward(torch.ones(3, 64, device=DEV), ys, row, gates, dys=torch.full_like(ys, 3.0))
    assert torch.equal(dg, torch.tensor([[64.0, 0.0], [0.0, 128.0], [0.0, 0.0]], device=DEV))
    assert (dys[2] == 0.5).all() and (dys[5] == 0.25).all() and (dys[[0, 1, 3, 4]] == 3.0).all()


def test_unsort_reports_rows_outside_and_skips_them():
    ys = torch.ones(4, 32, device=DEV)
    for bad in (4, -2, 2 ** 31 - 1, -2 ** 31):
        row = torch.tensor([[0, bad], [3, 1]], dtype=torch.int32, device=DEV)
        status = moe.new_status(DEV)
        y = moe.moe_unsort(ys, row, dev_status=status)
        assert moe.moe_read_status(status) == B.MOE_ERR_BAD_INDEX
        assert torch.equal(y, torch.tensor([1.0, 2.0], device=DEV)[:, None].expand(2, 32))
        moe.moe_clear_status(status)
        dys, dg = moe.moe_unsort_backward(2 * ys[:2], ys, row, dys=torch.zeros_like(ys), dev_status=status)
        assert moe.moe_read_status(status) == B.MOE_ERR_BAD_INDEX
        assert torch.equal(dg, torch.tensor([[64.0, 0.0], [64.0, 64.0]], device=DEV))
        assert dys[:, 0].tolist() == [2.0, 2.0, 0.0, 2.0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gates", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,E,N", [(1, 1, 4, 1), (5, 3, 4, 7), (600, 8, 64, 129), (33, 2, 8, 2048), (300, 17, 64, 264),
                                     (40, 64, 100, 1001)])
def test_unsort_backward(dtype, gates, T, k, E, N):
    rng, R, row = _back(T, k, E, 0.2, N + 1)
    ys, dy = torch.randn(R, N).to(dtype), torch.randn(T, N).to(dtype)
    g = None if gates is None else torch.from_numpy(rng.uniform(0, 1, (T, k)).astype(np.float32)).to(gates)
    gd = None if g is None else g.to(DEV)
    rd = torch.from_numpy(row.astype(np.int32)).to(DEV)
    dys, dg = moe.moe_unsort_backward(dy.to(DEV), ys.to(DEV), rd, gd)
    want = np.zeros((R, N))
    wg, mag = np.zeros((T, k)), np.zeros((T, k))
    for t, j in zip(*np.nonzero(row >= 0)):
        want[row[t, j]] = (1.0 if g is None else cpu64(g)[t, j]) * cpu64(dy)[t]
        terms = cpu64(dy)[t] * cpu64(ys)[row[t, j]]
        wg[t, j], mag[t, j] = terms.sum(), np.abs(terms).sum()
    # one product in fp32, and its rounding to bf16
    within(cpu64(dys), want, np.abs(want) * (U + (HALF[dtype] if dtype == torch.bfloat16 else 0.0)) * 1.001, "dys")
    within(cpu64(dg), wg, N * U * mag * 1.001 + 1e-300, "dgates")  # a sum of N terms in any order
    # each alone gives the same
    only, none = moe.moe_unsort_backward(dy.to(DEV), None, rd, gd, rows=R, want_dgates=False)
    assert none is None and torch.equal(only, dys)
    none, only = moe.moe_unsort_backward(dy.to(DEV), ys.to(DEV), rd, gd, want_dys=False)
    assert none is None and torch.equal(only, dg)


def test_gradients_against_differences():
    # y is linear in x (through sort), in ys and in gates, so a difference of step 1 is the derivative
    T, k, E, N = 90, 4, 8, 67
    sel = routing(np.random.default_rng(5), T, k, E, dropped=0.1)
    gen = torch.Generator().manual_seed(1)
    x, dx0, dy = (torch.randn(T, N, generator=gen).to(DEV) for _ in range(3))
    gates, dg0 = torch.rand(T, k, generator=gen).to(DEV), torch.randn(T, k, generator=gen).to(DEV)

    def forward(x, gates):
        r = moe.moe_sort(torch.from_numpy(sel).to(DEV), E, x)
        return moe.moe_unsort(r["xs"], r["row"], gates), r

    y0, r = forward(x, gates)
    dys, dg = moe.moe_unsort_backward(dy, r["xs"], r["row"], gates)
    dx = moe.moe_unsort(dys, r["row"])
    along = ((forward(x + dx0, gates)[0].double() - y0.double()) * dy.double()).sum()
    mag = (forward(x.abs() + dx0.abs(), gates)[0].double() * dy.abs().double()).sum()
    # roundings of x + dx0 and of both forwards (k + 2 each) and of the gradient (k + 2), each U of mag
    assert abs(float(along - (dx.double() * dx0.double()).sum())) <= 3 * (k + 2) * U * float(mag)
    along = ((forward(x, gates + dg0)[0].double() - y0.double()) * dy.double()).sum()
    mag = (forward(x.abs(), gates + dg0.abs())[0].double() * dy.abs().double()).sum()
    assert abs(float(along - (dg.double() * dg0.double()).sum())) <= (3 * (k + 2) + N) * U * float(mag)


@pytest.mark.parametrize("T", [64, 3000])
def test_streams_and_graphs(T):
    k, E, D = 4, 16, 96
    rng = np.random.default_rng(T)
    sels = [torch.from_numpy(routing(rng, T, k, E, dropped=0.1)).to(DEV) for _ in range(3)]
    xs = [torch.randn(T, D, device=DEV).to(torch.bfloat16) for _ in range(3)]
    gates = torch.rand(T, k, device=DEV)

    def step(sel, x, stream=None):
        r = moe.moe_sort(sel, E, x, out=dict(xs=torch.zeros(T * k, D, device=DEV, dtype=x.dtype)) if stream is None else None,
                         stream=stream)
        y = moe.moe_unsort(r["xs"], r["row"], gates, stream=stream)
        dys, dg = moe.moe_unsort_backward(x, r["xs"], r["row"], gates, stream=stream)
        return y, dg

    want = [step(s, x) for s, x in zip(sels, xs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(sels[0], xs[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    # two graphs of the same calls, replayed on changed inputs, one after the other and at once
    bufs, graphs, outs = [], [], []
    for _ in range(2):
        s, x = sels[2].clone(), xs[2].clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step(s, x)
        bufs.append((s, x)), graphs.append(g), outs.append(o)
    for (s, x), src_s, src_x in zip(bufs, sels, xs):
        s.copy_(src_s), x.copy_(src_x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
