"""The sorted rows and the 8-bit products at the places where their kernels change over, and the layer made of them."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_stable_b200 as moe
from sparse_mixture_experts_stable_b200 import binding as B
from sparse_mixture_experts_stable_b200.layer import SwiGLUMoEInt8
from tests.gpu_util import DEV, cpu, cpu64
from tests.sorted_util import HALF, U, ref_quantize, ref_sort, ref_unsort, routing, within
from tests.test_gpu_i8 import _dev, _ffn_ref, _i8, _product, _scale, _weights

pytestmark = pytest.mark.gpu


# around the super-blocks' sizes (1024 to 4096, or more where experts are many), and duplicated experts
@pytest.mark.parametrize("T,k,E", [(4095, 1, 2048), (4097, 1, 2048), (65536, 1, 3), (16384, 8, 256), (70000, 4, 16), (33000, 8, 2048),
                                   (5000, 64, 7), (100001, 3, 300)])
def test_order_large(T, k, E):
    rng = np.random.default_rng(T)
    sel = rng.integers(-1, E, (T, k))
    sel[: T // 3] = np.minimum(sel[: T // 3], E // 2)  # some experts far more often
    r = moe.moe_sort(torch.from_numpy(sel).to(DEV), E)
    off, row, src = ref_sort(sel, E)
    np.testing.assert_array_equal(cpu(r["offsets"]), off)
    np.testing.assert_array_equal(cpu(r["row"]), row)
    np.testing.assert_array_equal(cpu(r["source"]), src)


# narrow rows share a warp, wide ones take several steps; every alignment of rows that follow one another
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [1, 2, 3, 8, 16, 63, 64, 66, 72, 255, 257, 1030, 2047, 4100, 9001])
def test_there_and_back_at_every_alignment(dtype, D):
    T, k, E = 1100, 4, 16  # 4400 assignments: the form of several launches
    rng = np.random.default_rng(D)
    sel = routing(rng, T, k, E, dropped=0.1)
    sel[-3:] = -1
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(D)).to(dtype)
    off, row, src = ref_sort(sel, E)
    n = off[-1]
    xs = torch.full((T * k, D), 7.0, dtype=dtype, device=DEV)
    r = moe.moe_sort(torch.from_numpy(sel).to(DEV), E, x.to(DEV), out=dict(xs=xs))
    assert torch.equal(xs[:n].cpu(), x[torch.from_numpy(src[:n] // k)]) and (xs[n:] == 7).all()
    q = moe.moe_sort_i8(torch.from_numpy(sel).to(DEV), E, x.to(DEV))
    wq, wsc = ref_quantize(cpu64(x))
    np.testing.assert_array_equal(cpu64(q["xq"])[:n], wq[src[:n] // k])
    np.testing.assert_array_equal(cpu64(q["xscale"])[:n], wsc[src[:n] // k])
    g = torch.from_numpy(rng.uniform(0, 1, (T, k)).astype(np.float32))
    base = torch.randn(T, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    y = moe.moe_unsort(xs[:n], r["row"], g.to(DEV), base=base.to(DEV))
    want, mag = ref_unsort(cpu64(xs), row, cpu64(g), cpu64(base), D)
    sums = k * U * mag * 1.001
    within(cpu64(y), want, sums + HALF[dtype] * (np.abs(want) + sums), "y")
    dys = torch.full((T * k, D), 5.0, dtype=dtype, device=DEV)
    _, dg = moe.moe_unsort_backward(base.to(DEV), xs[:n], r["row"], g.to(DEV), dys=dys[:n])
    t = src[:n] // k
    want = cpu64(g).reshape(-1)[src[:n]][:, None] * cpu64(base)[t]
    within(cpu64(dys)[:n], want, np.abs(want) * (U + (HALF[dtype] if dtype == torch.bfloat16 else 0.0)) * 1.001, "dys")
    assert (dys[n:] == 5).all()
    terms = cpu64(base)[t] * cpu64(xs)[:n]
    wg, mg = np.zeros(T * k), np.zeros(T * k)
    wg[src[:n]], mg[src[:n]] = terms.sum(1), np.abs(terms).sum(1)
    within(cpu64(dg).reshape(-1), wg, D * U * mg * 1.001 + 1e-300, "dgates")


@pytest.mark.parametrize("shift", range(4))
def test_there_and_back_from_odd_addresses(shift):
    # rows of matrices that start off every boundary, with other values around them
    T, k, E, D = 1200, 4, 8, 130
    rng = np.random.default_rng(shift)
    sel = routing(rng, T, k, E)
    src = torch.from_numpy(ref_sort(sel, E)[2]).to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        def odd(rows, fill):
            flat = torch.full((rows * (D + 5) + 16,), fill, dtype=dtype, device=DEV)
            return flat, flat[shift:shift + rows * (D + 5)].view(rows, D + 5)[:, 2:2 + D]

        _, x = odd(T, 3.0)
        x.copy_(torch.randn(T, D))
        flat, xs = odd(T * k, 7.0)
        r = moe.moe_sort(torch.from_numpy(sel).to(DEV), E, x, out=dict(xs=xs))
        assert torch.equal(xs, x[src // k])
        assert int((flat == 7).sum()) >= flat.numel() - T * k * D
        yflat, y = odd(T, 9.0)
        moe.moe_unsort(xs, r["row"], y=y)
        want = k * x.double()
        assert ((y.double() - want).abs() <= (HALF[dtype] + k * U) * 1.001 * want.abs()).all()
        assert int((yflat == 9).sum()) >= yflat.numel() - T * D
        dflat, dys = odd(T * k, 5.0)
        _, dg = moe.moe_unsort_backward(x, xs, r["row"], dys=dys)
        assert torch.equal(dys, x[src // k])
        assert int((dflat == 5).sum()) >= dflat.numel() - T * k * D
        want = (x.double() ** 2).sum(1, keepdim=True).expand(T, k)
        assert ((dg.double() - want).abs() <= D * U * 1.001 * want).all()


def test_offsets_beyond_32_bits():
    # 320000 rows of 8192 bf16: 2.6e9 elements, 5.2 GB
    T, k, E, D = 160000, 2, 4, 8192
    g = torch.Generator(device=DEV).manual_seed(1)
    sel = torch.argsort(torch.rand(T, E, device=DEV, generator=g), dim=1)[:, :k].contiguous()
    x = torch.randn(T, 64, device=DEV, generator=g).to(torch.bfloat16).repeat(1, D // 64)
    r = moe.moe_sort(sel, E, x)
    some = torch.tensor([0, 1, T * k // 2, T * k - 2, T * k - 1], device=DEV)
    assert torch.equal(r["xs"][some], x[r["source"][some].long() // k])
    y = moe.moe_unsort(r["xs"], r["row"])
    assert torch.equal(y[-5:], 2 * x[-5:]) and torch.equal(y[:5], 2 * x[:5])
    dys, dg = moe.moe_unsort_backward(x, r["xs"], r["row"])
    assert torch.equal(dys[some], r["xs"][some])
    want = (x[-5:].double() ** 2).sum(1, keepdim=True).expand(5, k)
    assert ((dg[-5:].double() - want).abs() <= D * U * want).all()


def test_quantize_every_quotient_of_two_bf16():
    # all mantissas of the largest value against all values below it that differ from it by up to 2^9, at three scales
    for scale in (1.0, 2.0 ** 110, 2.0 ** -115):
        m = torch.arange(128, 256, dtype=torch.float32)
        e = torch.arange(0, 10, dtype=torch.float32)
        v = (m[None, :] * 2.0 ** -e[:, None]).reshape(-1)
        x = torch.where(v[None, :] <= m[:, None], v[None, :], 0.0)
        x = (torch.cat([m[:, None], x, -x], 1) * scale).to(torch.bfloat16)
        q, s = moe.moe_quantize_i8(x.to(DEV))
        want, ws = ref_quantize(cpu64(x))
        np.testing.assert_array_equal(cpu64(q), want)
        np.testing.assert_array_equal(cpu64(s), ws)


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** -100, 2.0 ** -125])
def test_quantize_near_ties_in_fp32_at_the_ends_of_the_range(scale):
    m = np.float32(1.7)
    t = (np.arange(-127, 127) + 0.5) * (np.float64(m) / 127)
    c = t.astype(np.float32)
    x = np.concatenate([[m], c, np.nextafter(c, np.float32(9)), np.nextafter(c, np.float32(-9))])[None]
    x = (x * np.float32(scale)).astype(np.float32)
    q, _ = moe.moe_quantize_i8(torch.from_numpy(x).to(DEV))
    np.testing.assert_array_equal(cpu64(q), ref_quantize(x.astype(np.float64))[0])


# few rows per group and many: depths around the few-row kernel's limit and its 256-byte pieces, features around 16 and 128,
# rows around 16, and the change to tiles
@pytest.mark.parametrize("M,K,N", [(15, 255, 15), (16, 256, 17), (17, 257, 127), (40, 2048, 129), (8, 2049, 100), (9, 4096, 300),
                                   (3, 4097, 40), (130, 1000, 257), (300, 2048, 900), (400, 2047, 1000), (2048, 64, 64),
                                   (2049, 64, 64), (70, 4095, 700), (1, 131071, 33), (257, 4200, 520)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dense_around_the_changes(M, K, N, dtype):
    xq, wq, xs, ws = _i8((M, K), 1), _i8((1, N, K), 2), _scale((M,), 3), _scale((1, N), 4)
    bias = _scale((1, N), 5) if N % 2 else None
    out = torch.full((M + 1, N + 2), 7.0, dtype=dtype, device=DEV)
    status = moe.new_status(DEV)
    moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), bias=None if bias is None else bias.to(DEV),
                      out=out[:M, 1:N + 1], dev_status=status)
    want, bound, _ = _product(xq, xs, wq, ws, bias, [0, M], dtype)
    within(cpu64(out)[:M, 1:N + 1], want, bound, "out")
    assert (out[M] == 7).all() and (out[:, 0] == 7).all() and (out[:, N + 1] == 7).all()
    assert moe.moe_read_status(status) == 0


def _storage_ends_with_the_last_value(t):
    """A copy on the GPU whose last row has nothing behind its K values."""
    K, ld = t.shape[-1], -(-t.shape[-1] // 16) * 16
    rows = t.numel() // K
    flat = torch.zeros((rows - 1) * ld + K, dtype=torch.int8, device=DEV)
    s = flat.as_strided(t.shape, (t.shape[-2] * ld, ld, 1)[-t.dim():])
    s.copy_(t.to(DEV))
    return s


@pytest.mark.parametrize("M,G", [(5, 1), (700, 1), (12, 4), (900, 4)])
@pytest.mark.parametrize("K", [5, 17, 250, 1001])
def test_rows_with_nothing_behind_the_last_one(M, G, K):
    N = 50
    xq, wq, xs, ws = _i8((M, K), 1), _i8((G, N, K), 2), _scale((M,), 3), _scale((G, N), 4)
    off = np.linspace(0, M, G + 1).astype(np.int32)
    out = moe.moe_matmul_i8(_storage_ends_with_the_last_value(xq), xs.to(DEV), _storage_ends_with_the_last_value(wq), ws.to(DEV),
                            offsets=torch.from_numpy(off).to(DEV), out_dtype=torch.float32)
    want, bound, _ = _product(xq, xs, wq, ws, None, off, torch.float32)
    within(cpu64(out), want, bound, "out")


# groups without rows in long runs, one full group among empty ones, as many groups as the few-row kernel takes and more
@pytest.mark.parametrize("counts", [[0] * 500 + [1] + [0] * 523, [0] * 1000 + [2, 0, 17, 33] + [0] * 21, [2] * 1024, [1] * 1025,
                                    [0, 64, 0, 0], [600] + [0] * 199, [4] * 60, [5] * 60])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_around_the_changes(counts, dtype):
    G, K, N = len(counts), 72, 40
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1])
    xq, wq, xs, ws = _i8((M, K), 1), _i8((G, N, K), 2), _scale((M,), 3), _scale((G, N), 4)
    status = moe.new_status(DEV)
    out = moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), offsets=torch.from_numpy(off).to(DEV), out_dtype=dtype,
                            dev_status=status)
    want, bound, _ = _product(xq, xs, wq, ws, None, off, dtype)
    within(cpu64(out), want, bound, "out")
    assert moe.moe_read_status(status) == 0


# few rows (the second product quantises the hidden rows itself, up to a width) and many, all kinds
@pytest.mark.parametrize("kind", ["swiglu", "gelu_mlp", "linear"])
@pytest.mark.parametrize("counts,D,F,Dout", [([1, 0, 2], 100, 260, 40), ([0, 9, 0, 0, 3, 1], 64, 4096, 24),
                                             ([2, 1], 33, 4100, 17), ([17, 0, 1], 2050, 50, 130), ([40, 300], 300, 130, 70)])
def test_ffn_around_the_changes(kind, counts, D, F, Dout):
    G = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1])
    q, s = ref_quantize(torch.randn(M, D, generator=torch.Generator().manual_seed(M)).double().numpy())
    xq, xs = torch.from_numpy(q).to(torch.int8), torch.from_numpy(s).float()
    w = _weights(kind, G, D, F, Dout, D)
    want, bound = _ffn_ref(kind, xq, xs, off, w, torch.float32)
    status = moe.new_status(DEV)
    ys = moe.moe_expert_ffn_i8(kind, _dev(xq), xs.to(DEV), torch.from_numpy(off.astype(np.int32)).to(DEV),
                               out_dtype=torch.float32, dev_status=status, **{n: _dev(t) for n, t in w.items()})
    within(cpu64(ys), want, bound, "ys")
    assert moe.moe_read_status(status) == 0


def test_few_and_many_rows_agree_bit_for_bit():
    # the same rows alone (few-row kernel) and among others (tiles): integer sums and the same scaling
    E, D, F = 4, 200, 96
    w = {n: _dev(t) for n, t in _weights("swiglu", E, D, F, D, 3).items()}
    q, s = moe.moe_quantize_i8(torch.randn(800, D, device=DEV))
    off = torch.tensor([0, 200, 400, 600, 800], dtype=torch.int32, device=DEV)
    all_rows = moe.moe_expert_ffn_i8("swiglu", q, s, off, out_dtype=torch.float32, **w)
    for e in range(E):
        one = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        one[e + 1:] = 3
        rows = _dev(q[200 * e:200 * e + 3].cpu())
        few = moe.moe_expert_ffn_i8("swiglu", rows, s[200 * e:200 * e + 3].contiguous(), one, out_dtype=torch.float32, **w)
        assert torch.equal(few, all_rows[200 * e:200 * e + 3])


def test_graphs_of_a_large_step_that_share_a_workspace():
    # tiles drawn from the counter (a memset before the kernel), replayed on changed inputs; two graphs, one workspace, in turn
    T, k, E, H, F = 6000, 4, 40, 256, 192
    rng = np.random.default_rng(1)
    w = {n: _dev(t) for n, t in _weights("swiglu", E, H, F, H, 9).items()}
    sels = [torch.from_numpy(routing(rng, T, k, E, dropped=0.1)).to(DEV) for _ in range(3)]
    xs = [torch.randn(T, H, device=DEV).to(torch.bfloat16) for _ in range(3)]
    gates = torch.rand(T, k, device=DEV)
    ws = torch.zeros(B.moe_expert_ffn_i8_workspace_size("swiglu", E, T * k, H, F, H), dtype=torch.uint8, device=DEV)
    wsort = torch.zeros(B.moe_sort_workspace_size(T, k, E), dtype=torch.uint8, device=DEV)

    def step(sel, x):
        s = moe.moe_sort_i8(sel, E, x, workspace=wsort)
        ys = moe.moe_expert_ffn_i8("swiglu", s["xq"], s["xscale"], s["offsets"], workspace=ws, **w)
        return moe.moe_unsort(ys, s["row"], gates)

    want = [step(s, x).clone() for s, x in zip(sels, xs)]
    again = step(sels[0], xs[0])
    assert torch.equal(again, want[0])
    graphs = []
    for _ in range(2):
        s, x = sels[2].clone(), xs[2].clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step(s, x)
        graphs.append((g, s, x, o))
    for i in (0, 1, 0):
        g, s, x, o = graphs[i]
        s.copy_(sels[i]), x.copy_(xs[i])
        ws.fill_(255), wsort.fill_(255)  # nothing is carried over in a workspace
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i])


def test_the_binding_refuses_what_does_not_fit():
    x = torch.randn(6, 32, device=DEV)
    sel = torch.zeros(6, 2, dtype=torch.int64, device=DEV)
    row = torch.zeros(6, 2, dtype=torch.int32, device=DEV)
    q, s = moe.moe_quantize_i8(x)
    wq, ws = moe.moe_quantize_i8(torch.randn(1, 8, 32, device=DEV))
    bad = [
        lambda: moe.moe_sort(sel.int(), 4), lambda: moe.moe_sort(sel, 0), lambda: moe.moe_sort(sel.t(), 4),
        lambda: moe.moe_sort(sel, 4, x[:5]), lambda: moe.moe_sort(sel, 4, x.half()), lambda: moe.moe_sort(sel, 4, x.t()),
        lambda: moe.moe_sort(sel, 4, x[:1].expand(6, 32)), lambda: moe.moe_sort(sel, 4, x, out=dict(xs=x)),
        lambda: moe.moe_sort(sel, 4, x, workspace=torch.zeros(8)), lambda: moe.moe_sort(sel, 4, x, dev_status=x),
        lambda: moe.moe_sort_i8(sel, 4, x, out=dict(xq=q)), lambda: moe.moe_unsort(x, row.long()),
        lambda: moe.moe_unsort(x, row, torch.rand(6, 3, device=DEV)), lambda: moe.moe_unsort(x, row, base=x.bfloat16()),
        lambda: moe.moe_unsort(x, row, y=x[:, :5]), lambda: moe.moe_unsort_backward(x[:5], x, row),
        lambda: moe.moe_unsort_backward(x, None, row), lambda: moe.moe_unsort_backward(x, x[:, :5], row),
        lambda: moe.moe_quantize_i8(x[0]), lambda: moe.moe_quantize_i8(x, q=q[:3]), lambda: moe.moe_quantize_i8(x, scale=s[:3]),
        lambda: moe.moe_matmul_i8(q, s[:3], wq, ws), lambda: moe.moe_matmul_i8(q, s, wq[..., :16], ws),
        lambda: moe.moe_matmul_i8(q, s, wq, ws[0, :3]), lambda: moe.moe_matmul_i8(q, s, wq, ws, bias=s),
        lambda: moe.moe_matmul_i8(q, s, wq, ws, out_dtype=torch.float16),
        lambda: moe.moe_matmul_i8(q, s, wq, ws, offsets=torch.zeros(3, dtype=torch.int32, device=DEV)),
        lambda: moe.moe_matmul_i8(q, s, wq, ws, stream=torch.cuda.Stream(), out=x[:3]),
        lambda: moe.moe_expert_ffn_i8("swiglu", q, s, None, wq, ws), lambda: moe.moe_expert_ffn_i8("linear", q, s, None, wq, ws, w2=wq),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            raise AssertionError(f"call {i} was taken")


@pytest.mark.parametrize("T,H,E,F,k,Fs", [(1, 64, 8, 32, 2, 0), (33, 136, 16, 40, 4, 56), (700, 256, 32, 128, 8, 128)])
def test_layer(T, H, E, F, k, Fs):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    wr, bias = torch.randn(E, H, generator=g).to(torch.bfloat16).to(DEV), torch.randn(E, generator=g).to(DEV)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.1).to(torch.bfloat16).to(DEV)  # noqa: E731
    experts = SwiGLUMoEInt8.quantize(mk(E, F, H), mk(E, F, H), mk(E, H, F))
    shared = SwiGLUMoEInt8.quantize(mk(1, Fs, H), mk(1, Fs, H), mk(1, H, Fs)) if Fs else None
    layer = SwiGLUMoEInt8(T, H, E, F, k, F_shared=Fs, aux_coef=0.01)
    for _ in range(2):  # the buffers are used again
        o = layer.forward(x, wr, bias, experts, shared)
    assert moe.moe_read_status(layer.status) == 0
    off, row, src = ref_sort(cpu(o["selected"]), E)
    q, sc = ref_quantize(cpu64(x))
    to = lambda d: {n: t.cpu() for n, t in d.items()}  # noqa: E731
    rows = torch.from_numpy(q[src // k]).to(torch.int8), torch.from_numpy(sc[src // k]).float()
    ys, bound = _ffn_ref("swiglu", *rows, off, to(experts), torch.bfloat16)
    gates = cpu64(o["gates_f32"])[..., None]
    want, mag, err = (gates * ys[row]).sum(1), (gates * (np.abs(ys) + bound)[row]).sum(1), (gates * bound[row]).sum(1)
    if Fs:
        b, eb = _ffn_ref("swiglu", torch.from_numpy(q).to(torch.int8), torch.from_numpy(sc).float(), [0, T], to(shared),
                         torch.bfloat16)
        want, mag, err = want + b, mag + np.abs(b) + eb, err + eb
    err = err + (k + 1) * U * mag
    within(cpu64(o["y"]), want, err + HALF[torch.bfloat16] * (np.abs(want) + err), "y")
