"""moe_matmul_i8 and moe_expert_ffn_i8 against plain 64-bit implementations, and the 8-bit layer they make up."""
import math

import numpy as np
import pytest
import torch

import sparse_mixture_experts_stable_b200 as moe
from sparse_mixture_experts_stable_b200 import binding as B
from tests.gpu_util import DEV, cpu64
from tests.sorted_util import HALF, U, ref_quantize, ref_sort, routing, within

pytestmark = pytest.mark.gpu


def _i8(shape, seed):
    """Random int8 with rows on multiples of 16 bytes and other values between the rows."""
    g = torch.Generator().manual_seed(seed)
    K = shape[-1]
    return torch.randint(-128, 128, (*shape[:-1], -(-K // 16) * 16), generator=g, dtype=torch.int8)[..., :K]


def _scale(shape, seed):
    return torch.rand(shape, generator=torch.Generator().manual_seed(seed)) * 0.02 + 1e-3


def _dev(t):
    """A copy on the GPU with the same strides."""
    if t.dtype != torch.int8:
        return t.to(DEV)
    pad = -(-t.shape[-1] // 16) * 16
    b = torch.full((*t.shape[:-1], pad), 77, dtype=torch.int8, device=DEV)
    b[..., :t.shape[-1]] = t.to(DEV)
    return b[..., :t.shape[-1]]


def _product(xq, xs, wq, ws, bias, offsets, dtype):
    """(value, bound, written): the exact sum, and the roundings of acc to fp32, of the two scales' product, of the
    product, of the sum with the bias, and to the type."""
    M, N = xq.shape[0], wq.shape[1]
    want, bound, written = np.zeros((M, N)), np.zeros((M, N)), np.zeros(M, bool)
    for g in range(wq.shape[0]):
        a, b = int(offsets[g]), int(offsets[g + 1])
        if a >= b:
            continue
        p = (cpu64(xq[a:b]) @ cpu64(wq[g]).T) * cpu64(xs)[a:b, None] * cpu64(ws)[g][None]
        v = p if bias is None else p + cpu64(bias)[g][None]
        e = 3.01 * U * np.abs(p) + (0 if bias is None else U * (np.abs(v) + 1e-6 * np.abs(p)))
        want[a:b], written[a:b] = v, True
        bound[a:b] = e + (HALF[dtype] * (np.abs(v) + e) if dtype == torch.bfloat16 else 0)
    return want, bound, written


# rows, depth, features: one of each, odd ones, whole tiles, one more than tiles, deep, wide
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 2048, 2048), (3, 17, 5), (31, 128, 256), (33, 129, 257), (256, 512, 512),
                                   (257, 100, 513), (300, 640, 770), (1003, 1000, 1537), (64, 20000, 40), (5, 131071, 3),
                                   (2, 16, 5000), (700, 48, 129)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dense(M, K, N, dtype):
    xq, wq, xs, ws = _i8((M, K), 1), _i8((1, N, K), 2), _scale((M,), 3), _scale((1, N), 4)
    bias = _scale((1, N), 5) if (M + N) % 2 else None
    status = moe.new_status(DEV)
    out = moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), bias=None if bias is None else bias.to(DEV),
                            out_dtype=dtype, dev_status=status)
    want, bound, _ = _product(xq, xs, wq, ws, bias, [0, M], dtype)
    within(cpu64(out), want, bound, "out")
    assert moe.moe_read_status(status) == 0


def test_largest_sums_are_exact():
    # 131071 products of -128 x -128 are the largest sum that int32 holds
    K = 131071
    x = torch.full((2, 131072), -128, dtype=torch.int8, device=DEV)[:, :K]
    w = x.clone().new_full((3, 131072), -128)[:, :K]
    one = torch.ones(3, device=DEV)
    out = moe.moe_matmul_i8(x, one[:2], w, one, out_dtype=torch.float32)
    assert torch.equal(out, torch.full((2, 3), float(np.float32(K * 128.0 * 128.0)), device=DEV))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_matmul_i8(torch.zeros(2, 131072, dtype=torch.int8, device=DEV), one[:2],
                          torch.zeros(3, 131072, dtype=torch.int8, device=DEV), one)
    assert e.value.code == B.MOE_ERR_UNSUPPORTED


COUNTS = [[0, 0, 0], [1], [0, 5, 0, 0, 1, 32, 33, 0], [300, 0, 1, 513, 256, 7], [1] * 40, [0] * 2047 + [3], [2, 0, 1] * 100]


@pytest.mark.parametrize("counts", COUNTS, ids=range(len(COUNTS)))
@pytest.mark.parametrize("K,N", [(96, 80), (260, 600)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped(counts, K, N, dtype):
    if len(counts) > 1000:
        K, N = 32, 24
    G = len(counts)
    front, behind = 3, 4  # rows outside the groups
    off = np.concatenate([[0], np.cumsum(counts)]) + front
    M = int(off[-1]) + behind
    xq, wq, xs, ws = _i8((M, K), 1), _i8((G, N, K), 2), _scale((M,), 3), _scale((G, N), 4)
    out = torch.full((M, N + 3), 7.0, dtype=dtype, device=DEV)
    status = moe.new_status(DEV)
    moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), offsets=torch.from_numpy(off.astype(np.int32)).to(DEV),
                      out=out[:, 1:N + 1], dev_status=status)
    want, bound, written = _product(xq, xs, wq, ws, None, off, dtype)
    got = cpu64(out)
    within(got[written][:, 1:N + 1], want[written], bound[written], "out")
    assert (got[~written] == 7).all() and (got[:, 0] == 7).all() and (got[:, N + 1:] == 7).all()
    assert moe.moe_read_status(status) == 0


def test_bad_offsets_stay_inside():
    M, K, N, G = 50, 64, 40, 4
    xq, wq, xs, ws = _i8((M, K), 1), _i8((G, N, K), 2), _scale((M,), 3), _scale((G, N), 4)
    status = moe.new_status(DEV)
    off = torch.tensor([-5, 10, 4, 30, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out = torch.full((M + 1, N), 7.0, device=DEV)
    moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), offsets=off, out=out[:M], dev_status=status)
    assert moe.moe_read_status(status) == B.MOE_ERR_BAD_INDEX
    want, bound, _ = _product(xq, xs, wq, ws, None, [0, 4, 4, 30, M], torch.float32)
    # group 0 has rows 0..9 and group 2 rows 4..29: rows 4..9 are either's
    sure = np.r_[0:4, 10:M]
    within(cpu64(out)[sure], want[sure], bound[sure], "out")
    assert (out[M] == 7).all()


def _hidden(kind, xq, xs, w1, s1, b1, w3, s3):
    """h in 64 bits and a bound on the kernel's error of it."""
    def lin(w, s, b):
        p = (cpu64(xq) @ cpu64(w).T) * cpu64(xs)[:, None] * cpu64(s)[None]
        return p + (0 if b is None else cpu64(b)[None]), 3.01 * U * np.abs(p) + 2 * U * np.abs(p + (0 if b is None else cpu64(b)[None]))

    a, ea = lin(w1, s1, b1)
    if kind == "gelu_mlp":
        phi = 0.5 * (1 + np.vectorize(math.erf)(a / math.sqrt(2)))
        # |gelu'| <= 1.13; z / sqrt 2, erf (2 steps), the sum and two products: less than 8 roundings of |a|
        return a * phi, 1.13 * ea + 8 * U * np.abs(a)
    b, eb = lin(w3, s3, None)
    sig = 1 / (1 + np.exp(-a))
    # d(a sig a)/da is at most 1.1; exp(-a): its argument times log2 e off by U |a| 1.45, the function by 2 steps;
    # the sum, the quotient (2 steps) and the product: less than (16 + 3 |a|) roundings of the result
    h = a * sig * b
    return h, 1.1 * ea * np.abs(b) + np.abs(a * sig) * eb + (16 + 3 * np.abs(a)) * U * np.abs(h) + 1e-37


def _ffn_ref(kind, xq, xs, off, w, dtype):
    """(value, bound) of the packed rows' FFN.  A hidden value within its error of a rounding tie may take either of the
    two neighbours; everything else is as in the product."""
    G = len(off) - 1
    if kind == "linear":
        v, bd, _ = _product(xq, xs, w["w1"], w["s1"], w.get("b1"), off, dtype)
        return v, bd
    M, Dout = xq.shape[0], w["w2"].shape[1]
    want, bound = np.zeros((M, Dout)), np.zeros((M, Dout))
    for g in range(G):
        a, b = int(off[g]), int(off[g + 1])
        if a >= b:
            continue
        h, e = _hidden(kind, xq[a:b], xs[a:b], w["w1"][g], w["s1"][g], None if w.get("b1") is None else w["b1"][g],
                       None if kind != "swiglu" else w["w3"][g], None if kind != "swiglu" else w["s3"][g])
        m = np.abs(h).max(1, keepdims=True)
        em = e[np.arange(len(h)), np.abs(h).argmax(1)][:, None] + e.max(1, keepdims=True)
        ok = m > 0
        ms = np.where(ok, m, 1.0)
        v = np.where(ok, 127 * h / ms, 0.0)
        ev = np.where(ok, 127 * (e / ms + np.abs(h) / ms * em / ms) * 1.01, 0.0)
        q = np.rint(v)
        near = np.abs(np.abs(v - q) - 0.5) <= ev  # may round to either side
        w2 = cpu64(w["w2"][g])
        scale = (m / 127) * cpu64(w["s2"][g])[None]
        p = (q @ w2.T) * scale
        flip = (near.astype(np.float64) @ np.abs(w2).T) * scale
        err = flip + (4.01 * U + em / ms * 1.01) * (np.abs(p) + flip)
        val = p if w.get("b2") is None else p + cpu64(w["b2"][g])[None]
        err = err + U * np.abs(val)
        want[a:b] = val
        bound[a:b] = err + (HALF[dtype] * (np.abs(val) + err) if dtype == torch.bfloat16 else 0)
    return want, bound


def _weights(kind, G, D, F, Dout, seed):
    g = torch.Generator().manual_seed(seed)

    def w(n, k):
        q, s = ref_quantize(torch.randn(G, n, k, generator=g).double().numpy())
        return torch.from_numpy(q).to(torch.int8), torch.from_numpy(s).float() * 0.3

    o = {}
    if kind == "linear":
        o["w1"], o["s1"] = w(Dout, D)
        o["b1"] = torch.randn(G, Dout, generator=g)
        return o
    o["w1"], o["s1"] = w(F, D)
    o["w2"], o["s2"] = w(Dout, F)
    if kind == "swiglu":
        o["w3"], o["s3"] = w(F, D)
    else:
        o["b1"], o["b2"] = torch.randn(G, F, generator=g), torch.randn(G, Dout, generator=g)
    return o


@pytest.mark.parametrize("kind", ["swiglu", "gelu_mlp", "linear"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,D,F,Dout", [([1], 16, 16, 16), ([0, 3, 0, 40, 1], 72, 40, 33), ([270, 0, 129], 256, 512, 300),
                                             ([20, 60], 130, 1100, 64), ([5, 0, 300], 64, 257, 17), ([7, 9], 33, 1, 5)])
def test_ffn(kind, dtype, counts, D, F, Dout):
    G = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1])
    x = torch.randn(M, D, generator=torch.Generator().manual_seed(M))
    q, s = ref_quantize(x.double().numpy())
    xq, xs = torch.from_numpy(q).to(torch.int8), torch.from_numpy(s).float()
    w = _weights(kind, G, D, F, Dout, D)
    want, bound = _ffn_ref(kind, xq, xs, off, w, dtype)
    ys = torch.full((M + 2, Dout), 7.0, dtype=dtype, device=DEV)
    status = moe.new_status(DEV)
    pad = lambda t: torch.cat([t, t[:1].expand(2, *t.shape[1:])])  # noqa: E731  two rows behind the last group
    moe.moe_expert_ffn_i8(kind, _dev(pad(xq)), pad(xs).to(DEV), torch.from_numpy(off.astype(np.int32)).to(DEV),
                          ys=ys, dev_status=status, **{n: _dev(t) for n, t in w.items()})
    within(cpu64(ys)[:M], want, bound, "ys")
    assert (ys[M:] == 7).all() and moe.moe_read_status(status) == 0


def test_ffn_dense_and_without_rows():
    w = {n: _dev(t) for n, t in _weights("swiglu", 1, 64, 48, 32, 1).items()}
    x = torch.randn(70, 64, device=DEV)
    q, s = moe.moe_quantize_i8(x)
    a = moe.moe_expert_ffn_i8("swiglu", q, s, None, **w)
    b = moe.moe_expert_ffn_i8("swiglu", q, s, torch.tensor([0, 70], dtype=torch.int32, device=DEV), **w)
    assert torch.equal(a, b)
    e = moe.moe_expert_ffn_i8("swiglu", q[:0], s[:0], None, **w)
    assert e.shape == (0, 32)
    z = moe.moe_expert_ffn_i8("swiglu", torch.zeros_like(q), s, None, **w)
    assert (z == 0).all()  # hidden rows of zeros


def test_tokens_that_are_not_finite_stay_alone():
    w = {n: _dev(t) for n, t in _weights("swiglu", 1, 64, 48, 32, 1).items()}
    x = torch.randn(70, 64, device=DEV)
    clean = moe.moe_expert_ffn_i8("swiglu", *moe.moe_quantize_i8(x), None, **w)
    x[33, 5] = float("nan")
    status = moe.new_status(DEV)
    got = moe.moe_expert_ffn_i8("swiglu", *moe.moe_quantize_i8(x, dev_status=status), None, dev_status=status, **w)
    assert moe.moe_read_status(status) == B.MOE_ERR_NONFINITE
    keep = [i for i in range(70) if i != 33]
    assert torch.isnan(got[33]).all() and torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("T,k,E,H,F", [(1, 1, 4, 64, 32), (50, 4, 16, 136, 72), (700, 8, 32, 256, 128)])
def test_run_together(T, k, E, H, F):
    """route -> sort_i8 -> expert_ffn_i8 -> unsort, as a serving layer runs them."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    wr = torch.randn(E, H, generator=g).to(torch.bfloat16)
    w = _weights("swiglu", E, H, F, H, 9)
    wd = {n: _dev(t) for n, t in w.items()}
    status = moe.new_status(DEV)
    r = moe.moe_route(x.to(DEV), k, w_router=wr.to(DEV), dev_status=status)
    s = moe.moe_sort_i8(r["selected"], E, x.to(DEV), dev_status=status)
    ys = moe.moe_expert_ffn_i8("swiglu", s["xq"], s["xscale"], s["offsets"], out_dtype=torch.float32, dev_status=status, **wd)
    y = moe.moe_unsort(ys, s["row"], r["gates_f32"], dev_status=status)
    assert moe.moe_read_status(status) == 0
    off, row, src = ref_sort(r["selected"].cpu().numpy(), E)
    q, sc = ref_quantize(cpu64(x))
    xq, xs = torch.from_numpy(q[src // k]).to(torch.int8), torch.from_numpy(sc[src // k]).float()
    want_ys, bound = _ffn_ref("swiglu", xq, xs, off, w, torch.float32)
    within(cpu64(ys), want_ys, bound, "ys")
    gates = cpu64(r["gates_f32"])
    want = (gates[..., None] * want_ys[row]).sum(1)
    mag = (gates[..., None] * (np.abs(want_ys) + bound)[row]).sum(1)
    within(cpu64(y), want, (gates[..., None] * bound[row]).sum(1) + (k + 1) * U * mag, "y")


def test_streams_and_graphs():
    T, k, E, H, F = 200, 4, 16, 128, 96
    rng = np.random.default_rng(1)
    wd = {n: _dev(t) for n, t in _weights("swiglu", E, H, F, H, 9).items()}
    sels = [torch.from_numpy(routing(rng, T, k, E, dropped=0.1)).to(DEV) for _ in range(3)]
    xs = [torch.randn(T, H, device=DEV).to(torch.bfloat16) for _ in range(3)]
    gates = torch.rand(T, k, device=DEV)

    def step(sel, x, stream=None):
        s = moe.moe_sort_i8(sel, E, x, stream=stream)
        ys = moe.moe_expert_ffn_i8("swiglu", s["xq"], s["xscale"], s["offsets"], stream=stream, **wd)
        return moe.moe_unsort(ys, s["row"], gates, stream=stream)

    want = [step(s, x) for s, x in zip(sels, xs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(sels[0], xs[0], stream=side)
    also = step(sels[1], xs[1])  # at the same time on the current stream
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0]) and torch.equal(also, want[1])
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
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
