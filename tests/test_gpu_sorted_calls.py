"""The sorted rows and the 8-bit products: types, padding, full experts and rows that are not finite, at every kernel that a
call can reach."""
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

BF16, F32 = torch.bfloat16, torch.float32


# k: each number of rows taken together; N: 16-byte vectors, one value, both ends of a warp's steps
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (40, 2, 7), (33, 2, 2048), (600, 4, 132), (300, 17, 264), (700, 8, 1024), (20, 64, 1001)])
@pytest.mark.parametrize("gates", [None, F32, BF16])
@pytest.mark.parametrize("base", [None, F32, BF16])
def test_unsort_of_fp32_rows_into_bf16(T, k, N, gates, base):
    """The sum is rounded once, whatever the base's type."""
    rng = np.random.default_rng(T + N)
    _, row, src = ref_sort(routing(rng, T, k, 24, dropped=0.2), 24)
    R = max(int((src >= 0).sum()), 1)
    ys = torch.randn(R, N, generator=torch.Generator().manual_seed(N))
    g = None if gates is None else torch.from_numpy(rng.uniform(0, 1, (T, k)).astype(np.float32)).to(gates)
    b = None if base is None else torch.randn(T, N, generator=torch.Generator().manual_seed(T)).to(base)
    want, mag = ref_unsort(cpu64(ys), row, None if g is None else cpu64(g), None if b is None else cpu64(b), N)
    sums = k * U * mag * 1.001  # k fused multiply-adds in fp32, each off by U of a partial sum that is at most mag
    bound = sums + HALF[BF16] * (np.abs(want) + sums)
    args = ys.to(DEV), torch.from_numpy(row.astype(np.int32)).to(DEV), None if g is None else g.to(DEV)
    b = None if b is None else b.to(DEV)
    y = moe.moe_unsort(*args, base=b, out_dtype=BF16)
    assert y.dtype is BF16
    within(cpu64(y), want, bound, "y")
    # rows of wider matrices, on 4 and on 2 bytes
    wide = torch.full((T, N + 5), 9.0, dtype=BF16, device=DEV)
    odd = torch.full((R, N + 3), 7.0, device=DEV)
    odd[:, 1:N + 1] = args[0]
    moe.moe_unsort(odd[:, 1:N + 1], *args[1:], base=b, y=wide[:, 1:N + 1])
    assert torch.equal(wide[:, 1:N + 1], y) and (wide[:, 0] == 9).all() and (wide[:, N + 1:] == 9).all()


def test_unsort_of_fp32_rows_into_bf16_on_a_stream_and_in_a_graph():
    row = torch.arange(80, dtype=torch.int32, device=DEV).view(20, 4)
    ys, base = torch.randn(80, 136, device=DEV), torch.randn(20, 136, device=DEV).to(BF16)
    want = moe.moe_unsort(ys, row, base=base, out_dtype=BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_unsort(ys, row, base=base, out_dtype=BF16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    src = torch.zeros_like(ys)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = moe.moe_unsort(src, row, base=base, out_dtype=BF16)
    src.copy_(ys)
    graph.replay()
    assert torch.equal(y, want)


def test_types_that_unsort_refuses():
    row = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    f, h = torch.zeros(4, 16, device=DEV), torch.zeros(4, 16, dtype=BF16, device=DEV)
    for call in (lambda: moe.moe_unsort(h, row, out_dtype=F32), lambda: moe.moe_unsort(h, row, y=f),
                 lambda: moe.moe_unsort(h, row, base=f), lambda: moe.moe_unsort(f, row, base=h),
                 lambda: moe.moe_unsort(f, row, y=h, out_dtype=F32), lambda: moe.moe_unsort(f, row, out_dtype=torch.float16),
                 lambda: moe.moe_unsort(f, row, y=f.half()), lambda: moe.moe_unsort(f, row, base=[0]),
                 lambda: moe.moe_unsort(f, row, y=h[:3])):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(ValueError):
        SwiGLUMoEInt8(4, 16, 4, 16, 1, dtype=F32, rows_dtype=BF16)


@pytest.mark.parametrize("T,H,E,F,k,Fs", [(1, 64, 8, 32, 2, 0), (33, 136, 16, 40, 4, 56), (700, 256, 32, 128, 8, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_rounds_once(T, H, E, F, k, Fs, dtype):
    """The experts' and the shared expert's rows reach the sum unrounded."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(dtype).to(DEV)
    wr, bias = torch.randn(E, H, generator=g).to(dtype).to(DEV), torch.randn(E, generator=g).to(DEV)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.1).to(dtype).to(DEV)  # noqa: E731
    experts = SwiGLUMoEInt8.quantize(mk(E, F, H), mk(E, F, H), mk(E, H, F))
    shared = SwiGLUMoEInt8.quantize(mk(1, Fs, H), mk(1, Fs, H), mk(1, H, Fs)) if Fs else None
    layer = SwiGLUMoEInt8(T, H, E, F, k, F_shared=Fs, dtype=dtype)
    for _ in range(2):  # the buffers are used again
        o = layer.forward(x, wr, bias, experts, shared)
    assert moe.moe_read_status(layer.status) == 0 and o["y"].dtype is dtype
    off, row, src = ref_sort(cpu(o["selected"]), E)
    q, sc = ref_quantize(cpu64(x))
    q, sc = torch.from_numpy(q).to(torch.int8), torch.from_numpy(sc).float()
    to = lambda d: {n: t.cpu() for n, t in d.items()}  # noqa: E731
    ys, bound = _ffn_ref("swiglu", q[src // k], sc[src // k], off, to(experts), F32)
    gates = cpu64(o["gates_f32"])[..., None]
    want, mag, err = (gates * ys[row]).sum(1), (gates * (np.abs(ys) + bound)[row]).sum(1), (gates * bound[row]).sum(1)
    if Fs:
        b, eb = _ffn_ref("swiglu", q, sc, [0, T], to(shared), F32)
        want, mag, err = want + b, mag + np.abs(b) + eb, err + eb
    err = err + (k + 1) * U * mag
    within(cpu64(o["y"]), want, err + HALF[dtype] * (np.abs(want) + err), "y")


# (T, k, D in steps of a warp, columns before xq): one launch with few and many tokens per block, teams of 1, 2 and 4 warps,
# rows in shared memory (one segment, two), a warp per token for rows off their boundary
ROW_KERNELS = [(40, 3, 2.5, 0), (3000, 1, 2.5, 0), (3000, 3, 2.5, 0), (3000, 3, 7, 0), (3000, 3, 13, 0), (1500, 3, 30.5, 0),
               (1400, 3, 70.5, 0), (3000, 3, 18.25, 3)]


def _sort_i8_at(sel, E, x, skip, status):
    """moe_sort_i8 into rows that begin `skip` bytes after a boundary."""
    T, D = x.shape
    if not skip:
        return moe.moe_sort_i8(sel, E, x, dev_status=status)
    xq = torch.full((sel.numel(), D + 2 * skip), 77, dtype=torch.int8, device=DEV)[:, skip:skip + D]
    return moe.moe_sort_i8(sel, E, x, out=dict(xq=xq), dev_status=status)


@pytest.mark.parametrize("T,k,steps,skip", ROW_KERNELS)
@pytest.mark.parametrize("dtype,step", [(F32, 128), (BF16, 256)])
def test_padding_tokens_may_hold_anything(T, k, steps, skip, dtype, step):
    """Tokens of which no choice takes part: no status, and the others' rows as without them."""
    D, E = int(steps * step), 24
    sel = routing(np.random.default_rng(T + D), T, k, E)
    pads = [0, 7, T // 2, T - 1]
    sel[pads] = -1
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(D)).to(dtype)
    q, s = ref_quantize(cpu64(x))
    x[pads[0]], x[pads[1], D - 1], x[pads[2], D // 2], x[pads[3], 0] = float("nan"), float("inf"), float("nan"), -float("inf")
    _, row, _ = ref_sort(sel, E)
    status = moe.new_status(DEV)
    r = _sort_i8_at(torch.from_numpy(sel).to(DEV), E, x.to(DEV), skip, status)
    t, j = np.nonzero(row >= 0)
    np.testing.assert_array_equal(cpu(r["xq"])[row[t, j]], q[t])
    np.testing.assert_array_equal(cpu(r["xscale"])[row[t, j]], s.astype(np.float32)[t])
    assert moe.moe_read_status(status) == 0
    sel[pads[2], k - 1] = 5  # one choice is enough
    _sort_i8_at(torch.from_numpy(sel).to(DEV), E, x.to(DEV), skip, status)
    assert moe.moe_read_status(status) == B.MOE_ERR_NONFINITE


@pytest.mark.parametrize("K", [16, 300])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_thousands_of_short_tiles(K, dtype):
    """One and three steps of the depth per tile: the tiles' queue is filled and emptied as fast as it can be, and no tile is
    taken twice or for another."""
    G, N = 700, 520
    gen = torch.Generator(device=DEV).manual_seed(K)
    counts = torch.randint(0, 60, (G,), device=DEV, generator=gen)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    M = int(off[-1])
    assert M > 8 * G  # tiles, not the few-row kernel
    pad = -(-K // 16) * 16
    xq = torch.randint(-128, 128, (M, pad), device=DEV, generator=gen).to(torch.int8)[:, :K]
    wq = torch.randint(-128, 128, (G, N, pad), device=DEV, generator=gen).to(torch.int8)[..., :K]
    one = torch.ones(G * max(M, N), device=DEV)
    want = torch.cat([xq[off[g]:off[g + 1]].double() @ wq[g].double().T for g in range(G)])
    assert want.abs().max() < 2 ** 24  # exact in fp32
    want = want.to(dtype)
    for _ in range(20):
        out = moe.moe_matmul_i8(xq, one[:M], wq, one[:G * N].view(G, N), offsets=off.int(), out_dtype=dtype)
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["swiglu", "gelu_mlp"])
def test_groups_of_every_number_of_rows(kind):
    """Tiles whose tokens end at every place of the warps that share them; for SwiGLU two warps exchange gate and up."""
    counts = list(range(70)) + [127, 128, 129, 191, 193, 250, 255, 256, 257, 319, 321, 383, 385, 511, 513]
    G, D, F, Dout = len(counts), 48, 200, 40
    off = np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1])
    assert M > 8 * G  # tiles, not the few-row kernel
    q, s = ref_quantize(torch.randn(M, D, generator=torch.Generator().manual_seed(M)).double().numpy())
    xq, xs = torch.from_numpy(q).to(torch.int8), torch.from_numpy(s).float()
    w = _weights(kind, G, D, F, Dout, D)
    want, bound = _ffn_ref(kind, xq, xs, off, w, F32)
    status = moe.new_status(DEV)
    args = _dev(xq), xs.to(DEV), torch.from_numpy(off.astype(np.int32)).to(DEV)
    wd = {n: _dev(t) for n, t in w.items()}
    ys = moe.moe_expert_ffn_i8(kind, *args, out_dtype=F32, dev_status=status, **wd)
    within(cpu64(ys), want, bound, "ys")
    assert moe.moe_read_status(status) == 0
    for _ in range(10):
        assert torch.equal(moe.moe_expert_ffn_i8(kind, *args, out_dtype=F32, **wd), ys)


@pytest.mark.parametrize("given", [False, True])
def test_entries_of_out_that_are_no_cuda_tensors(given):
    """With a stream as without: an entry that the call does not know stays as it is, a wrong one is refused."""
    stream = torch.cuda.Stream() if given else None
    sel, x = torch.arange(12, device=DEV).reshape(6, 2) % 4, torch.randn(6, 32, device=DEV)
    torch.cuda.synchronize()
    for call, name in ((moe.moe_sort, "xs"), (moe.moe_sort_i8, "xq")):
        r = call(sel, 4, x, out=dict(note="kept", nothing=None), stream=stream)
        torch.cuda.synchronize()
        assert r["note"] == "kept" and r["nothing"] is None and torch.equal(r[name], call(sel, 4, x)[name])
        for bad in (5, "offsets", torch.zeros(5, dtype=torch.int32), torch.zeros(5, device=DEV)):
            with pytest.raises((ValueError, TypeError)):
                call(sel, 4, x, out=dict(offsets=bad), stream=stream)
        for bad in (5, torch.zeros(12, 32), torch.zeros(12, 32, dtype=torch.float64, device=DEV)):
            with pytest.raises((ValueError, TypeError)):
                call(sel, 4, x, out={name: bad}, stream=stream)


# 8 rows: the few-row kernel; 2100: tiles
@pytest.mark.parametrize("M", [8, 2100])
def test_swiglu_where_the_sigmoid_saturates(M):
    """Gates from -300 to 300: exp(-gate) from 0 to beyond fp32."""
    D, F, Dout = 32, 200, 24
    g = torch.Generator().manual_seed(M)
    xq = torch.randint(-127, 128, (M, D), generator=g, dtype=torch.int8)
    xs = torch.full((M,), 1 / 127)
    w = _weights("swiglu", 1, D, F, Dout, 3)
    # row f of the gate: +-127 at one place, scaled so that the gate runs from 0 to 300 in size
    w["w1"] = torch.zeros(1, F, D, dtype=torch.int8)
    w["w1"][0, torch.arange(F), torch.arange(F) % D] = torch.where(torch.arange(F) % 3 == 0, 127, -127).to(torch.int8)
    w["s1"] = (torch.arange(F) * 1.5 / 127)[None]
    off = [0, M]
    want, bound = _ffn_ref("swiglu", xq, xs, off, w, F32)
    status = moe.new_status(DEV)
    ys = moe.moe_expert_ffn_i8("swiglu", _dev(xq), xs.to(DEV), None, out_dtype=F32, dev_status=status,
                               **{n: _dev(t) for n, t in w.items()})
    assert moe.moe_read_status(status) == 0 and torch.isfinite(ys).all()
    within(cpu64(ys), want, bound, "ys")


# 1024 rows in 256 groups: 4 on average, so the few-row kernel takes them, whatever their distribution; at a real size
@pytest.mark.parametrize("full", [1024, 512, 17])
@pytest.mark.parametrize("N,K", [(2048, 512), (512, 2048)])
def test_one_very_full_expert_in_the_few_row_kernel(full, N, K):
    G, M = 256, 1024
    gen = torch.Generator(device=DEV).manual_seed(full)
    counts = torch.bincount(torch.randint(0, G, (M - full,), device=DEV, generator=gen), minlength=G)
    counts[77] += full
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    xq = torch.randint(-128, 128, (M, K), device=DEV, generator=gen).to(torch.int8)
    wq = torch.randint(-128, 128, (G, N, K), device=DEV, generator=gen).to(torch.int8)
    xs, ws = (torch.rand(n, device=DEV, generator=gen) + 0.5 for n in (M, G * N))
    out = moe.moe_matmul_i8(xq, xs, wq, ws.view(G, N), offsets=off.int(), out_dtype=F32)
    for g in counts.nonzero().flatten().tolist():
        a, b = int(off[g]), int(off[g + 1])
        want = (xq[a:b].double() @ wq[g].double().T) * xs[a:b, None].double() * ws.view(G, N)[g].double()
        assert ((out[a:b].double() - want).abs() <= 3.01 * U * want.abs()).all()  # to fp32, and the two scales


def _not_finite(D, dtype):
    """(column, value): infinities and NaNs of both signs, with the smallest and the largest payload, over the row's ends."""
    bits = torch.tensor([0x7f800000, -0x800000, 0x7f800001 if dtype is F32 else 0x7f810000, -1], dtype=torch.int32)
    return list(zip([0, D - 1, D // 2, D - 1], bits.view(F32).to(dtype) if dtype is F32 else
                    (bits >> 16).to(torch.int16).view(BF16)))


def _check_not_finite(x, bad):
    """x's rows bad[i] get the values; returns what each row must be."""
    D = x.shape[1]
    q, s = ref_quantize(cpu64(x))
    for i, (col, v) in zip(bad, _not_finite(D, x.dtype)):
        x[i, col] = v
        q[i], s[i] = 0, np.nan
    assert not torch.isfinite(x[bad].float()).all(1).any()
    return q, s.astype(np.float32)


# teams of 1, 2, 4 and 8 warps, a block per row: few rows of a team's width, and wider ones
@pytest.mark.parametrize("M,steps", [(1300, 3.5), (1300, 7), (700, 13.25), (400, 30.5), (40, 30.5), (400, 41)])
@pytest.mark.parametrize("dtype,step", [(F32, 128), (BF16, 256)])
def test_quantize_reports_rows_that_are_not_finite_at_every_width(M, steps, dtype, step):
    x = torch.randn(M, int(steps * step), generator=torch.Generator().manual_seed(M)).to(dtype)
    q, s = _check_not_finite(x, [3, M // 2, M - 2, M - 1])
    status = moe.new_status(DEV)
    got, scale = moe.moe_quantize_i8(x.to(DEV), dev_status=status)
    assert moe.moe_read_status(status) == B.MOE_ERR_NONFINITE
    np.testing.assert_array_equal(cpu(got), q)
    np.testing.assert_array_equal(cpu(scale), s)


@pytest.mark.parametrize("T,k,steps,skip", ROW_KERNELS)
@pytest.mark.parametrize("dtype,step", [(F32, 128), (BF16, 256)])
def test_sort_i8_reports_rows_that_are_not_finite_at_every_width(T, k, steps, skip, dtype, step):
    D, E = int(steps * step), 24
    sel = routing(np.random.default_rng(T + D), T, k, E)
    _, row, _ = ref_sort(sel, E)
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(D)).to(dtype)
    q, s = _check_not_finite(x, [3, T // 2, T - 2, T - 1])
    status = moe.new_status(DEV)
    r = _sort_i8_at(torch.from_numpy(sel).to(DEV), E, x.to(DEV), skip, status)
    assert moe.moe_read_status(status) == B.MOE_ERR_NONFINITE
    t, j = np.nonzero(row >= 0)
    np.testing.assert_array_equal(cpu(r["xq"])[row[t, j]], q[t])
    np.testing.assert_array_equal(cpu(r["xscale"])[row[t, j]], s[t])


# 12 rows per group on average: tiles; 4: the few-row kernel
@pytest.mark.parametrize("G", [4, 12])
def test_every_row_under_offsets_that_run_backwards(G):
    """The rows that two groups claim belong to the first, as the running maximum of the offsets says."""
    M, K, N = 50, 64, 40
    xq, wq, xs, ws = _i8((M, K), 1), _i8((G, N, K), 2), _scale((M,), 3), _scale((G, N), 4)
    raw = [-5, 10, 4, 30] + [2 ** 31 - 1] * (G - 3)
    status = moe.new_status(DEV)
    out = torch.full((M + 1, N), 7.0, device=DEV)
    moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), out=out[:M], dev_status=status,
                      offsets=torch.tensor(raw, dtype=torch.int32, device=DEV))
    assert moe.moe_read_status(status) == B.MOE_ERR_BAD_INDEX
    want, bound, written = _product(xq, xs, wq, ws, None, [0, 10, 10, 30] + [M] * (G - 3), F32)
    assert written.all()
    within(cpu64(out)[:M], want, bound, "out")
    assert (out[M] == 7).all()


def test_layer_biases():
    """No router bias, and E values of any shape."""
    T, H, E, F = 9, 64, 8, 32
    g = torch.Generator().manual_seed(2)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.1).to(BF16).to(DEV)  # noqa: E731
    x, wr, experts = mk(T, H), mk(E, H), SwiGLUMoEInt8.quantize(mk(E, F, H), mk(E, F, H), mk(E, H, F))
    layer = SwiGLUMoEInt8(T, H, E, F, 2)
    run = lambda bias: layer.forward(x, wr, bias, experts)["y"].clone()  # noqa: E731
    bias = torch.randn(E, device=DEV)
    assert torch.equal(run(None), run(torch.zeros(E, device=DEV)))
    assert torch.equal(run(bias), run(bias[None]))
    for bad in (bias[:3], bias.cpu()):
        with pytest.raises(ValueError):
            run(bad)
    assert moe.moe_read_status(layer.status) == 0
