"""The sorted rows and the 8-bit products at calls that are allowed and rare: scales far apart, offsets that run backwards, and
tensors that are given up while another stream still works on them."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_stable_b200 as moe
from sparse_mixture_experts_stable_b200 import binding as B
from sparse_mixture_experts_stable_b200.layer import SwiGLUMoEInt8
from tests.gpu_util import DEV, cpu, cpu64
from tests.sorted_util import ref_quantize, ref_sort, routing, within
from tests.test_gpu_i8 import _dev, _i8, _product, _scale

pytestmark = pytest.mark.gpu


# 8 rows: the few-row kernel; 2100: tiles
@pytest.mark.parametrize("M", [8, 2100])
def test_scales_far_apart(M):
    """Results in the normal range of fp32 although the two scales' product is not (or is subnormal)."""
    K, N = 200, 72
    xq, wq = _i8((M, K), 1), _i8((N, K), 2)
    xq[3] = 0
    # |sum| <= 200 128^2 < 3.3e6, so |out| < 7e37
    xs = torch.tensor([1e-37, 1e-30, 1.0, 1e30])[torch.arange(M) % 4]
    ws = torch.tensor([1e-3, 0.5, 20.0])[torch.arange(N) % 3]
    out = moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), out_dtype=torch.float32)
    want, bound, _ = _product(xq, xs, wq[None], ws[None], None, [0, M], torch.float32)
    assert torch.isfinite(out).all()
    # a subnormal result is off by half its step, 2^-150, besides
    within(cpu64(out), want, bound + 2.0 ** -149, "out")
    # a sum of zero stays zero where the scales' product overflows
    big = torch.full((M,), 1e25, device=DEV)
    zero = moe.moe_matmul_i8(_dev(torch.zeros_like(xq)), big, _dev(wq), torch.full((N,), 1e25, device=DEV))
    assert (zero == 0).all()


# 4 rows per group on average: the few-row kernel; 40: tiles
@pytest.mark.parametrize("M", [4 * 16, 40 * 16])
def test_offsets_that_run_backwards(M):
    """The largest offset so far counts: each row has one group, the same in every run."""
    K, N, G = 96, 40, 16
    xq, wq, xs, ws = _i8((M, K), 1), _i8((G, N, K), 2), _scale((M,), 3), _scale((G, N), 4)
    raw = np.array([2, M, 0, M // 2, -7] + [M // 4] * (G - 5) + [M])
    raw[1] = M // 2 + 5
    off = np.maximum.accumulate(np.clip(raw, 0, M))
    status = moe.new_status(DEV)
    out = torch.full((M, N), 7.0, device=DEV)
    moe.moe_matmul_i8(_dev(xq), xs.to(DEV), _dev(wq), ws.to(DEV), out=out, dev_status=status,
                      offsets=torch.from_numpy(raw.astype(np.int32)).to(DEV))
    assert moe.moe_read_status(status) == B.MOE_ERR_BAD_INDEX
    want, bound, written = _product(xq, xs, wq, ws, None, off, torch.float32)
    got = cpu64(out)
    within(got[written], want[written], bound[written], "out")
    assert (got[~written] == 7).all()


def test_tensors_given_up_while_another_stream_works():
    """Inputs that the caller drops after the call are not reused before the other stream is done with them."""
    side = torch.cuda.Stream()
    x = torch.randn(512, 1000, generator=torch.Generator().manual_seed(0)).to(DEV)
    sel = torch.arange(1024, device=DEV).reshape(512, 2) % 8
    q, s = moe.moe_quantize_i8(x)
    r = moe.moe_sort(sel, 8, x)
    y = moe.moe_unsort(r["xs"], r["row"])
    torch.cuda.synchronize()
    got = []
    for run in (lambda t: moe.moe_quantize_i8(t, stream=side)[0], lambda t: moe.moe_sort(sel, 8, t, stream=side)["xs"],
                lambda t: moe.moe_unsort(t, r["row"], stream=side)):
        t = (r["xs"] if len(got) == 2 else x).clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # some 10 ms
        size = t.shape
        got.append(run(t))
        del t
        again = torch.full(size, 9.0, device=DEV)  # would take the memory of t
        torch.cuda.synchronize()
        del again
    for a, b in zip(got, (q, r["xs"], y)):
        np.testing.assert_array_equal(cpu(a), cpu(b))


def test_expert_count_beyond_32_bits():
    sel = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    for E in (0, -1, (1 << 32) + 1):
        with pytest.raises(ValueError):
            moe.moe_sort(sel, E)


# where the kernels change over: rows of 4, 8, 16 and 32 steps of a warp (256 values of bf16, 128 of fp32), odd widths and
# unaligned rows, up to 64 experts per token, fewer and more rows than the teams
@pytest.mark.parametrize("dtype,step", [(torch.float32, 128), (torch.bfloat16, 256)])
@pytest.mark.parametrize("steps,more", [(4, 0), (4, 1), (8, 0), (8, 4), (16, 0), (16, 8), (32, 0), (32, 3)])
@pytest.mark.parametrize("T,k", [(4200, 1), (1400, 3), (70, 64), (2400, 2)])
def test_rows_in_8_bits_at_every_width(dtype, step, steps, more, T, k):
    D, E = step * steps + more, 24
    rng = np.random.default_rng(D + T)
    sel = routing(rng, T, k, E, dropped=0.05)
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(D)).to(dtype)
    x[5], x[6, 0] = 0, 100.0
    q, s = ref_quantize(cpu64(x))
    off, row, _ = ref_sort(sel, E)
    status = moe.new_status(DEV)
    got, gs = moe.moe_quantize_i8(x.to(DEV), dev_status=status)
    np.testing.assert_array_equal(cpu(got), q)
    np.testing.assert_array_equal(cpu(gs), s.astype(np.float32))
    r = moe.moe_sort_i8(torch.from_numpy(sel).to(DEV), E, x.to(DEV), dev_status=status)
    rows, scales = cpu(r["xq"]), cpu(r["xscale"])
    t, j = np.nonzero(row >= 0)
    np.testing.assert_array_equal(rows[row[t, j]], q[t])
    np.testing.assert_array_equal(scales[row[t, j]], s.astype(np.float32)[t])
    assert off[-1] == len(t) and moe.moe_read_status(status) == 0


def test_layer_captured_with_its_second_stream():
    T, H, E, F, k, Fs = 40, 256, 16, 128, 4, 96
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.1).to(torch.bfloat16).to(DEV)  # noqa: E731
    xs = [torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3)]
    wr, bias = mk(E, H), torch.randn(E, generator=g).to(DEV)
    experts = SwiGLUMoEInt8.quantize(mk(E, F, H), mk(E, F, H), mk(E, H, F))
    shared = SwiGLUMoEInt8.quantize(mk(1, Fs, H), mk(1, Fs, H), mk(1, H, Fs))
    layer = SwiGLUMoEInt8(T, H, E, F, k, F_shared=Fs)
    want = [layer.forward(x, wr, bias, experts, shared)["y"].clone() for x in xs]
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x, wr, bias, experts, shared)["y"]
    for i in (1, 2, 0):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(y, want[i])
    assert moe.moe_read_status(layer.status) == 0
