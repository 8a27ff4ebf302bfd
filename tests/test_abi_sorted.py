"""Refusals of the sorted-row and 8-bit entry points, on the CPU: no kernel is launched, no pointer is read."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_stable_b200 as moe
from sparse_mixture_experts_stable_b200 import binding as B

P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4104)
N = None


def sort(L, sel=P, T=8, k=2, E=4, x=P, dt=1, D=16, ldx=16, off=P, row=P, src=P, xs=P, ldxs=16, ws=P, nb=1 << 20):
    return L.moe_sort(sel, T, k, E, x, dt, D, ldx, off, row, src, xs, ldxs, N, ws, nb, N)


def sort_i8(L, sel=P, T=8, k=2, E=4, x=P, dt=1, D=16, ldx=16, off=P, row=P, src=P, xq=P, ldq=16, xs=P, ws=P, nb=1 << 20):
    return L.moe_sort_i8(sel, T, k, E, x, dt, D, ldx, off, row, src, xq, ldq, xs, N, ws, nb, N)


def unsort(L, ys=P, ldys=16, rows=16, row=P, g=P, gdt=0, T=8, k=2, n=16, base=N, ldb=0, y=P, ldy=16, dt=1):
    return L.moe_unsort(ys, ldys, rows, row, g, gdt, T, k, n, base, ldb, y, ldy, dt, N, N)


def back(L, dy=P, lddy=16, ys=P, ldys=16, rows=16, row=P, g=P, gdt=0, T=8, k=2, n=16, dys=P, lddys=16, dg=P, dt=1):
    return L.moe_unsort_backward(dy, lddy, ys, ldys, rows, row, g, gdt, T, k, n, dys, lddys, dg, dt, N, N)


def quant(L, x=P, dt=1, M=4, K=16, ldx=16, q=P, ldq=16, s=P):
    return L.moe_quantize_i8(x, dt, M, K, ldx, q, ldq, s, N, N)


def matmul(L, xq=P, xs=P, M=4, ldx=16, off=N, wq=P, ws=P, ldw=16, b=N, G=1, n=8, K=16, out=P, ldo=8, dt=1, wk=P, nb=256):
    return L.moe_matmul_i8(xq, xs, M, ldx, off, wq, ws, ldw, b, G, n, K, out, ldo, dt, N, wk, nb, N)


def ffn(L, kind=2, xq=P, xs=P, M=4, ldx=16, off=P, G=3, D=16, F=16, Do=16, w1=P, s1=P, ld1=16, b1=N, w2=P, s2=P, ld2=16,
        b2=N, w3=P, s3=P, ys=P, ldy=16, dt=1, ws=P, nb=1 << 20):
    return L.moe_expert_ffn_i8(kind, xq, xs, M, ldx, off, G, D, F, Do, w1, s1, ld1, b1, w2, s2, ld2, b2, w3, s3, ys, ldy, dt,
                               N, ws, nb, N)


BAD, NO, WS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("call,args,code", [
    (sort, dict(T=-1), BAD), (sort, dict(k=0), BAD), (sort, dict(E=0), BAD), (sort, dict(sel=N), BAD),
    (sort, dict(off=N), BAD), (sort, dict(row=N), BAD), (sort, dict(src=N), BAD), (sort, dict(xs=N), BAD),
    (sort, dict(D=0), BAD), (sort, dict(ldx=15), BAD), (sort, dict(ldxs=15), BAD), (sort, dict(dt=2), BAD),
    (sort, dict(k=65), NO), (sort, dict(E=2049), NO), (sort, dict(T=1 << 30), NO), (sort, dict(T=1 << 29, k=2), NO),
    (sort, dict(T=5000, ws=N), WS), (sort, dict(T=5000, nb=8), WS),
    (sort_i8, dict(x=N), BAD), (sort_i8, dict(xq=N), BAD), (sort_i8, dict(xs=N), BAD), (sort_i8, dict(D=0), BAD),
    (sort_i8, dict(ldq=15), BAD), (sort_i8, dict(dt=-1), BAD), (sort_i8, dict(E=2049), NO), (sort_i8, dict(T=5000, nb=8), WS),
    (unsort, dict(dt=3), BAD), (unsort, dict(gdt=3), BAD), (unsort, dict(T=-1), BAD), (unsort, dict(n=0), BAD),
    (unsort, dict(k=0), BAD), (unsort, dict(ldys=15), BAD), (unsort, dict(ldy=15), BAD), (unsort, dict(row=N), BAD),
    (unsort, dict(y=N), BAD), (unsort, dict(ys=N), BAD), (unsort, dict(rows=-1), BAD), (unsort, dict(base=P, ldb=15), BAD),
    (unsort, dict(k=65), NO), (unsort, dict(T=1 << 29, k=2), NO),
    (back, dict(dt=3), BAD), (back, dict(dy=N), BAD), (back, dict(row=N), BAD), (back, dict(ys=N), BAD),
    (back, dict(ldys=15), BAD), (back, dict(lddys=15), BAD), (back, dict(lddy=15), BAD), (back, dict(k=65), NO),
    (quant, dict(dt=2), BAD), (quant, dict(K=0), BAD), (quant, dict(ldx=15), BAD), (quant, dict(ldq=15), BAD),
    (quant, dict(x=N), BAD), (quant, dict(q=N), BAD), (quant, dict(s=N), BAD), (quant, dict(M=-1), BAD),
    (quant, dict(M=1 << 31), NO),
    (matmul, dict(xq=N), BAD), (matmul, dict(xs=N), BAD), (matmul, dict(wq=N), BAD), (matmul, dict(ws=N), BAD),
    (matmul, dict(out=N), BAD), (matmul, dict(K=0), BAD), (matmul, dict(n=0), BAD), (matmul, dict(ldx=15), BAD),
    (matmul, dict(ldo=7), BAD), (matmul, dict(dt=5), BAD), (matmul, dict(G=2), BAD), (matmul, dict(M=-1), BAD),
    (matmul, dict(xq=ODD), NO), (matmul, dict(wq=ODD), NO), (matmul, dict(ldx=24), NO), (matmul, dict(ldw=24), NO),
    (matmul, dict(K=131072, ldx=131072, ldw=131072), NO), (matmul, dict(G=2049, off=P), NO),
    (matmul, dict(G=16, off=P, M=4096, wk=N), WS), (matmul, dict(G=16, off=P, M=4096, nb=255), WS),
    (ffn, dict(kind=3), BAD), (ffn, dict(G=0), BAD), (ffn, dict(F=0), BAD), (ffn, dict(Do=0), BAD), (ffn, dict(ys=N), BAD),
    (ffn, dict(w2=N), BAD), (ffn, dict(s2=N), BAD), (ffn, dict(w3=N), BAD), (ffn, dict(s3=N), BAD), (ffn, dict(b1=P), BAD),
    (ffn, dict(ld2=15), BAD), (ffn, dict(ldy=15), BAD), (ffn, dict(dt=9), BAD), (ffn, dict(w2=ODD), NO),
    (ffn, dict(w3=ODD), NO), (ffn, dict(ld2=24), NO), (ffn, dict(F=131072, ld2=131072, nb=1 << 30), NO), (ffn, dict(ws=N), WS),
    (ffn, dict(nb=64), WS), (ffn, dict(off=N), BAD),
])
def test_refusals(call, args, code):
    assert call(moe.lib(), **args) == code


def test_nothing_to_do():
    L = moe.lib()
    assert unsort(L, T=0, row=N, y=N) == B.MOE_OK
    assert back(L, T=0, row=N, dy=N) == B.MOE_OK
    assert back(L, dys=N, dg=N) == B.MOE_OK
    assert quant(L, M=0, x=N, q=N, s=N) == B.MOE_OK
    assert matmul(L, M=0, xq=N, xs=N, out=N, wk=N, nb=0) == B.MOE_OK
    assert ffn(L, M=0, xq=N, xs=N, ys=N, ws=N, nb=0) == B.MOE_OK


def test_workspace_sizes():
    assert B.moe_sort_workspace_size(16, 8, 256) == 0 and B.moe_sort_workspace_size(16384, 8, 256) > 0
    assert B.moe_sort_workspace_size(0, 8, 256) == 0 and B.moe_sort_workspace_size(16384, 65, 256) == 0
    assert B.moe_matmul_i8_workspace_size(1, 1, 64, 64) == 0
    assert B.moe_matmul_i8_workspace_size(131072, 256, 64, 64) > 0
    big = B.moe_expert_ffn_i8_workspace_size("swiglu", 256, 131072, 2048, 512, 2048)
    assert big >= 131072 * 512 * 5 + 131072 * 4
    assert B.moe_expert_ffn_i8_workspace_size("linear", 256, 131072, 2048, 0, 2048) < 4096
    assert B.moe_expert_ffn_i8_workspace_size("swiglu", 256, 0, 2048, 512, 2048) == 0


def test_the_binding_takes_cuda_tensors_only():
    cpu = torch.zeros(4, 2, dtype=torch.int64)
    x = torch.zeros(4, 16)
    q = torch.zeros(4, 16, dtype=torch.int8)
    for call in (lambda: moe.moe_sort(cpu, 4, x), lambda: moe.moe_sort_i8(cpu, 4, x),
                 lambda: moe.moe_unsort(x, cpu.int()), lambda: moe.moe_unsort_backward(x, x, cpu.int()),
                 lambda: moe.moe_quantize_i8(x), lambda: moe.moe_matmul_i8(q, x[:, 0], q, x[:, 0]),
                 lambda: moe.moe_expert_ffn_i8("linear", q, x[:, 0], None, q, x[:, 0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        moe.moe_expert_ffn_i8("relu", q, x[:, 0], None, q, x[:, 0])


@pytest.mark.parametrize("call,args", [
    (sort, dict(T=5000, ws=ODD)), (sort_i8, dict(T=5000, ws=ODD)), (matmul, dict(G=16, off=P, M=4096, wk=ODD)),
    (ffn, dict(ws=ODD)), (ffn, dict(kind=0, M=4096, ws=ODD)),
])
def test_a_workspace_off_its_boundary(call, args):
    assert call(moe.lib(), **args) == WS
