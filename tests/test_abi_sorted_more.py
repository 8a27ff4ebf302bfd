"""More refusals of the sorted-row and 8-bit entry points, on the CPU: no kernel is launched, no pointer is read."""
import pytest
import torch

import sparse_mixture_experts_stable_b200 as moe
from sparse_mixture_experts_stable_b200 import binding as B
from sparse_mixture_experts_stable_b200.layer import SwiGLUMoEInt8
from tests.test_abi_sorted import BAD, NO, N, P, ffn, matmul


def unsort_ex(L, ys=P, ldys=16, rows=16, dt=0, row=P, g=P, gdt=0, T=8, k=2, n=16, base=N, ldb=0, bdt=0, y=P, ldy=16, ydt=1):
    return L.moe_unsort_ex(ys, ldys, rows, dt, row, g, gdt, T, k, n, base, ldb, bdt, y, ldy, ydt, N, N)


@pytest.mark.parametrize("args,code", [
    (dict(dt=2), BAD), (dict(gdt=2), BAD), (dict(bdt=2), BAD), (dict(ydt=2), BAD), (dict(T=-1), BAD), (dict(n=0), BAD),
    (dict(ys=N), BAD), (dict(row=N), BAD), (dict(y=N), BAD), (dict(ldys=15), BAD), (dict(ldy=15), BAD), (dict(k=65), NO),
    (dict(base=P, ldb=15), BAD), (dict(dt=1, ydt=0), NO), (dict(dt=1, ydt=1, base=P, ldb=16, bdt=0), NO),
    (dict(dt=0, ydt=0, base=P, ldb=16, bdt=1), NO), (dict(T=0, row=N, y=N), B.MOE_OK),
])
def test_unsort_ex(args, code):
    assert unsort_ex(moe.lib(), **args) == code


BIG = 1 << 60  # times 16 it is 0 in 64 bits


@pytest.mark.parametrize("call,args,code", [
    (ffn, dict(G=16, Do=BIG, ldy=BIG), NO), (ffn, dict(kind=1, w3=N, s3=N, G=16, Do=BIG, ldy=BIG), NO),
    (ffn, dict(kind=0, G=16, Do=BIG, ldy=BIG), NO), (ffn, dict(G=16, F=BIG, ld2=BIG), NO), (ffn, dict(M=1 << 30), NO),
    (ffn, dict(ld2=1 << 38), NO), (ffn, dict(ld1=1 << 38), NO), (ffn, dict(D=BIG, ldx=BIG, ld1=BIG), NO),
    (matmul, dict(n=BIG, ldo=BIG), NO), (matmul, dict(M=16, n=BIG, ldo=BIG), NO), (matmul, dict(G=16, off=P, n=BIG, ldo=BIG), NO),
    (matmul, dict(M=1 << 30), NO), (matmul, dict(M=16, K=BIG, ldx=BIG, ldw=BIG), NO),
])
def test_sizes_whose_products_leave_64_bits(call, args, code):
    assert call(moe.lib(), **args) == code


def test_workspace_sizes_beyond_the_limits():
    for kind in ("swiglu", "gelu_mlp", "linear"):
        assert B.moe_expert_ffn_i8_workspace_size(kind, 16, 4, 16, 16, BIG) == 0
        assert B.moe_expert_ffn_i8_workspace_size(kind, 16, 1 << 30, 16, 16, 16) == 0
    assert B.moe_expert_ffn_i8_workspace_size("swiglu", 16, 4, 16, BIG, 16) == 0
    assert B.moe_expert_ffn_i8_workspace_size("linear", 16, 4, 16, BIG, 16) > 0  # F is not used


def test_the_layer_takes_what_its_buffers_were_made_for():
    """The router writes T rows of x's type into the layer's buffers, so others are refused before it is called."""
    T, H, E = 6, 32, 4
    x, wr, b = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(E, H, dtype=torch.bfloat16), torch.zeros(E)
    layer = SwiGLUMoEInt8(T, H, E, 16, 2, device="cpu")
    for name, args in (("x", (x[:5], wr, b)), ("x", (x.repeat(2, 1), wr, b)), ("x", (x[:, :16], wr, b)), ("x", (x.float(), wr, b)),
                       ("x", (x.to("meta"), wr, b)), ("w_router", (x, wr.repeat(2, 1), b)), ("w_router", (x, wr.float(), b)),
                       ("w_router", (x, wr[:, :16], b)), ("router_bias", (x, wr, b[:3])), ("router_bias", (x, wr, b.to("meta")))):
        with pytest.raises(ValueError, match=f"^{name} must be"):
            layer.forward(*args, experts={})
    with pytest.raises(ValueError, match="shared expert"):
        SwiGLUMoEInt8(T, H, E, 16, 2, F_shared=16, device="cpu").forward(x, wr, b, {})
