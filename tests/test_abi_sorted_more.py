"""More refusals of the sorted-row and 8-bit entry points, on the CPU: no kernel is launched, no pointer is read."""
import pytest

import sparse_mixture_experts_stable_b200 as moe
from sparse_mixture_experts_stable_b200 import binding as B
from tests.test_abi_sorted import BAD, NO, N, P


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
