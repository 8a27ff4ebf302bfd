"""Plain 64-bit implementations of the sorted rows and the 8-bit products, for the tests."""
import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # largest relative error of one rounding
U = 2.0 ** -24


def ref_sort(sel, E):
    """(offsets, row, source) of the stable order by (expert, assignment); indices outside [0, E) take no part."""
    flat = sel.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.flatnonzero(ok)
    order = order[np.argsort(flat[order], kind="stable")]
    row = np.full(flat.shape, -1, np.int64)
    row[order] = np.arange(len(order))
    source = np.full(flat.shape, -1, np.int64)
    source[:len(order)] = order
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))])
    return offsets, row.reshape(sel.shape), source


def ref_unsort(ys, row, gates, base, n):
    """(y, magnitude of its terms)."""
    y = np.zeros((row.shape[0], n)) if base is None else base.copy()
    mag = np.abs(y)
    for t in range(row.shape[0]):
        for j in range(row.shape[1]):
            if row[t, j] >= 0:
                term = (1.0 if gates is None else gates[t, j]) * ys[row[t, j]]
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def ref_quantize(x):
    """q and the fp32 scale of float64 rows that hold fp32 values: 127 x is exact in fp64 and the quotient is off by 2^-46,
    while one that is not a tie is at least 2^-34 from it, so the rounding is the exact quotient's."""
    m = np.abs(x).max(-1, keepdims=True)
    q = np.where(m > 0, np.rint(127.0 * x / np.where(m > 0, m, 1.0)), 0.0)
    return q, (m[..., 0].astype(np.float32) / np.float32(127)).astype(np.float64)


def within(got, want, bound, what=""):
    got, want, bound = np.asarray(got, np.float64), np.asarray(want, np.float64), np.asarray(bound, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if not got.size:
        return
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) - bound, -np.inf)), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; at {i}: got {got[i]!r} want "
                             f"{want[i]!r} bound {np.broadcast_to(bound, got.shape)[i]!r}")


def routing(rng, T, k, E, skew=1.0, dropped=0.0):
    """(T, k) expert indices with a popularity skew, distinct within a token where E allows; a share of them -1."""
    score = rng.standard_normal((T, E)) + skew * rng.standard_normal(E)
    if k <= E:
        sel = np.argsort(-score, axis=1, kind="stable")[:, :k].astype(np.int64)
    else:
        sel = rng.integers(0, E, (T, k))
    sel[rng.random((T, k)) < dropped] = -1
    return np.ascontiguousarray(sel)
