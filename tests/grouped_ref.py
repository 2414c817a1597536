"""References in 64 bits and error bounds for the grouped products over plain weights and their neighbours."""
from __future__ import annotations

import numpy as np
import torch

# half a step of each result type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TORCH_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t) -> torch.Tensor:
    return t.detach().cpu().to(torch.float64)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def gathered(x, perm, k, rows):
    """x[perm[p] // k] for p < rows in 64 bits (zeros where perm names no row), or x itself."""
    x = f64(x)
    if perm is None:
        return x
    perm = perm.cpu().long()[:rows]
    src = torch.div(perm, k, rounding_mode="floor")
    ok = (perm >= 0) & (src < x.shape[0])
    out = torch.zeros((rows, x.shape[1]), dtype=torch.float64)
    out[ok] = x[src[ok]]
    return out


def product(op, x, w, y, offsets):
    """(value, sum of |terms|, terms per sum) of the grouped product `op`, in 64 bits: x [rows, K] gathered,
    w [E, N, K], y [rows, N]; rows that belong to no group are NaN."""
    E, rows = len(offsets) - 1, (x if x is not None else y).shape[0]
    N, K = (w.shape[1], w.shape[2]) if w is not None else (y.shape[1], x.shape[1])
    if op == "dw":
        out, mag = (torch.zeros((E, N, K), dtype=torch.float64) for _ in range(2))
    else:
        out, mag = (torch.full((rows, N if op == "y" else K), float("nan"), dtype=torch.float64) for _ in range(2))
    n = {"y": K, "dx": N, "dw": max(1, int(np.diff(offsets).max()))}[op]
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo >= hi:
            continue
        if op == "y":
            a, b, dst = x[lo:hi], w[e].T, slice(lo, hi)
        elif op == "dx":
            a, b, dst = y[lo:hi], w[e], slice(lo, hi)
        else:
            a, b, dst = y[lo:hi].T, x[lo:hi], e
        out[dst] = a @ b
        mag[dst] = a.abs() @ b.abs()
    return out, mag, n


def assert_product(got, value, mag, n, what=""):
    """Every element of `got` within the bound of an fp32 sum of n exact products and one rounding.

    A sum of n terms takes n - 1 additions; each is off by at most one step (2^-23, rounded or truncated)
    of a partial sum, and no partial sum exceeds the sum of the terms' magnitudes by more than those errors:
    |error| <= n 2^-23 mag (1 + small).  fp32 products round once more, 2^-24 each, inside the same bound for
    one more addition.  The result is then rounded to its type once."""
    half = HALF_STEP[got.dtype]
    g = f64(got)
    placed = ~torch.isnan(value)
    acc = (n + 1) * 2.0 ** -23 * mag
    bound = acc + half * (value.abs() + acc) + 1e-37
    err = (g - value).abs()
    bad = placed & ~(err <= bound)
    assert not bad.any(), "%s: %d of %d off, first at %s: got %r, want %r, bound %.3e" % (
        what, int(bad.sum()), int(placed.sum()), tuple(torch.nonzero(bad)[0].tolist()), float(g[bad][0]),
        float(value[bad][0]), float(bound[bad][0]))
