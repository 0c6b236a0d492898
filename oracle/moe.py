"""Plain float64 oracle of the expert routing operators and of the products of a few
unquantized rows with packed weights (test infrastructure only, as mxfp4.py).

Slot s = token * top_k + j is a token's j-th choice; pos[t, j] is its row in expert
order, -1 where it takes part in nothing.
"""
from __future__ import annotations

import numpy as np

from .mxfp4 import ROW, dequantize

__all__ = ["moe_plan", "moe_dispatch", "moe_combine", "moe_combine_bwd", "gemv", "gemv_grouped"]


def moe_plan(ids, experts: int):
    """(offs [experts + 1], src [slots], pos [tokens, top_k]): slots in a stable order by
    expert; ids outside 0 .. experts - 1 leave their slot out."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    src = np.full(flat.size, -1, dtype=np.int32)
    pos = np.full(flat.size, -1, dtype=np.int32)
    offs = np.zeros(experts + 1, dtype=np.int64)
    row = 0
    for e in range(experts):
        for s in np.nonzero(flat == e)[0]:
            src[row], pos[s] = s, row
            row += 1
        offs[e + 1] = row
    return offs, src, pos.reshape(ids.shape)


def _slots(pos, rows):
    return [(t, j, int(pos[t, j])) for t, j in np.ndindex(*pos.shape) if 0 <= pos[t, j] < rows]


def moe_dispatch(x, pos, weights, out):
    """out (a copy of it, float64) with out[pos[t, j]] = weights[t, j] * x[t]."""
    out = np.array(out, dtype=np.float64)
    for t, j, row in _slots(pos, out.shape[0]):
        out[row] = np.asarray(x[t], np.float64) * (1.0 if weights is None else float(weights[t, j]))
    return out


def moe_combine(z, pos, weights):
    """(y, sum of magnitudes): y[t] = sum_j weights[t, j] z[pos[t, j]]."""
    y = np.zeros((pos.shape[0], z.shape[1]))
    mag = np.zeros_like(y)
    for t, j, row in _slots(pos, z.shape[0]):
        term = np.asarray(z[row], np.float64) * (1.0 if weights is None else float(weights[t, j]))
        y[t] += term
        mag[t] += np.abs(term)
    return y, mag


def moe_combine_bwd(dy, z, pos, weights, dz):
    """(dz, dweights, sum of magnitudes of dweights' terms); dz keeps rows no slot maps to."""
    dz = moe_dispatch(dy, pos, weights, dz)
    dw = np.zeros(pos.shape)
    mag = np.zeros(pos.shape)
    for t, j, row in _slots(pos, z.shape[0]):
        terms = np.asarray(dy[t], np.float64) * np.asarray(z[row], np.float64)
        dw[t, j], mag[t, j] = terms.sum(), np.abs(terms).sum()
    return dz, dw, mag


def gemv(x, codes, scales, alpha: float = 1.0):
    """(y, sum of magnitudes) of alpha x deq(W)^T; scales may have more bytes per row than
    the matrix has blocks."""
    N, K = codes.shape[0], 2 * codes.shape[1]
    w = dequantize(codes, np.ascontiguousarray(scales[:, :K // 32]), N, K, ROW)
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        return alpha * (x @ w.T), abs(alpha) * (np.abs(x) @ np.abs(w).T)


def gemv_grouped(x, codes, scales, offs, src, top_k: int, rows: int, alpha: float = 1.0):
    """(y, magnitudes) [rows, N]; rows that are not computed are NaN."""
    N = codes.shape[1]
    y = np.full((rows, N), np.nan)
    mag = np.full((rows, N), np.nan)
    for e in range(len(offs) - 1):
        for r in range(int(offs[e]), min(int(offs[e + 1]), rows)):
            xr = r if src is None else (int(src[r]) // top_k if src[r] >= 0 else -1)
            if 0 <= xr < len(x):
                y[r:r + 1], mag[r:r + 1] = gemv(x[xr:xr + 1], codes[e], scales[e], alpha)
    return y, mag
