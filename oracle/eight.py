"""Plain float64 oracle of the 8-bit matrices and their products, the gated activation with its
8-bit checkpoint, and the expert router (test infrastructure only, as mxfp4.py).

An 8-bit matrix here is (codes [rows, cols], scales [rows, ceil(cols / 128)]), without the padding
that the library's rows have.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["E4M3", "SILU", "GELU", "quantize8", "dequantize8", "gemm8", "linear8_fwd", "linear8_bwd", "glu",
           "glu_bwd", "activation", "route", "route_bwd"]

SILU, GELU = 0, 1


def _e4m3_values():
    """The 256 E4M3 values by their bits: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = (math.nan if (c & 127) == 127 else a) * (-1.0 if c & 128 else 1.0)
    return v


E4M3 = _e4m3_values()


def _nearest(a):
    """Codes of the E4M3 magnitudes nearest to a >= 0 (float64, at most 448), ties to the even code."""
    grid = E4M3[:127]
    high = np.clip(np.searchsorted(grid, a), 1, 126)   # grid[high - 1] < a <= grid[high]
    below, above = a - grid[high - 1], grid[high] - a
    up = (above < below) | ((above == below) & (high % 2 == 0))
    return np.where(up, high, high - 1)


def quantize8(x, height: int = 1, width: int = 128):
    """(codes, scales) of blocks of height x width; each row has its block's byte.  Blocks along the
    rows of x are those of its transpose."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, -(-cols // width)), np.uint8)
    for r in range(0, rows, height):
        band = x[r:r + height]
        for b in range(scales.shape[1]):
            block = band[:, b * width:(b + 1) * width]
            if not np.isfinite(block).all():
                scales[r:r + height, b] = 255
                continue
            amax = np.abs(block).max(initial=0.0)
            e = -127
            if amax > 0:
                m, q = math.frexp(amax)           # amax = m 2^q, m in [1/2, 1); 448 = 7/8 2^9
                e = max(-127, q - 9 if m <= 7 / 8 else q - 8)
            scales[r:r + height, b] = e + 127
            code = _nearest(np.abs(block) * 2.0 ** -e)
            codes[r:r + height, b * width:(b + 1) * width] = code + 128 * np.signbit(block)
    return codes, scales


def dequantize8(codes, scales):
    """Exact values; a block with scale byte 255 is NaN."""
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return E4M3[codes] * np.repeat(s, 128, axis=1)[:, :codes.shape[1]]


def gemm8(a, b, alpha: float = 1.0):
    """(C, sum of magnitudes) of alpha A B^T."""
    a, b = dequantize8(*a), dequantize8(*b)
    with np.errstate(invalid="ignore"):
        return alpha * (a @ b.T), abs(alpha) * (np.abs(a) @ np.abs(b).T)


def linear8_fwd(x, w):
    """((y, magnitudes), xq, wq): 1x128 blocks of x, 128x128 tiles of w."""
    xq, wq = quantize8(x), quantize8(w, 128, 128)
    return gemm8(xq, wq), xq, wq


def linear8_bwd(dy, xq, wq):
    """((dx, magnitudes), (dw, magnitudes)): dy in 1x128 blocks times the weight's values; dy and the kept
    x in blocks of 128 rows."""
    w = dequantize8(*wq)
    d = dequantize8(*quantize8(dy))
    dx = d @ w, np.abs(d) @ np.abs(w)
    dt = dequantize8(*quantize8(np.asarray(dy, np.float64).T))
    xt = dequantize8(*quantize8(dequantize8(*xq).T))
    return dx, (dt @ xt.T, np.abs(dt) @ np.abs(xt).T)


# ------------------------------------------------------------------ gated activation
def activation(g, act: int):
    """act(g), act'(g)."""
    g = np.asarray(g, np.float64)
    if act == SILU:
        s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
        return g * s, s + g * s * (1 - s)
    erfc = np.vectorize(math.erfc, otypes=[np.float64])
    phi = 0.5 * erfc(-g / math.sqrt(2.0))
    return g * phi, phi + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def glu(z, act: int):
    g, u = np.split(np.asarray(z, np.float64), 2, axis=1)
    return activation(g, act)[0] * u


def glu_bwd(dh, g, u, act: int):
    """dz from the values g and u that the checkpoint holds."""
    a, da = activation(g, act)
    dh = np.asarray(dh, np.float64)
    return np.concatenate((dh * u * da, dh * a), axis=1)


# ------------------------------------------------------------------ router
def _softmax(row):
    e = np.exp(row - row.max())
    return e / e.sum()


def route(logits, top_k: int, renormalize: bool, mask=None):
    """(ids, weights, counts, sums, loss) of finite or -Inf logits."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids = np.full((T, top_k), -1, np.int32)
    p = np.zeros((T, top_k))
    counts, sums, n = np.zeros(E, np.int64), np.zeros(E), 0
    for t in range(T):
        if (mask is not None and not mask[t]) or (logits[t] == -np.inf).all():
            continue
        n += 1
        s = _softmax(logits[t])
        sums += s
        order = sorted((e for e in range(E) if logits[t, e] > -np.inf), key=lambda e: (-logits[t, e], e))[:top_k]
        ids[t, :len(order)] = order
        p[t, :len(order)] = s[order]
        if renormalize:
            p[t] /= p[t].sum()
        counts[order] += 1
    loss = E * float(np.dot(counts / (n * top_k), sums / n)) if n else 0.0
    return ids, p, np.append(counts, n).astype(np.int32), sums, loss


def route_bwd(logits, ids, counts, dp, dloss: float, renormalize: bool, mask=None):
    """(dlogits, magnitudes of its terms): the softmax's Jacobian times the gradient of its outputs."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k, n = ids.shape[1], int(counts[E])
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    G0 = dloss * E * counts[:E] / (n * k) / n if n else np.zeros(E)
    for t in range(T):
        if (mask is not None and not mask[t]) or (logits[t] == -np.inf).all():
            continue
        s = _softmax(logits[t])
        G, A = G0.copy(), np.abs(G0)
        taken = [(int(e), float(dp[t, j])) for j, e in enumerate(ids[t]) if e >= 0]
        share = sum(s[e] for e, _ in taken) if renormalize else 1.0
        inner = sum(s[e] / share * v for e, v in taken) if renormalize else 0.0
        bound = sum(s[e] / share * abs(v) for e, v in taken) if renormalize else 0.0
        for e, v in taken:
            G[e] += (v - inner) / share
            A[e] += (abs(v) + bound) / share
        d[t] = s * (G - np.dot(s, G))
        mag[t] = s * (A + np.dot(s, A))
    return d, mag
