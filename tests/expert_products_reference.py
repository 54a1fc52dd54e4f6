"""64-bit references of the bf16 and 8-bit products, their gradients, the 8-bit rows and combine's gradient."""
from __future__ import annotations

import numpy as np


def expert_of_rows(layout, E, rows):
    """Expert of each row of the receive buffer, -1 where it holds no entry (a plain layout of the oracle)."""
    out = np.full(rows, -1)
    for e in range(E):
        o = layout.expert_offset[e]
        out[o:o + layout.tokens_per_expert[e]] = e
    return out


def product(x, w, of_row):
    """x [rows,H], w [E,M,H] -> [rows,M], zeros where no expert, and the sums of absolute products."""
    y, size = np.zeros((len(of_row), w.shape[1])), np.zeros((len(of_row), w.shape[1]))
    for e in np.unique(of_row[of_row >= 0]):
        r = of_row == e
        y[r] = x[r] @ w[e].T
        size[r] = np.abs(x[r]) @ np.abs(w[e]).T
    return y, size


def product_dw(d, x, of_row, E):
    """sum over the rows of each expert of d[r]^T x[r] -> [E,N,H], and the sums of absolute products."""
    dw, size = np.zeros((E, d.shape[1], x.shape[1])), np.zeros((E, d.shape[1], x.shape[1]))
    for e in np.unique(of_row[of_row >= 0]):
        r = of_row == e
        dw[e] = d[r].T @ x[r]
        size[e] = np.abs(d[r]).T @ np.abs(x[r])
    return dw, size


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def silu_slope(g):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return s * (1.0 + g * (1.0 - s))


def quantize_i8(x):
    """x [rows,H] float64 (bf16 values) -> int8 codes, fp32 scales; the definition's two fp32 divisions."""
    broken = ~np.isfinite(x).all(1)
    top = np.where(broken, 0.0, np.abs(np.where(np.isfinite(x), x, 0.0)).max(1)).astype(np.float32)
    scale = top / np.float32(127.0)
    some = (scale > 0)[:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        q = np.where(np.isfinite(x), x, 0.0).astype(np.float32) / np.where(some, scale[:, None], np.float32(1.0))
    code = np.where(some, np.clip(np.rint(q), -127, 127), 0).astype(np.int8)
    return np.where(broken[:, None], 0, code).astype(np.int8), np.where(broken, np.float32(np.nan), scale).astype(np.float32)


def combine_backward(d_out, y, w, pos, rows):
    """d_y [rows,H] (NaN where no entry), d_w [S,K], and the sums of absolute products behind d_w."""
    S, K = pos.shape
    d_y = np.full((rows, d_out.shape[1]), np.nan)
    d_w, size = np.zeros((S, K)), np.zeros((S, K))
    for t in range(S):
        for k in range(K):
            if pos[t, k] >= 0:
                d_y[pos[t, k]] = w[t, k] * d_out[t]
                d_w[t, k] = (d_out[t] * y[pos[t, k]]).sum()
                size[t, k] = np.abs(d_out[t] * y[pos[t, k]]).sum()
    return d_y, d_w, size
