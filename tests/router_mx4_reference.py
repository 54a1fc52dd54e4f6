"""Plain references in 64 bits for the router, the balance loss and the MXFP4
operators, written from the formulas in include/moe_ep.h (numpy, CPU)."""
from __future__ import annotations

import numpy as np

NEG = -np.inf


def router_reference(z, K, n_groups=1, topk_groups=None, renorm=True, seq_len=0, alpha=1.0, mask=None, given=None):
    """z [S,E] float64.  Returns a dict: idx, w, count, coef, loss, p, counts (token counts), broken."""
    S, E = z.shape
    tg = n_groups if topk_groups is None else topk_groups
    live = np.ones(S, bool) if mask is None else mask.astype(bool)
    broken = live & (np.isnan(z) | (z == np.inf)).any(1)
    counts = live & (broken | (z > NEG).any(1))
    good = counts & ~broken
    p = np.zeros((S, E))
    with np.errstate(invalid="ignore"):
        e = np.exp(z[good] - z[good].max(1, keepdims=True)) if good.any() else z[good]
    p[good] = e / e.sum(1, keepdims=True) if good.any() else e
    p[broken] = np.nan
    if given is None:
        idx, w = np.full((S, K), -1, np.int64), np.zeros((S, K))
        for t in np.nonzero(good)[0]:
            row = z[t] + 0.0
            size = E // n_groups
            best = np.argsort(-row.reshape(n_groups, size).max(1), kind="stable")[:tg]
            left = np.full(E, NEG)
            for g in best:
                left[g * size:(g + 1) * size] = row[g * size:(g + 1) * size]
            order = [i for i in np.argsort(-left, kind="stable")[:K] if left[i] > NEG]
            idx[t, :len(order)] = order
            if renorm:
                q = np.exp(left[order] - left[order].max())
                w[t, :len(order)] = q / q.sum()
            else:
                w[t, :len(order)] = p[t, order]
    else:
        idx, w = given.astype(np.int64), None
    T = seq_len or S
    G = S // T if seq_len else 1
    count, coef = np.zeros((G, E), np.int64), np.zeros((G, E))
    n = np.zeros(G, np.int64)
    for g in range(G):
        rows = slice(g * T, (g + 1) * T)
        ids = idx[rows][counts[rows]].reshape(-1)
        np.add.at(count[g], ids[(ids >= 0) & (ids < E)], 1)
        n[g] = counts[rows].sum()
    used = max(int((n > 0).sum()), 1)
    loss = 0.0
    for g in range(G):
        if n[g]:
            f = E * count[g] / (K * n[g])
            P = p[g * T:(g + 1) * T].sum(0) / n[g]
            loss += alpha * (f * P).sum() / used
            coef[g] = alpha * E * count[g] / (K * n[g] ** 2 * used)
    return dict(idx=idx, w=w, count=count, coef=coef, loss=loss, p=p, counts=counts, broken=broken)


def router_gradient(ref, z, renorm=True, seq_len=0, d_w=None, d_loss=None):
    """The formula's d logits, and for every element the size of the terms it is
    made of (what rounding errors are relative to)."""
    S, E = z.shape
    p = ref["p"]
    d, size = np.zeros((S, E)), np.zeros((S, E))
    seq = np.arange(S) // (seq_len or max(S, 1))
    if d_loss is not None:
        c = ref["coef"][seq] if S else np.zeros((0, E))
        inner = (c * p).sum(1, keepdims=True)
        d += d_loss * p * (c - inner)
        size += abs(d_loss) * p * (c + inner)
    if d_w is not None:
        for t in range(S):
            got = ref["idx"][t] >= 0
            i, w, g = ref["idx"][t][got], ref["w"][t][got], d_w[t][got]
            inner, ainner = (w * g).sum(), (w * np.abs(g)).sum()
            if renorm:
                d[t, i] += w * (g - inner)
                size[t, i] += w * (np.abs(g) + ainner)
            elif len(i):
                dp = np.zeros(E)
                dp[i] = g
                d[t] += p[t] * (dp - inner)
                size[t] += p[t] * (np.abs(dp) + ainner)
    d[~ref["counts"]] = 0.0
    d[ref["broken"]] = np.nan
    return d, size


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_values(bits):
    """bf16 bit patterns (uint16) -> float64."""
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16(v):
    """float64 -> bf16 bits, to nearest, ties to even, by the distance to both neighbours (finite values)."""
    v = np.asarray(v, np.float64)
    f = v.astype(np.float32)                     # a start within one bf16 step, then corrected
    lo = (f.view(np.uint32) >> 16).astype(np.uint32)
    cand = np.stack([np.maximum(lo, 1) - 1, lo, lo + 1])
    cand = np.where((cand & 0x8000) == (lo & 0x8000), cand, lo)
    val = (cand.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    dist = np.where(np.isfinite(val), np.abs(val - v), np.inf)
    odd = (cand & 1).astype(np.int64)
    best = np.lexsort((odd, dist), axis=0)[0]
    return np.take_along_axis(cand, best[None], 0)[0].astype(np.uint16)


def mx4_quantize(x):
    """x [rows,H] float64 (bf16 values) -> codes [rows,H/2], scales [rows,H/32] uint8."""
    rows, H = x.shape
    b = x.reshape(rows, H // 32, 32)
    bad = ~np.isfinite(b).all(2)
    top = np.where(bad, 0.0, np.abs(b).max(2))
    e = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2, -127)
    # log2 of a power of two's neighbours rounds to the right side: bf16 values have 8 bits
    e = np.clip(e, -127, 127)
    with np.errstate(invalid="ignore"):
        m = np.abs(b) / np.exp2(e)[:, :, None]
        d = np.abs(m[..., None] - E2M1)
    d = np.where(np.isnan(d), np.inf, d)
    near = d == d.min(-1, keepdims=True)
    # of two equally near magnitudes the even code
    code = np.where(near, np.where(np.arange(8) % 2 == 0, np.arange(8), np.arange(8) + 100), 1000).min(-1) % 100
    code = code + 8 * np.signbit(b)
    code = np.where(bad[..., None], 0, code).reshape(rows, H).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def mx4_values(codes, scales):
    """Packed MXFP4 -> float64 (last axis H/2 -> H)."""
    code = np.stack([codes & 15, codes >> 4], -1).reshape(*scales.shape, 32)
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def expert_product(x, w, expert_of_row, swiglu):
    """x [rows,H], w [E,M,H] float64, expert_of_row [rows] (-1: none) -> [rows,N] float64 (NaN where none), and the
    sum of the absolute products (of gate and up: two arrays)."""
    rows = x.shape[0]
    M = w.shape[1]
    y, size = np.full((rows, M), np.nan), np.zeros((rows, M))
    for e in np.unique(expert_of_row[expert_of_row >= 0]):
        r = expert_of_row == e
        y[r] = x[r] @ w[e].T
        size[r] = np.abs(x[r]) @ np.abs(w[e]).T
    if not swiglu:
        return y, y, size
    g, u = y[:, :M // 2], y[:, M // 2:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u, y, size
