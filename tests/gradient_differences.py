"""Gradients against differences: along a direction s, (F(p + s) - F(p - s)) / 2 is the gradient times s, up to roundings
and the third derivative, both bounded here.

F(x, w_in, w_out) = sum over the rows that hold an entry of dy * y, y the experts' gated feed-forward block.  A direction has
the gradient's own signs, so that its terms add up and the derivative stands far above the bound: whoever calls this
asserts by how much.
"""
from __future__ import annotations

import numpy as np

from expert_products_reference import silu, silu_slope
from router_mx4_reference import bf16_values, to_bf16

HALF_STEP = 2.0 ** -8      # bf16: a rounding's part of the value, at most
# fp32 sums of at most 48 terms, the hardware's exponential and reciprocal (|g| < 16) and the products after them:
# (48/32 + 16) + (8 + 16) + 8 units of 2^-23, below 2^-17, of the sum of absolute terms
FP32 = 2.0 ** -17
STEPS = {"x": 2.0 ** -3, "w_in": 2.0 ** -6, "w_out": 2.0 ** -2}


def inputs(rng, rows, E, H, N):
    """Multiples of powers of two that bf16 holds, with a step of STEPS added or taken away too: sums of the first product
    are exact in fp32.  w_out and dy are mostly positive: the bound adds what the gradient of h may cancel."""
    return dict(x=rng.integers(-2, 3, (rows, H)) / 2.0, w_in=rng.integers(-4, 5, (E, 2 * N, H)) / 16.0,
                w_out=rng.integers(-1, 5, (E, H, N)) / 4.0, dy=rng.integers(-1, 5, (rows, H)) * 1.0)


def block(v, of_row):
    """Each held row's (g, u, h, y) in 64 bits."""
    held = np.nonzero(of_row >= 0)[0]
    e, N = of_row[held], v["w_out"].shape[2]
    pre = np.einsum("rh,rnh->rn", v["x"][held], v["w_in"][e])
    g, u = pre[:, :N], pre[:, N:]
    h = silu(g) * u
    return g, u, h, np.einsum("rn,rhn->rh", h, v["w_out"][e])


def gradients(v, of_row, slope=silu_slope):
    """The formulas in 64 bits (slope: silu's derivative, of g), with the gradient of pre."""
    held = np.nonzero(of_row >= 0)[0]
    e = of_row[held]
    g, u, h, _ = block(v, of_row)
    dy, dh = v["dy"][held], np.einsum("rh,rhn->rn", v["dy"][held], v["w_out"][e])
    d_pre = np.concatenate([dh * u * slope(g), dh * silu(g)], 1)
    out = {k: np.zeros_like(v[k]) for k in ("x", "w_in", "w_out")}
    out["x"][held] = np.einsum("rn,rnh->rh", d_pre, v["w_in"][e])
    np.add.at(out["w_in"], e, d_pre[:, :, None] * v["x"][held][:, None, :])
    np.add.at(out["w_out"], e, dy[:, :, None] * h[:, None, :])
    return out, d_pre


def direction(v, of_row, name):
    return np.sign(gradients(v, of_row)[0][name]) * STEPS[name]


def loss(y, v, of_row):
    """F from the held rows' y."""
    return float((y * v["dy"][of_row >= 0]).sum())


def rounded_block(v, of_row):
    """y with the roundings of the calls: h, then y, to bf16."""
    held = np.nonzero(of_row >= 0)[0]
    h = bf16_values(to_bf16(block(v, of_row)[2]))
    return bf16_values(to_bf16(np.einsum("rn,rhn->rh", h, v["w_out"][of_row[held]])))


def bound(v, of_row, name, s):
    """Of |(F(p + s) - F(p - s)) / 2 - gradient * s|."""
    held = np.nonzero(of_row >= 0)[0]
    e = of_row[held]
    dy = np.abs(v["dy"][held])
    g, u, h, _ = block(v, of_row)
    total = 0.0
    for sign in (1, -1):
        p = dict(v, **{name: v[name] + sign * s})
        _, _, hp, yp = block(p, of_row)
        through = np.einsum("rh,rhn->rn", dy, np.abs(p["w_out"][e]))         # of an error of h
        # h and y are rounded to bf16 (y from a rounded h: its own step may be of a value that much larger)
        err_h = np.abs(hp) * (HALF_STEP + FP32)
        err_y = np.einsum("rn,rhn->rh", err_h + FP32 * np.abs(hp), np.abs(p["w_out"][e]))
        total += 0.5 * ((err_h * through).sum() + (dy * (HALF_STEP * (np.abs(yp) + err_y) + err_y * FP32)).sum())
        total += 0.5 * FP32 * (np.abs(hp) * through).sum()
    if name != "w_out":
        # the third derivative of silu(g + t a) * (u + t b) in t: |silu''| <= 1/2, |silu'''| <= 2/3
        # (sigma' <= e^-|g| and |sigma'''| <= sigma', |sigma''| < 1/10: 3 * 0.1 + |g| e^-|g| <= 0.3 + 1/e)
        if name == "x":
            d = np.einsum("rh,rnh->rn", s[held], v["w_in"][e])
        else:
            d = np.einsum("rh,rnh->rn", v["x"][held], s[e])
        N = g.shape[1]
        a, b = np.abs(d[:, :N]), np.abs(d[:, N:])
        dh = np.abs(np.einsum("rh,rhn->rn", v["dy"][held], v["w_out"][e]))
        total += (dh * (2.0 / 3.0 * a ** 3 * (np.abs(u) + b) + 1.5 * a ** 2 * b)).sum() / 6.0
    # the gradient: what it is made of is rounded to bf16 (h, or the gradient of pre), and so is it
    grads, d_pre = gradients(v, of_row)
    terms = np.zeros_like(v[name])
    size_dh = np.einsum("rh,rhn->rn", dy, np.abs(v["w_out"][e]))
    kept = (HALF_STEP + FP32) * np.abs(d_pre) + FP32 * np.concatenate([size_dh * (np.abs(u) + 1), size_dh * (np.abs(g) + 1)], 1)
    if name == "w_out":
        np.add.at(terms, e, dy[:, :, None] * ((HALF_STEP + 2 * FP32) * np.abs(h))[:, None, :])
    elif name == "w_in":
        np.add.at(terms, e, kept[:, :, None] * np.abs(v["x"][held])[:, None, :])
    else:
        terms[held] = np.einsum("rn,rnh->rh", kept, np.abs(v["w_in"][e]))
    total += (np.abs(s) * (terms * (1 + HALF_STEP) + HALF_STEP * np.abs(grads[name]))).sum()
    return float(total)
