"""silu and its gradient at the ends of its argument's range, through the products: the reciprocal of the hardware has no
subnormal results, so below g = -126 ln 2 = -87.3 the sigmoid, at most 2^-126 there, is 0; infinities as the header says."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
G = [-60.0, -80.0, -87.0, -87.5, -88.0, -89.0, -90.0, -91.5, -100.0, -120.0, -200.0, -1e30, 0.0, 60.0, 88.0, 89.0, 200.0, 1e30]


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def through(moe, g, u, rows):
    """h, and the gradient of (g, u) for dh = 1, of `rows` equal rows with these arguments of the activation."""
    N, H = 256, 1024
    desc = moe.LayoutDesc(rows, 1, 1, 1)
    lay = moe.moe_layout(desc, torch.zeros((rows, 1), dtype=torch.int32, device=DEV))
    # one channel of x and of d_out: no product with an infinity but the argument's own
    x = torch.zeros((rows, H), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    w = torch.zeros((1, 2 * N, H), dtype=torch.bfloat16, device=DEV)
    w[0, :len(g), 0] = torch.tensor(g, device=DEV)
    w[0, N:, 0] = u
    wo = torch.zeros((1, H, N), dtype=torch.bfloat16, device=DEV)
    wo[0, 0] = 1
    pre = torch.empty((rows, 2 * N), device=DEV)
    h = moe.moe_expert_gemm(desc, lay, x, w, act=moe.MOE_ACT_SWIGLU, pre=pre)
    d = moe.moe_expert_gemm_backward_x(desc, lay, x, wo, pre=pre)
    n = len(g)
    return [t[:, :n].double().cpu() for t in (pre, h, d)] + [d[:, N:N + n].double().cpu()]


@pytest.mark.parametrize("rows", [2, 6000])   # streamed weights, tiles
@pytest.mark.parametrize("u", [1.0, -0.5])
def test_far_arguments(moe, rows, u):
    pre, h, dg, du = through(moe, G, u, rows)
    for i in range(len(G)):
        g = float(pre[0, i])
        s = 1.0 / (1.0 + math.exp(-g)) if g > -700 else 0.0
        lost = 2.0 ** -126 * (abs(g) + 1) if -200 < g < -87 else 0.0     # a sigmoid below 2^-126 is 0
        # silu within (8 + |g|) units of 2^-23, its slope within 16 (1 + |g|), then half a step of bf16
        for got, want, units in ((h, g * s * u, 8 + abs(g)), (dg, u * s * (1 + g * (1 - s)), 16 * (1 + abs(g))), (du, g * s, 8 + abs(g))):
            allowed = (2.0 ** -8 + min(units, 4096) * 2.0 ** -23) * abs(want) + lost * 1.01 + 2.0 ** -133
            assert (got[:, i] - want).abs().max() <= allowed, (g, float(got[0, i]), want)


@pytest.mark.parametrize("rows", [2, 6000])
def test_infinities(moe, rows):
    pre, h, dg, du = through(moe, [-math.inf, math.inf, 1.0], 1.0, rows)
    assert pre[:, 0].eq(-math.inf).all() and pre[:, 1].eq(math.inf).all()
    assert h[:, 0].isnan().all() and dg[:, 0].isnan().all() and du[:, 0].isnan().all()
    assert h[:, 1].eq(math.inf).all() and dg[:, 1].isnan().all() and du[:, 1].eq(math.inf).all()
    assert h[:, 2].isfinite().all() and dg[:, 2].isfinite().all() and du[:, 2].isfinite().all()
