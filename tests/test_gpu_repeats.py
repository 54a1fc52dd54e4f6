"""The bf16 and 8-bit calls give the same bits when they are made again: sums are in an order that the layout alone decides."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import test_gpu_expert_products as products
from parity_helpers import dev_bf16
from workloads import PAD_MULTIPLE, PAD_NONE, normal_bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


@pytest.mark.parametrize("S,K,E,H,N,mode,pad,slots", [
    (3, 2, 8, 1024, 136, PAD_NONE, 0, None),          # streamed weights
    (256, 2, 16, 512, 264, PAD_MULTIPLE, 16, None),
    (6000, 4, 12, 1032, 520, PAD_NONE, 0, None),      # tiles, several rounds of them
    (3000, 2, 8, 256, 72, PAD_NONE, 0, 3),            # replicas' rows in the weights' gradients
])
def test_same_bits(moe, S, K, E, H, N, mode, pad, slots):
    rng = np.random.default_rng(S + H)
    c = products.Case(moe, rng, S, K, E, 1 if slots is None else 2, mode, pad, slots)
    x, dy = (c.poisoned(normal_bf16_bits(rng, (c.rows, H))) for _ in range(2))
    w_in, w_out = (dev_bf16(normal_bf16_bits(rng, s), DEV) for s in ((E, 2 * N, H), (E, H, N)))
    d_out, tw = dev_bf16(normal_bf16_bits(rng, (S, H)), DEV), torch.rand((S, K), device=DEV)
    H16 = H // 16 * 16
    x16 = x[:, :H16].contiguous()
    w8, s8 = moe.moe_quantize_i8(w_in[:, :, :H16].contiguous())

    def once():
        pre = torch.zeros((c.rows, 2 * N), device=DEV)
        row = lambda width: torch.zeros((c.rows, width), dtype=torch.bfloat16, device=DEV)   # rows without an entry stay 0
        h = moe.moe_expert_gemm(c.desc, c.lay, x, w_in, act=moe.MOE_ACT_SWIGLU, out=row(N), pre=pre, **c.kw)
        y = moe.moe_expert_gemm(c.desc, c.lay, h, w_out, out=row(H), **c.kw)
        d_pre = moe.moe_expert_gemm_backward_x(c.desc, c.lay, dy, w_out, pre=pre, out=row(2 * N), **c.kw)
        dx = moe.moe_expert_gemm_backward_x(c.desc, c.lay, d_pre, w_in, out=row(H), **c.kw)
        dw_in = moe.moe_expert_gemm_backward_w(c.desc, c.lay, d_pre, x, **c.kw)
        dw_out = moe.moe_expert_gemm_backward_w(c.desc, c.lay, dy, h, dtype=torch.float32, **c.kw)
        codes, scales = torch.zeros((c.rows, H16), dtype=torch.int8, device=DEV), torch.zeros(c.rows, device=DEV)
        moe.moe_quantize_i8(x16, codes, scales, layout=c.lay)
        y8 = moe.moe_expert_gemm_i8(c.desc, c.lay, codes, scales, w8, s8, act=moe.MOE_ACT_SWIGLU, out=row(N), **c.kw)
        d_rows, d_w = moe.moe_combine_backward(c.desc, c.lay, d_out, y, tw, d_expert_out=row(H))
        return pre, h, y, d_pre, dx, dw_in, dw_out, codes, scales, y8, d_rows, d_w

    first = once()
    assert all(bool(torch.isfinite(t.float()).all()) for t in first)
    for _ in range(3):
        for a, b in zip(first, once()):
            assert torch.equal(a, b)
