"""Combine's gradient on the GPU: the rows bit for bit (one product, one rounding), the weights within a bound.

A weight's gradient is a sum of H products of bf16 values, each exact in fp32,
by fused steps: (H + 2) * 2^-24 of the sum of their absolute values at most, in
any order.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from expert_products_reference import combine_backward
from parity_helpers import POISON_BF16, dev_bf16, host_bits
from router_mx4_reference import bf16_values, to_bf16
from workloads import PAD_CAPACITY, PAD_MULTIPLE, PAD_NONE, normal_bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("S,K,E,R,H,mode,pad", [
    (1, 1, 1, 1, 8, PAD_NONE, 0), (1, 8, 8, 2, 7168, PAD_NONE, 0), (130, 8, 64, 8, 7168, PAD_CAPACITY, 12),
    (77, 3, 12, 4, 2184, PAD_MULTIPLE, 16), (300, 16, 40, 5, 392, PAD_NONE, 0), (64, 5, 9, 3, 16392, PAD_MULTIPLE, 100),
    (200, 2, 6, 2, 520, PAD_CAPACITY, 3),
])
def test_combine_backward(moe, S, K, E, R, H, mode, pad):
    rng = np.random.default_rng(S * K + H)
    idx = rng.integers(-1, E, (S, K)).astype(np.int32)
    desc = moe.LayoutDesc(S, K, E, R, mode, pad)
    lay = moe.moe_layout(desc, dev(idx))
    ref = oracle.layout(idx, E, R, mode, pad)
    rows, held = len(ref.src), ref.src >= 0
    db, yb = normal_bf16_bits(rng, (S, H)), normal_bf16_bits(rng, (rows, H))
    w = rng.random((S, K)).astype(np.float32)
    d, y = dev_bf16(db, DEV), dev_bf16(np.where(held[:, None], yb, POISON_BF16).astype(np.uint16), DEV)
    for weight in (w, None):
        # one fp32 product per element, as the kernel's: exact in 64 bits, then fp32, then bf16
        ones = np.ones((S, K), np.float32) if weight is None else weight
        want_y, want_w, size = combine_backward(bf16_values(db), bf16_values(yb), ones.astype(np.float64), ref.pos.reshape(S, K), rows)
        W = None if weight is None else dev(weight)
        out = torch.full((rows + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)
        d_y, d_w = moe.moe_combine_backward(desc, lay, d, y, W, d_expert_out=out)
        bits = host_bits(d_y)
        assert (bf16_values(bits)[:rows][~held] == 7.0).all() and (bf16_values(bits)[rows:] == 7.0).all()
        assert np.array_equal(bits[:rows][held], to_bf16(want_y[held].astype(np.float32)))
        off = np.abs(d_w.cpu().numpy() - want_w)
        assert (off <= (H + 2) * 2.0 ** -24 * size).all()
        # each alone, and the rows into the experts' own
        assert torch.equal(moe.moe_combine_backward(desc, lay, d, y, W, rows=False)[1], d_w)
        alone = torch.full_like(out, 7.0)
        assert moe.moe_combine_backward(desc, lay, d, None, W, d_expert_out=alone, weights=False)[1] is None
        assert torch.equal(alone, out)
        own = y.clone()
        _, again = moe.moe_combine_backward(desc, lay, d, own, W, d_expert_out=own)
        assert torch.equal(again, d_w)
        assert np.array_equal(host_bits(own)[held], bits[:rows][held])
        assert np.array_equal(host_bits(own)[~held], host_bits(y)[~held])


def test_empty_batch(moe):
    desc = moe.LayoutDesc(0, 2, 4, 2, moe.MOE_PAD_CAPACITY, 3)
    lay = moe.moe_layout(desc, torch.zeros((0, 2), dtype=torch.int32, device=DEV))
    y = torch.full((12, 16), 7.0, dtype=torch.bfloat16, device=DEV)
    _, d_w = moe.moe_combine_backward(desc, lay, torch.zeros((0, 16), dtype=torch.bfloat16, device=DEV), y, d_expert_out=y)
    assert d_w.shape == (0, 2) and (y == 7.0).all()


def test_broken_values(moe):
    """A NaN or an infinity in one token's gradient or one row stays with that token."""
    rng = np.random.default_rng(3)
    S, K, E, H = 9, 2, 4, 64
    desc = moe.LayoutDesc(S, K, E, 1)
    lay = moe.moe_layout(desc, dev(rng.integers(0, E, (S, K)).astype(np.int32)))
    pos = lay.pos.cpu().numpy()
    db, yb = normal_bf16_bits(rng, (S, H)), normal_bf16_bits(rng, (S * K, H))
    db[4, 7], yb[pos[6, 1], 3] = 0x7FC0, 0x7F80
    d_y, d_w = moe.moe_combine_backward(desc, lay, dev_bf16(db, DEV), dev_bf16(yb, DEV))
    bad = ~np.isfinite(d_w.cpu().numpy())
    assert bad[4].all() and bad[6, 1] and bad.sum() == 3
    bad = ~np.isfinite(bf16_values(host_bits(d_y)))
    assert bad[pos[4], 7].all() and bad.sum() == 2
