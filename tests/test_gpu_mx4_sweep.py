"""Products of shapes drawn at random, on both sides of the rule between the two kernels, wide scales and NaN blocks in
either; and every scale byte with every code through the conversion back.  Bounds as in test_gpu_mx4.py."""
from __future__ import annotations

import random

import numpy as np
import pytest
import torch

import oracle
from parity_helpers import host_bits
from router_mx4_reference import E2M1, bf16_values
from test_gpu_mx4 import dev, expert_of_rows, mx4_random, product_check
from workloads import PAD_CAPACITY, PAD_MULTIPLE, PAD_NONE

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


@pytest.mark.parametrize("layout", ["plain", "rows in use"])
def test_every_scale_with_every_code(moe, layout):
    """Exact up to bf16's range; 2^128 and more are infinities, a scale of 255 is NaN."""
    scales = np.repeat(np.arange(256, dtype=np.uint8), 16 * 4).reshape(-1, 4)      # rows of 128 channels
    low = np.tile(np.arange(16, dtype=np.uint8), 256)
    codes = (low[:, None] | (np.arange(64, dtype=np.uint8) % 16 << 4)[None]).astype(np.uint8)
    n = len(scales)
    lay = None
    if layout != "plain":
        lay = moe.moe_layout(moe.LayoutDesc(n, 1, 1, 1), torch.zeros((n, 1), dtype=torch.int32, device=DEV))
    got = bf16_values(host_bits(moe.moe_dequantize_mx4(dev(codes), dev(scales), layout=lay)))
    code = np.stack([codes & 15, codes >> 4], -1).reshape(n, 128)
    want = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0) * np.exp2(np.repeat(scales, 32, 1).astype(np.float64) - 127)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    nan = np.repeat(scales, 32, 1) == 255
    assert np.isnan(got[nan]).all()
    assert np.array_equal(got[~nan], want[~nan]) and np.array_equal(np.signbit(got[~nan]), np.signbit(want[~nan]))


@pytest.mark.parametrize("seed", range(24))
def test_products_drawn(moe, seed):
    rng, r = np.random.default_rng(seed), random.Random(seed)
    E = r.choice([1, 2, 3, 5, 8, 20, 64])
    R = r.choice([d for d in (1, 2, 4) if E % d == 0])
    S, K = int(np.exp(r.uniform(0, np.log(6000)))), r.randint(1, min(E, 4))
    H, N = 128 * r.randint(1, 9), 8 * int(np.exp(r.uniform(0, np.log(80))))
    mode = r.choice([PAD_NONE, PAD_MULTIPLE, PAD_CAPACITY])
    pad = {PAD_NONE: 0, PAD_MULTIPLE: r.choice([8, 100]), PAD_CAPACITY: max(1, S * K // E)}[mode]
    act = r.choice([moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU])
    p = rng.random(E) ** r.choice([0, 3]) + 1e-4
    idx = rng.choice(E, (S, K), p=p / p.sum()).astype(np.int32)
    idx[rng.random((S, K)) < 0.05] = -1
    desc = moe.LayoutDesc(S, K, E, R, mode, pad)
    lay = moe.moe_layout(desc, dev(idx))
    ref = oracle.layout(idx, E, R, mode, pad)
    rows = len(ref.src)
    M = N * (2 if act == moe.MOE_ACT_SWIGLU else 1)
    xc, xs = mx4_random(rng, (rows,), H, 120, 130)
    wc, ws = mx4_random(rng, (E, M), H, 113, 123)
    product_check(moe, desc, lay, expert_of_rows(ref, E, rows), xc, xs, wc, ws, act, exact=False)


@pytest.mark.parametrize("S,E,H,N", [(3000, 4, 1152, 520), (1500, 3, 640, 264), (600, 1, 384, 1032)])
def test_nan_blocks_of_long_segments(moe, S, E, H, N):
    """A NaN block of one token row spoils that row, one of a weight row that channel of its expert; nothing else."""
    rng = np.random.default_rng(S)
    idx = rng.integers(0, E, (S, 2)).astype(np.int32)
    desc = moe.LayoutDesc(S, 2, E, 1)
    lay = moe.moe_layout(desc, dev(idx))
    of_row = expert_of_rows(oracle.layout(idx, E, 1, PAD_NONE, 0), E, 2 * S)
    xc, xs = mx4_random(rng, (2 * S,), H, 120, 130)
    wc, ws = mx4_random(rng, (E, N), H, 113, 123)
    product_check(moe, desc, lay, of_row, xc, xs, wc, ws, moe.MOE_ACT_NONE, exact=False)
    for block in (0, H // 32 - 1):
        for row in (0, 255, 2 * S - 1):
            bad = xs.copy()
            bad[row, block] = 255
            nan = np.isnan(bf16_values(host_bits(moe.moe_expert_gemm_mx4(desc, lay, dev(xc), dev(bad), dev(wc), dev(ws)))))
            assert nan[row].all() and nan.sum() == N
        for n in (0, N - 1):
            bad = ws.copy()
            bad[E - 1, n, block] = 255
            nan = np.isnan(bf16_values(host_bits(moe.moe_expert_gemm_mx4(desc, lay, dev(xc), dev(xs), dev(wc), dev(bad)))))
            assert nan[of_row == E - 1][:, n].all() and nan.sum() == (of_row == E - 1).sum()


@pytest.mark.parametrize("S,N", [(5, 40), (2500, 520)], ids=["short", "long"])
@pytest.mark.parametrize("xlo,wlo", [(0, 253), (253, 0), (40, 213), (0, 128)])
def test_scales_at_both_ends(moe, S, N, xlo, wlo):
    """The lowest scales of one operand against the highest of the other: their product alone counts."""
    rng = np.random.default_rng(S + xlo)
    E, H = 2, 640
    idx = rng.integers(0, E, (S, 2)).astype(np.int32)
    desc = moe.LayoutDesc(S, 2, E, 1)
    lay = moe.moe_layout(desc, dev(idx))
    of_row = expert_of_rows(oracle.layout(idx, E, 1, PAD_NONE, 0), E, 2 * S)
    xc, xs = mx4_random(rng, (2 * S,), H, xlo, xlo + 1)
    wc, ws = mx4_random(rng, (E, N), H, wlo, wlo + 1)
    product_check(moe, desc, lay, of_row, xc, xs, wc, ws, moe.MOE_ACT_NONE, exact=True)
