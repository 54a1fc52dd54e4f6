"""Arrays whose bytes pass 2^32: the router's logits and gradient, the MXFP4 dispatch's receive rows and their conversion
by layout.  Rows repeat, so that a small call says what the last ones hold."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from parity_helpers import dev_bf16, host_bits
from router_mx4_reference import bf16_values, mx4_quantize, mx4_values
from workloads import normal_bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def test_router(moe):
    n, E, K, reps = 1024, 1000, 4, 1100
    S = n * reps
    assert S * E * 4 > 1 << 32
    z = torch.randn((n, E), generator=torch.Generator().manual_seed(3)).to(DEV)
    small = moe.moe_router(moe.RouterDesc(n, E, K, n_groups=8, topk_groups=3), z)
    desc = moe.RouterDesc(S, E, K, n_groups=8, topk_groups=3, seq_len=n)
    big = z.repeat(reps, 1)
    r = moe.moe_router(desc, big)
    serving = moe.moe_router(desc, big, loss=False)
    for at in (0, 1, reps // 2, reps - 1):
        rows = slice(at * n, (at + 1) * n)
        assert torch.equal(r.topk_idx[rows], small.topk_idx) and torch.equal(r.topk_w[rows], small.topk_w)
        assert torch.equal(serving.topk_idx[rows], small.topk_idx) and torch.equal(serving.topk_w[rows], small.topk_w)
        assert torch.equal(r.expert_count[at], small.expert_count[0])
    # every sequence has the same loss, and the coefficients share it out: each is rounded once (2^-24)
    assert torch.all((r.balance_coef.double() * reps - small.balance_coef.double()).abs() <= 2.0 ** -23 * small.balance_coef)
    assert abs(float(r.balance_loss) - float(small.balance_loss)) <= 2.0 ** -22 * float(small.balance_loss)
    dw = torch.randn((n, K), generator=torch.Generator().manual_seed(4)).to(DEV)
    want = moe.moe_router_backward(moe.RouterDesc(n, E, K), z, small, d_topk_w=dw)
    got = moe.moe_router_backward(desc, big, r, d_topk_w=dw.repeat(reps, 1))
    for at in (0, reps // 2, reps - 1):
        assert torch.equal(got[at * n:(at + 1) * n], want)


def test_dispatch_and_conversions_by_layout(moe):
    n, reps, K, E, H = 500, 320, 8, 16, 7168
    S = n * reps
    assert S * K * (H // 2) > 1 << 32
    rng = np.random.default_rng(2)
    bits = normal_bf16_bits(rng, (n, H))
    hid = dev_bf16(bits, DEV).repeat(reps, 1)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(S)]).astype(np.int32)).to(DEV)
    desc = moe.LayoutDesc(S, K, E, 2)
    lay = moe.moe_layout(desc, idx)
    recv, scales, _ = moe.moe_dispatch_mx4(desc, lay, hid)
    del hid
    wc, ws = mx4_quantize(bf16_values(bits))
    out = moe.moe_dequantize_mx4(recv, scales, layout=lay)
    again = moe.moe_quantize_mx4(out, layout=lay)
    rows = S * K
    for first in (0, rows // 2, rows - 300):
        part = slice(first, first + 300)
        token = lay.src[part].cpu().numpy() // K % n
        assert np.array_equal(recv[part].cpu().numpy(), wc[token]) and np.array_equal(scales[part].cpu().numpy(), ws[token])
        v = mx4_values(wc[token], ws[token])
        assert np.array_equal(bf16_values(host_bits(out[part])), v)
        # a block's largest magnitude became 4 or 6, which has the same scale: a second rounding changes nothing
        c, s = (t[part].cpu().numpy() for t in again)
        assert np.array_equal(mx4_values(c, s), v)
