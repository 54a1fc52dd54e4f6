"""The gradients of the experts' block, of a plain product and of combine against differences of their forward calls.

The GPU tests compare the calls with each other alone.  On the CPU the same comparison runs on the formulas in 64 bits, with
mistakes planted in the gradient: it has to find every one."""
from __future__ import annotations

import numpy as np
import pytest

import gradient_differences as gd
import oracle
from expert_products_reference import expert_of_rows, silu
from router_mx4_reference import bf16_values
from workloads import PAD_CAPACITY, PAD_MULTIPLE, PAD_NONE

NAMES = ("x", "w_in", "w_out")
# S, K, E, H, N, pad mode, pad rows
SHAPES = [(14, 2, 5, 24, 16, PAD_MULTIPLE, 8), (1, 2, 3, 24, 8, PAD_NONE, 0), (9, 3, 4, 40, 24, PAD_CAPACITY, 5)]
shapes = pytest.mark.parametrize("S,K,E,H,N,mode,pad", SHAPES, ids=[f"{p[0]}x{p[1]}e{p[2]}h{p[3]}n{p[4]}" for p in SHAPES])
names = pytest.mark.parametrize("name", NAMES)
FAR = 12       # a direction's derivative, in bounds


def case(S, K, E, H, N, mode, pad):
    rng = np.random.default_rng(S * 100 + H)
    idx = np.stack([rng.permutation(E)[:K] for _ in range(S)]).astype(np.int32)
    idx[rng.random((S, K)) < 0.1] = -1
    lay = oracle.layout(idx, E, 1, mode, pad)
    of_row = expert_of_rows(lay, E, len(lay.src))
    return idx, of_row, gd.inputs(rng, len(of_row), E, H, N)


def differs(gradient, s, up, down, tolerance):
    """Whether the gradient is further from the difference than the bound allows."""
    return abs((up - down) / 2 - float((gradient * s).sum())) > tolerance


def sides(v, of_row, name, s, block):
    return [gd.loss(block(dict(v, **{name: v[name] + sign * s}), of_row), v, of_row) for sign in (1, -1)]


@names
@shapes
def test_finds_mistakes(S, K, E, H, N, mode, pad, name):
    _, of_row, v = case(S, K, E, H, N, mode, pad)
    s = gd.direction(v, of_row, name)
    tolerance = gd.bound(v, of_row, name, s)
    right = gd.gradients(v, of_row)[0][name]
    assert (np.abs(right * s)).sum() > FAR * tolerance
    up, down = sides(v, of_row, name, s, gd.rounded_block)
    assert not differs(right, s, up, down, tolerance)
    up, down = sides(v, of_row, name, s, lambda *a: gd.block(*a)[3])
    assert not differs(right, s, up, down, tolerance)
    wrong = {"zero": 0 * right, "sign": -right, "a quarter more": 1.25 * right, "half": right / 2}
    if name != "w_out":
        wrong["no slope"] = gd.gradients(v, of_row, slope=lambda g: silu(g))[0][name]
        wrong["no up gradient"] = gd.gradients(dict(v), of_row, slope=lambda g: 0 * g)[0][name]
    if name == "w_in":
        wrong["halves swapped"] = np.roll(right, N, 1)
    if name == "w_out":
        wrong["experts shifted"] = np.roll(right, 1, 0)
    for what, gradient in wrong.items():
        assert differs(gradient, s, up, down, tolerance), what


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------

DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def dev_values(v, held=None):
    """Values that bf16 holds -> a device tensor; NaN in rows that hold no entry."""
    import torch
    from parity_helpers import dev_bf16
    bits = (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    assert np.array_equal(bf16_values(bits), v)
    if held is not None:
        bits = np.where(held[:, None], bits, 0x7FA5).astype(np.uint16)
    return dev_bf16(bits, DEV)


def host_values(t):
    from parity_helpers import host_bits
    return bf16_values(host_bits(t.detach()))


@pytest.mark.gpu
@names
@shapes
def test_experts(moe, S, K, E, H, N, mode, pad, name):
    """expert_ffn, forward at two points and backward between them."""
    import torch
    idx, of_row, v = case(S, K, E, H, N, mode, pad)
    held = of_row >= 0
    desc = moe.LayoutDesc(S, K, E, 1, mode, pad)
    lay = moe.moe_layout(desc, torch.from_numpy(idx).to(DEV))

    def leaves(p):
        return {k: dev_values(p[k], held if k == "x" else None).requires_grad_() for k in NAMES}

    def block(p, _):
        with torch.no_grad():
            return host_values(moe.expert_ffn(desc, lay, **leaves(p)))[held]

    s = gd.direction(v, of_row, name)
    tolerance = gd.bound(v, of_row, name, s)
    at = leaves(v)
    y = moe.expert_ffn(desc, lay, **at)
    grads = dict(zip(NAMES, torch.autograd.grad(y, [at[k] for k in NAMES], dev_values(v["dy"], held))))
    got = host_values(grads[name])
    assert np.abs((got * s).sum()) > FAR / 2 * tolerance
    assert not differs(got, s, *sides(v, of_row, name, s, block), tolerance)


def whole(rng, shape, most):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


@pytest.mark.gpu
@pytest.mark.parametrize("S,K,E,H,N,mode,pad", [(60, 2, 5, 64, 24, PAD_MULTIPLE, 8), (700, 2, 3, 40, 136, PAD_NONE, 0), (1, 1, 1, 8, 8, PAD_NONE, 0)])
def test_product_exactly(moe, S, K, E, H, N, mode, pad):
    """A plain product is linear in either argument, and with whole numbers up to 128 bf16 holds every result: the
    difference equals the gradient."""
    import torch
    rng = np.random.default_rng(S)
    idx = rng.integers(0, E, (S, K)).astype(np.int32)
    desc = moe.LayoutDesc(S, K, E, 1, mode, pad)
    lay = moe.moe_layout(desc, torch.from_numpy(idx).to(DEV))
    ref = oracle.layout(idx, E, 1, mode, pad)
    of_row = expert_of_rows(ref, E, len(ref.src))
    held = of_row >= 0
    x, w, d = whole(rng, (len(held), H), 1), whole(rng, (E, N, H), 1), whole(rng, (len(held), N), 1)
    X, W, D = dev_values(x, held), dev_values(w), dev_values(d, held)

    def loss(x, w):
        y = host_values(moe.moe_expert_gemm(desc, lay, dev_values(x, held), dev_values(w)))[held]
        assert np.abs(y).max() <= 2 * H <= 256
        return float((y * d[held]).sum())

    dw = moe.moe_expert_gemm_backward_w(desc, lay, D, X, dtype=torch.float32).cpu().numpy().astype(np.float64)
    dx = host_values(moe.moe_expert_gemm_backward_x(desc, lay, D, W))
    dx[~held] = 0
    for gradient, points in ((dw, lambda s: (loss(x, w + s), loss(x, w - s))), (dx, lambda s: (loss(x + s, w), loss(x - s, w)))):
        s = np.sign(gradient)
        up, down = points(s)
        # every term is a whole number: no part of the sum is lost, and none of it cancels
        assert (up - down) / 2 == float(np.abs(gradient).sum()) > 0


@pytest.mark.gpu
def test_combine_exactly(moe):
    """combine is linear in its rows and in its weights; multiples of 1/4 up to 64 are held by bf16."""
    import torch
    rng = np.random.default_rng(4)
    S, K, E, H = 50, 3, 6, 72
    idx = rng.integers(0, E, (S, K)).astype(np.int32)
    idx[rng.random((S, K)) < 0.1] = -1
    desc = moe.LayoutDesc(S, K, E, 2, PAD_MULTIPLE, 4)
    lay = moe.moe_layout(desc, torch.from_numpy(idx).to(DEV))
    held = lay.src.cpu().numpy() >= 0
    y, d, shared = whole(rng, (len(held), H), 4), whole(rng, (S, H), 2), whole(rng, (S, H), 4)
    w = rng.integers(1, 5, (S, K)) / 4.0

    def weights(w):
        return torch.from_numpy(w.astype(np.float32)).to(DEV)

    def loss(y, w, shared):
        out = host_values(moe.moe_combine(desc, lay, dev_values(y, held), weights(w), dev_values(shared)))
        assert np.abs(out).max() <= 64
        return float((out * d).sum())

    leaves = (dev_values(y, held).requires_grad_(), weights(w).requires_grad_(), dev_values(shared).requires_grad_())
    grads = torch.autograd.grad(moe.combine(desc, lay, *leaves), leaves, dev_values(d))
    dy, dw, ds = host_values(grads[0]), grads[1].cpu().numpy().astype(np.float64), host_values(grads[2])
    assert (dy[~held] == 0).all()
    for gradient, points in ((dy, lambda s: (loss(y + s, w, shared), loss(y - s, w, shared))),
                             (dw, lambda s: (loss(y, w + s / 4, shared), loss(y, w - s / 4, shared))),
                             (ds, lambda s: (loss(y, w, shared + s), loss(y, w, shared - s)))):
        up, down = points(np.sign(gradient))
        step = 0.25 if gradient is dw else 1.0
        assert (up - down) / 2 == float(np.abs(gradient).sum()) * step > 0
