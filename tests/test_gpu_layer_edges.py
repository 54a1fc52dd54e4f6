"""dispatch, expert_ffn and combine as autograd functions at their edges: no token, no expert with a row, each subset of
gradients, a pass walked twice, a stream of its own, gradients that are no arrays of their own."""
from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

import test_gpu_expert_products as products
from workloads import PAD_CAPACITY, PAD_MULTIPLE, PAD_NONE

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E, H, N = 4, 72, 40


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def leaves(S, K, rows=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(S * 10 + K)

    def leaf(*shape, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV) * 0.2).to(dtype).requires_grad_()

    return leaf(S, H), leaf(E, 2 * N, H), leaf(E, H, N), leaf(S, K, dtype=torch.float32), leaf(S, H)


def layer(moe, desc, lay, t):
    hidden, w_in, w_out, tw, shared = t
    return moe.combine(desc, lay, moe.expert_ffn(desc, lay, moe.dispatch(desc, lay, hidden), w_in, w_out), tw, shared)


@pytest.mark.parametrize("mode,pad", [(PAD_NONE, 0), (PAD_MULTIPLE, 8), (PAD_CAPACITY, 3)])
@pytest.mark.parametrize("S", [0, 5])
def test_nothing_routed(moe, S, mode, pad):
    """The result is the shared output alone, the weights' gradients are zero."""
    K = 2
    desc = moe.LayoutDesc(S, K, E, 2, mode, pad)
    lay = moe.moe_layout(desc, torch.full((S, K), -1, dtype=torch.int32, device=DEV))
    t = leaves(S, K)
    out = layer(moe, desc, lay, t)
    assert torch.equal(out, t[4])
    d = torch.ones_like(out)
    grads = torch.autograd.grad(out, t, d)
    assert all(g.shape == p.shape and g.dtype == p.dtype for g, p in zip(grads, t))
    assert all(bool((g == 0).all()) for g in grads[:4]) and torch.equal(grads[4], d)


@pytest.fixture(scope="module")
def case(moe):
    rng = np.random.default_rng(2)
    c = products.Case(moe, rng, 60, 3, E, 2, PAD_MULTIPLE, 8)
    t = leaves(60, 3)
    d = torch.randn((60, H), device=DEV).bfloat16()
    out = layer(moe, c.desc, c.lay, t)
    return c, t, d, out, torch.autograd.grad(out, t, d, retain_graph=True)


@pytest.mark.parametrize("wanted", [w for n in (1, 2) for w in itertools.combinations(range(5), n)], ids=str)
def test_each_subset_of_gradients(moe, case, wanted):
    c, t, d, out, want = case
    own = [p.detach().requires_grad_(i in wanted) for i, p in enumerate(t)]
    got = layer(moe, c.desc, c.lay, own)
    assert torch.equal(got, out)
    for i, g in zip(wanted, torch.autograd.grad(got, [own[i] for i in wanted], d)):
        assert torch.equal(g, want[i])


def test_walked_twice(moe, case):
    c, t, d, out, want = case
    for _ in range(2):
        for a, b in zip(torch.autograd.grad(out, t, d, retain_graph=True), want):
            assert torch.equal(a, b)


def test_one_value_for_every_gradient(moe, case):
    """A sum's gradient is one element seen everywhere, and a transposed one has strides of its own."""
    c, t, d, out, _ = case
    ones = torch.autograd.grad(out, t, torch.ones_like(out), retain_graph=True)
    for a, b in zip(torch.autograd.grad(out.sum(), t, retain_graph=True), ones):
        assert torch.equal(a, b)
    strided = d.t().contiguous().t()
    assert not strided.is_contiguous()
    for a, b in zip(torch.autograd.grad(out, t, strided, retain_graph=True), case[4]):
        assert torch.equal(a, b)


def test_on_another_stream(moe, case):
    c, t, d, out, want = case
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        own = [p.detach().clone().requires_grad_() for p in t]
        got = layer(moe, c.desc, c.lay, own)
        grads = torch.autograd.grad(got, own, d)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, out)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_one_rows_tensor_used_twice(moe, case):
    """Rows that two blocks read get both gradients."""
    c, t, d, _, _ = case
    hidden, w_in, w_out, tw, _ = (p.detach().requires_grad_() for p in t)
    rows = moe.dispatch(c.desc, c.lay, hidden)
    y = moe.expert_ffn(c.desc, c.lay, rows, w_in, w_out) + moe.expert_ffn(c.desc, c.lay, rows, w_in, w_out)
    dy = torch.randn(y.shape, device=DEV).bfloat16()
    both = torch.autograd.grad(y, (rows, w_in, w_out), dy, retain_graph=True)
    one = torch.autograd.grad(moe.expert_ffn(c.desc, c.lay, rows, w_in, w_out), (rows, w_in, w_out), dy, retain_graph=True)
    # twice a bf16 value is exact
    assert all(torch.equal(a, 2 * b) for a, b in zip(both, one))
