"""Router, balance loss and their gradients on the GPU against the 64-bit reference.

Tolerances, in steps u = 2^-24 (half a unit of fp32, relative).  A probability
is exp(z - max) over a sum of E of them: the difference has one rounding, which
the exponential turns into |z - max| u; the exponential itself, within one unit
(2u); a lane's V <= 16 terms and 6 wave steps of the sum, of positive terms
(22u); the reciprocal and the product (2u).  With |z - max| <= 40 for anything
above e^-40 of the largest, that is under 66u + 2u for what is dropped below:
REL = 80u covers p and the weights.  (An exponential may come out as a
subnormal or zero where the exact one is below 2^-126: ABS.)  The loss adds up
to 16 probabilities per wave and 4 waves in fp32 (20u), then in 64 bits, rounds
coefficients once and itself once: 2*REL.  A gradient element is a difference
of products of such numbers: 4*REL relative to the sum of its terms' sizes,
plus the rounding to its type (half a unit: 2^-8 for bf16, 2^-24 for fp32).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from router_mx4_reference import router_gradient, router_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
REL, ABS = 80 * U, 2.0 ** -120


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def close(got, want, rel, size=None, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    ok = ~np.isnan(want)
    bound = rel * np.abs(want if size is None else size) + ABS
    off = np.abs(got - want)
    assert np.all(off[ok] <= bound[ok]), f"{what}: off by {np.max((off / bound)[ok]):.3g} of the bound"


def check(moe, z, K, mask=None, given=None, d_w=True, d_loss=True, rng=None, **kw):
    """One forward and backward pass against the reference.  z: torch tensor on the device."""
    S, E = z.shape
    bf16 = z.dtype == torch.bfloat16
    desc = moe.RouterDesc(S, E, K, **kw)
    z64 = z.double().cpu().numpy()
    m = None if mask is None else torch.from_numpy(mask).to(DEV)
    ref = router_reference(z64, K, mask=mask, given=given, **kw)
    before = z.clone()
    if given is None:
        r = moe.moe_router(desc, z, m)
        assert np.array_equal(r.topk_idx.cpu().numpy(), ref["idx"]), "picks"
        close(r.topk_w.cpu(), ref["w"], REL, what="weights")
        serving = moe.moe_router(desc, z, m, loss=False)
        assert torch.equal(serving.topk_idx, r.topk_idx) and torch.equal(serving.topk_w, r.topk_w)
    else:
        r = moe.moe_balance_loss(desc, z, torch.from_numpy(given.astype(np.int32)).to(DEV), m)
    assert np.array_equal(r.expert_count.cpu().numpy(), ref["count"]), "counts"
    close(r.balance_coef.cpu(), ref["coef"], 2 * REL, what="coef")
    close(r.balance_loss.cpu(), [ref["loss"]], 2 * REL, what="loss")
    rng = rng or np.random.default_rng(7)
    gw = rng.standard_normal((S, K)).astype(np.float32) if d_w and given is None else None
    gl = np.float32(1.7) if d_loss else None
    renorm = kw.get("renorm", True)
    want, size = router_gradient(ref, z64, renorm, kw.get("seq_len", 0), gw, gl)
    got = moe.moe_router_backward(desc, z, r, None if gw is None else torch.from_numpy(gw).to(DEV),
                                  None if gl is None else torch.full((1,), float(gl), device=DEV), m)
    assert got.dtype == z.dtype
    g = got.double().cpu().numpy()
    # the rounding to the gradient's type is relative to its value, the rest to the terms
    rnd = (2.0 ** -8 if bf16 else U) * np.abs(want) + (2.0 ** -133 if bf16 else 0.0)
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = ~np.isnan(want)
    bound = 4 * REL * size + rnd + ABS
    assert np.all(np.abs(g - want)[ok] <= bound[ok]), f"gradient: {np.max((np.abs(g - want) / bound)[ok]):.3g} of the bound"
    assert torch.equal(before.view(torch.int16 if bf16 else torch.int32), z.view(torch.int16 if bf16 else torch.int32))
    return r, got


SHAPES = [
    # S, E, K, keywords
    (1, 1, 1, {}),
    (1, 8, 8, {}),
    (3, 60, 4, dict(renorm=False)),
    (5, 64, 6, dict(alpha=0.01)),
    (16, 65, 2, {}),
    (17, 128, 16, dict(renorm=False)),
    (33, 130, 5, {}),
    (129, 256, 8, dict(n_groups=8, topk_groups=4)),
    (64, 255, 8, dict(n_groups=5, topk_groups=2, renorm=False)),
    (100, 385, 7, dict(n_groups=11, topk_groups=3)),
    (48, 512, 8, dict(n_groups=64, topk_groups=9)),
    (31, 1000, 16, dict(n_groups=8, topk_groups=8)),
    (64, 1024, 2, dict(n_groups=64, topk_groups=1, renorm=False)),
    (96, 96, 3, dict(seq_len=1)),
    (600, 48, 2, dict(seq_len=300, renorm=False)),
    (1200, 24, 3, dict(seq_len=24, alpha=3.0)),
    (5000, 16, 4, {}),
    (4608, 64, 6, dict(seq_len=1536)),
    (2100, 48, 2, dict(seq_len=1)),          # more parts of the loss than the last workgroup adds
    (9000, 8, 2, dict(seq_len=1, renorm=False)),   # more sequences than it counts
    (18000, 40, 3, dict(seq_len=9000)),      # more tokens than workgroups' waves
]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("S,E,K,kw", SHAPES, ids=[f"{s}x{e}k{k}" for s, e, k, _ in SHAPES])
def test_router(moe, S, E, K, kw, bf16):
    g = torch.Generator().manual_seed(S * 1031 + E)
    z = (torch.randn((S, E), generator=g) * 2).to(torch.bfloat16 if bf16 else torch.float32).to(DEV)
    check(moe, z, K, **kw)


@pytest.mark.parametrize("S,E,K,kw", SHAPES, ids=[f"{s}x{e}k{k}" for s, e, k, _ in SHAPES])
def test_balance_loss_of_a_given_routing(moe, S, E, K, kw):
    """Ids outside the experts count for nothing, repeated ones twice."""
    rng = np.random.default_rng(S + E)
    z = torch.from_numpy(rng.standard_normal((S, E)).astype(np.float32)).to(DEV)
    given = rng.integers(-2, E + 2, (S, K))
    mask = rng.random(S) < 0.8
    check(moe, z, K, mask=mask, given=given, **{k: v for k, v in kw.items() if k in ("seq_len", "alpha")})


def test_balance_loss_with_more_picks_than_experts(moe):
    rng = np.random.default_rng(1)
    z = torch.from_numpy(rng.standard_normal((40, 3)).astype(np.float32)).to(DEV)
    check(moe, z, 16, given=rng.integers(0, 3, (40, 16)))


@pytest.mark.parametrize("part", ["weights", "loss"])
@pytest.mark.parametrize("renorm", [True, False])
def test_one_gradient_alone(moe, part, renorm):
    z = torch.randn((70, 72), generator=torch.Generator().manual_seed(3)).to(DEV)
    check(moe, z, 5, d_w=part == "weights", d_loss=part == "loss", renorm=renorm, n_groups=4, topk_groups=2)


def test_ties_go_to_the_lower_index(moe):
    """Logits of three values, -0 and +0 among them, so that groups and picks tie everywhere."""
    rng = np.random.default_rng(5)
    z = torch.from_numpy(rng.choice(np.array([0.0, -0.0, 1.0], np.float32), (200, 96))).to(DEV)
    for kw in (dict(), dict(n_groups=8, topk_groups=3), dict(n_groups=32, topk_groups=8, renorm=False)):
        check(moe, z, 8, **kw)


def test_experts_and_rows_at_minus_infinity(moe):
    """Fewer pickable experts than picks, none at all, a whole group out, and the type's lowest value."""
    rng = np.random.default_rng(6)
    z = rng.standard_normal((64, 40)).astype(np.float32)
    z[0] = -np.inf                                     # nothing to pick: the token does not count
    z[1] = -np.inf
    z[1, 17] = 0.25                                    # one pick, the rest empty
    z[2, :] = np.finfo(np.float32).min                 # every logit the lowest: uniform
    z[3, 1:] = np.finfo(np.float32).min
    z[4, ::2] = -np.inf
    z[5:30, 8:16] = -np.inf
    z[6, 0] = np.finfo(np.float32).max
    mask = np.ones(64, bool)
    mask[40:50] = False
    for renorm in (True, False):
        for kw in (dict(), dict(n_groups=5, topk_groups=2), dict(n_groups=5, topk_groups=2, seq_len=16)):
            check(moe, torch.from_numpy(z).to(DEV), 6, mask=mask, renorm=renorm, **kw)
    zb = torch.from_numpy(z).to(torch.bfloat16).to(DEV)
    zb[7, 3:] = torch.finfo(torch.bfloat16).min
    check(moe, zb, 6, mask=mask)


def test_masked_tokens_may_hold_anything(moe):
    rng = np.random.default_rng(8)
    z = rng.standard_normal((96, 32)).astype(np.float32)
    mask = rng.random(96) < 0.6
    mask[32:64] = False                                # a sequence without a token
    z[~mask] = np.array([np.nan, np.inf, -np.inf, 3e38] * 8, np.float32)
    r, d = check(moe, torch.from_numpy(z).to(DEV), 4, mask=mask, seq_len=32)
    assert (r.topk_idx.cpu().numpy()[~mask] == -1).all() and not d.cpu().numpy()[~mask].any()
    assert torch.isfinite(r.balance_loss).all()
    # no token at all
    r, d = check(moe, torch.from_numpy(z).to(DEV), 4, mask=np.zeros(96, bool))
    assert float(r.balance_loss) == 0.0 and not d.any()


def test_broken_tokens_show(moe):
    """A NaN or +inf in a token that counts: not routed, NaN loss, NaN row of the gradient, other rows as ever."""
    rng = np.random.default_rng(9)
    z = rng.standard_normal((20, 130)).astype(np.float32)
    z[3, 129] = np.nan
    z[11, 0] = np.inf
    z[12, :] = np.nan
    for kw in (dict(), dict(renorm=False, n_groups=10, topk_groups=3)):
        r, d = check(moe, torch.from_numpy(z).to(DEV), 4, **kw)
        assert np.isnan(float(r.balance_loss))
        assert torch.isnan(d).all(1).nonzero().flatten().tolist() == [3, 11, 12]
    check(moe, torch.from_numpy(z).to(DEV), 4, given=rng.integers(0, 130, (20, 4)))


def test_gradients_of_entries_without_a_pick_are_not_read(moe):
    z = torch.full((2, 8), -np.inf, device=DEV)
    z[0, 2] = 1.0
    desc = moe.RouterDesc(2, 8, 3, alpha=0.0)
    r = moe.moe_router(desc, z)
    assert r.topk_idx.tolist() == [[2, -1, -1], [-1, -1, -1]] and r.topk_w.tolist() == [[1.0, 0.0, 0.0], [0.0] * 3]
    dw = torch.tensor([[1.0, np.nan, np.nan], [np.nan] * 3], dtype=torch.float32, device=DEV)
    assert not moe.moe_router_backward(desc, z, r, dw).any()


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_rows_off_the_vector_grid(moe, bf16):
    """Logits and gradient that start one element off a 16-byte boundary."""
    t = torch.bfloat16 if bf16 else torch.float32
    base = torch.randn(20 * 256 + 1, generator=torch.Generator().manual_seed(2)).to(t).to(DEV)
    z = base[1:].view(20, 256)
    assert z.data_ptr() % 16
    r, d = check(moe, z, 8, n_groups=8, topk_groups=4)
    out = torch.full((20 * 256 + 2,), 7.0, dtype=t, device=DEV)
    desc = moe.RouterDesc(20, 256, 8, n_groups=8, topk_groups=4)
    moe.moe_router_backward(desc, z, r, d_loss=torch.ones(1, device=DEV), d_logits=out[1:-1].view(20, 256))
    assert float(out[0]) == 7.0 and float(out[-1]) == 7.0


def test_gradient_over_the_logits(moe):
    """d_logits may be the logits' own buffer."""
    z = torch.randn((50, 300), generator=torch.Generator().manual_seed(4)).to(DEV)
    desc = moe.RouterDesc(50, 300, 4)
    r = moe.moe_router(desc, z)
    dl = torch.ones(1, device=DEV)
    want = moe.moe_router_backward(desc, z, r, d_loss=dl)
    moe.moe_router_backward(desc, z, r, d_loss=dl, d_logits=z)
    assert torch.equal(z, want)


def test_empty_batches(moe):
    z = torch.empty((0, 16), device=DEV)
    r = moe.moe_router(moe.RouterDesc(0, 16, 2), z)
    assert float(r.balance_loss) == 0.0 and not r.expert_count.any() and not r.balance_coef.any()
    r = moe.moe_router(moe.RouterDesc(0, 16, 2, seq_len=8), z)
    assert float(r.balance_loss) == 0.0 and r.expert_count.shape == (0, 16)
    assert moe.moe_router_backward(moe.RouterDesc(0, 16, 2), z, moe.moe_router(moe.RouterDesc(0, 16, 2), z),
                                   d_loss=torch.ones(1, device=DEV)).shape == (0, 16)


def test_same_bits_every_time_and_on_any_stream(moe):
    z = torch.randn((3000, 256), generator=torch.Generator().manual_seed(12)).to(DEV)
    desc = moe.RouterDesc(3000, 256, 8, seq_len=1000)
    dw, dl = torch.randn((3000, 8), generator=torch.Generator().manual_seed(13)).to(DEV), torch.ones(1, device=DEV)
    r0 = moe.moe_router(desc, z)
    d0 = moe.moe_router_backward(desc, z, r0, dw, dl)
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in side:                                     # two calls at once, each with its own workspace
        r = moe.moe_router(desc, z, stream=s)
        got.append((r, moe.moe_router_backward(desc, z, r, dw, dl, stream=s)))
    torch.cuda.synchronize()
    for r, d in got:
        assert torch.equal(r.topk_idx, r0.topk_idx) and torch.equal(r.topk_w, r0.topk_w)
        assert torch.equal(r.balance_loss, r0.balance_loss) and torch.equal(r.balance_coef, r0.balance_coef)
        assert torch.equal(d, d0)


def test_graph_replay(moe):
    """Forward and backward captured once, replayed with new logits between; eager calls in between."""
    desc = moe.RouterDesc(700, 64, 6, seq_len=350, alpha=0.1)
    z = torch.randn((700, 64), device=DEV)
    dw, dl = torch.randn((700, 6), device=DEV), torch.ones(1, device=DEV)
    r = moe.alloc_router(desc, torch.device(DEV))
    out = torch.empty_like(z)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_router(desc, z, router=r)
        moe.moe_router_backward(desc, z, r, dw, dl, d_logits=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_router(desc, z, router=r)
        moe.moe_router_backward(desc, z, r, dw, dl, d_logits=out)
    for k in range(4):
        z.copy_(torch.randn((700, 64), generator=torch.Generator().manual_seed(20 + k)))
        graph.replay()
        torch.cuda.synchronize()
        e = moe.moe_router(desc, z)
        assert torch.equal(e.topk_idx, r.topk_idx) and torch.equal(e.topk_w, r.topk_w)
        assert torch.equal(e.expert_count, r.expert_count) and torch.equal(e.balance_loss, r.balance_loss)
        assert torch.equal(moe.moe_router_backward(desc, z, e, dw, dl), out)


def test_autograd(moe):
    """router and balance_loss inside a graph of other operations, against the calls they are made of."""
    z = torch.randn((60, 32), generator=torch.Generator().manual_seed(30)).to(DEV)
    desc = moe.RouterDesc(60, 32, 4, n_groups=4, topk_groups=2, seq_len=20, alpha=0.5)
    leaf = z.clone().requires_grad_()
    idx, w, loss, count = moe.router(desc, leaf * 2.0)
    assert not idx.requires_grad and not count.requires_grad and loss.shape == ()
    r = moe.moe_router(desc, z * 2.0)
    assert torch.equal(idx, r.topk_idx) and torch.equal(w, r.topk_w) and torch.equal(loss.view(1), r.balance_loss)
    (w.square().sum() + 3.0 * loss).backward()
    want = moe.moe_router_backward(desc, z * 2.0, r, 2.0 * r.topk_w, torch.full((1,), 3.0, device=DEV))
    assert torch.equal(leaf.grad, 2.0 * want)
    # each output alone; a bf16 leaf
    for pick in (0, 1):
        leaf = z.to(torch.bfloat16).requires_grad_()
        _, w, loss, _ = moe.router(desc, leaf)
        (w * 2.0).sum().backward() if pick == 0 else loss.backward()
        r = moe.moe_router(desc, z.to(torch.bfloat16))
        want = moe.moe_router_backward(desc, z.to(torch.bfloat16), r, torch.full_like(r.topk_w, 2.0) if pick == 0 else None,
                                       None if pick == 0 else torch.ones(1, device=DEV))
        assert torch.equal(leaf.grad, want)
    leaf = z.clone().requires_grad_()
    loss, count = moe.balance_loss(desc, leaf, idx)
    loss.backward()
    r = moe.moe_balance_loss(desc, z, idx)
    assert torch.equal(leaf.grad, moe.moe_router_backward(desc, z, r, d_loss=torch.ones(1, device=DEV)))
    assert torch.equal(count, r.expert_count)


def test_autograd_twice_and_not_at_all(moe, monkeypatch):
    """A graph walked twice, gradients that add up, leaves that need none, and a backward pass under capture."""
    z = torch.randn((33, 24), generator=torch.Generator().manual_seed(31)).to(DEV)
    desc = moe.RouterDesc(33, 24, 3, alpha=2.0)
    r = moe.moe_router(desc, z)
    once = moe.moe_router_backward(desc, z, r, torch.ones_like(r.topk_w), torch.ones(1, device=DEV))
    leaf = z.clone().requires_grad_()
    _, w, loss, _ = moe.router(desc, leaf)
    total = w.sum() + loss                                # the sum's gradient comes expanded, not contiguous
    total.backward(retain_graph=True)
    assert torch.equal(leaf.grad, once)
    total.backward(retain_graph=True)
    assert torch.equal(leaf.grad, once + once)
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="captured"):
            total.backward()
    with torch.no_grad():
        _, w, loss, _ = moe.router(desc, leaf)
    assert not w.requires_grad and not loss.requires_grad
    _, w, loss, _ = moe.router(desc, z)
    assert not w.requires_grad and not loss.requires_grad


def test_python_refusals(moe):
    z = torch.zeros((4, 8), device=DEV)
    desc = moe.RouterDesc(4, 8, 2)
    with pytest.raises(TypeError):
        moe.moe_router(desc, z.half())
    with pytest.raises(ValueError):
        moe.moe_router(desc, z.t().contiguous())
    with pytest.raises(ValueError):
        moe.moe_router(desc, torch.zeros((8, 4), device=DEV).t())
    with pytest.raises(ValueError):
        moe.moe_router(desc, z, token_mask=torch.ones(3, dtype=torch.bool, device=DEV))
    with pytest.raises(TypeError):
        moe.moe_router(desc, z, token_mask=torch.ones(4, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_router(moe.RouterDesc(4, 8, 9), z)
    r = moe.moe_router(desc, z, loss=False)
    with pytest.raises(ValueError):
        moe.moe_router_backward(desc, z, r, d_loss=torch.ones(1, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_router_backward(desc, z, r)
    with pytest.raises(ValueError):
        moe.moe_router(desc, z, router=r)              # no buffers for the loss
    with pytest.raises(TypeError):
        moe.moe_balance_loss(desc, z, torch.zeros((4, 2), dtype=torch.int64, device=DEV))
