"""The experts' products in bf16 and 8-bit integers and their gradients on the GPU.

With small whole numbers times a power of two every product and every sum is
exact in fp32 in any order (a sum stays under 2^24 units), so a result that is
rounded once has to equal the rounded exact one, bit for bit.  With arbitrary
values a sum's error is bounded by 2^-23 of the sum of absolute products for
each instruction (32 terms) and each of the few joins, and 8 more for the
instruction's own tree: (terms/32 + 16) * 2^-23 * size.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import expert_products_reference as ref64
import oracle
from parity_helpers import POISON_BF16, dev_bf16, host_bits
from router_mx4_reference import bf16_values, to_bf16
from workloads import PAD_CAPACITY, PAD_MULTIPLE, PAD_NONE, normal_bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -23


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def whole(rng, shape, most=4, step=1.0):
    """Whole numbers up to `most` times `step`, as bf16 bits and as values."""
    v = rng.integers(-most, most + 1, shape) * step
    return to_bits(v), v


def to_bits(v):
    """Values that bf16 holds exactly -> bits."""
    return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def routing(rng, S, K, E):
    """A few experts get most rows, some none; some ids are no expert."""
    p = rng.random(E) ** 3 + 1e-4
    idx = rng.choice(E, (S, K), p=p / p.sum()).astype(np.int32)
    idx[rng.random((S, K)) < 0.05] = -1
    return idx


class Case:
    """A layout with its rows' experts; row arrays hold NaN where a row holds no entry."""

    def __init__(self, moe, rng, S, K, E, R, mode=PAD_NONE, pad=0, slots=None):
        self.idx = routing(rng, S, K, E)
        self.E, self.desc = E, moe.LayoutDesc(S, K, E, R, mode, pad)
        self.kw = {}
        if slots is None:
            self.lay = moe.moe_layout(self.desc, dev(self.idx))
            l = oracle.layout(self.idx, E, R, mode, pad)
            self.rows = len(l.src)
            self.of_row = ref64.expert_of_rows(l, E, self.rows)
        else:
            self.lay, bal = moe.moe_layout_balanced(self.desc, slots, dev(self.idx))
            src = self.lay.src.cpu().numpy()
            self.rows = S * K
            self.of_row = np.where(src >= 0, self.idx.reshape(-1)[np.maximum(src, 0)], -1)
            self.kw = dict(balance=bal, slots_per_rank=slots)
        self.held = self.of_row >= 0

    def poisoned(self, bits):
        return dev_bf16(np.where(self.held[:, None], bits, POISON_BF16).astype(np.uint16), DEV)

    def out(self, width):
        return torch.full((self.rows + 1, width), 7.0, dtype=torch.bfloat16, device=DEV)

    def result(self, out):
        """Bits of the rows that hold an entry; the others have to be as they were."""
        bits = host_bits(out)
        got = bf16_values(bits)
        assert (got[:self.rows][~self.held] == 7.0).all() and (got[self.rows:] == 7.0).all(), "a row without an entry was written"
        return bits[:self.rows][self.held]


def within(got_bits, want, bound):
    """bound on the value before the rounding to bf16, which is off by half a step at most."""
    got = bf16_values(got_bits)
    limit = bound + 2.0 ** -8 * (np.abs(want) + bound) + 2.0 ** -126
    assert got.shape == want.shape and np.isfinite(got).all()
    off = np.abs(got - want)
    assert np.all(off <= limit), f"off by {np.max(off / limit):.3g} of the bound"


def silu_bound(g, u, g_err=0.0, u_err=0.0):
    """Of silu(g) * u in fp32, g and u off by so much: silu's slope lies within [-0.1, 1.1], and the hardware's
    exponential and reciprocal and the products take (8 + |g|) units."""
    s = np.abs(ref64.silu(g))
    return 1.1 * g_err * np.abs(u) + (s + 1.1 * g_err) * u_err + (8 + np.abs(g)) * U * s * np.abs(u)


def slope_bound(g):
    """Of silu'(g) in fp32: s = sigmoid(g) is within (4 + |g|) units of itself, 1 - s within that much of s and a
    unit, and what is made of them takes a few more."""
    s = 1.0 / (1.0 + np.exp(-g))
    return s * ((8 + np.abs(g)) * np.abs(1.0 + g * (1.0 - s)) + np.abs(g) * (s * (4 + np.abs(g)) + 2) + 2) * U


SHAPES = [
    # S, K, E, R, H, N, pad mode, pad rows
    (1, 1, 1, 1, 8, 8, PAD_NONE, 0),
    (1, 4, 8, 2, 256, 64, PAD_NONE, 0),
    (1, 8, 16, 1, 1032, 136, PAD_CAPACITY, 4),
    (5, 2, 4, 2, 72, 40, PAD_MULTIPLE, 16),
    (64, 2, 8, 2, 512, 96, PAD_NONE, 0),
    (100, 4, 6, 3, 392, 264, PAD_MULTIPLE, 100),
    (256, 2, 3, 1, 904, 72, PAD_CAPACITY, 130),
    (400, 3, 2, 1, 256, 520, PAD_NONE, 0),
    (33, 16, 80, 8, 264, 24, PAD_NONE, 0),
    (700, 1, 5, 5, 56, 200, PAD_MULTIPLE, 64),
    (1500, 4, 6, 2, 768, 384, PAD_NONE, 0),
    (2000, 2, 300, 4, 520, 272, PAD_MULTIPLE, 8),
    (30000, 1, 10, 1, 64, 520, PAD_NONE, 0),
    (9000, 3, 7, 1, 248, 776, PAD_NONE, 0),
]
IDS = [f"{p[0]}x{p[1]}e{p[2]}h{p[4]}n{p[5]}" for p in SHAPES]
shapes = pytest.mark.parametrize("S,K,E,R,H,N,mode,pad", SHAPES, ids=IDS)


def check_forward(moe, c, rng, H, N):
    xb, x = whole(rng, (c.rows, H))
    wb, w = whole(rng, (c.E, N, H))
    out = c.out(N)
    moe.moe_expert_gemm(c.desc, c.lay, c.poisoned(xb), dev_bf16(wb, DEV), out=out, **c.kw)
    y, size = ref64.product(x, w, c.of_row)
    assert size.max(initial=0) < 2 ** 24
    assert np.array_equal(c.result(out), to_bf16(y[c.held]))


def check_gated(moe, c, rng, H, N):
    xb, x = whole(rng, (c.rows, H))
    wb, w = whole(rng, (c.E, 2 * N, H), step=2.0 ** -5)
    out, pre = c.out(N), c.out(2 * N)
    moe.moe_expert_gemm(c.desc, c.lay, c.poisoned(xb), dev_bf16(wb, DEV), act=moe.MOE_ACT_SWIGLU, out=out, pre=pre, **c.kw)
    y = ref64.product(x, w, c.of_row)[0][c.held]
    assert np.array_equal(c.result(pre), to_bf16(y))
    g, u = y[:, :N], y[:, N:]
    within(c.result(out), ref64.silu(g) * u, silu_bound(g, u))
    again = c.out(N)
    moe.moe_expert_gemm(c.desc, c.lay, c.poisoned(xb), dev_bf16(wb, DEV), act=moe.MOE_ACT_SWIGLU, out=again, **c.kw)
    assert torch.equal(out, again)
    # the values before the activation in fp32
    pre = torch.full((c.rows, 2 * N), 7.0, device=DEV)
    moe.moe_expert_gemm(c.desc, c.lay, c.poisoned(xb), dev_bf16(wb, DEV), act=moe.MOE_ACT_SWIGLU, out=again, pre=pre, **c.kw)
    assert torch.equal(out, again)
    got = pre.cpu().numpy().astype(np.float64)
    assert np.array_equal(got[c.held], y)
    assert (got[~c.held] == 7).all()


def check_backward_x(moe, c, rng, H, N):
    db, d = whole(rng, (c.rows, N))
    wb, w = whole(rng, (c.E, N, H))
    out = c.out(H)
    moe.moe_expert_gemm_backward_x(c.desc, c.lay, c.poisoned(db), dev_bf16(wb, DEV), out=out, **c.kw)
    dx, size = ref64.product(d, w.transpose(0, 2, 1), c.of_row)
    assert size.max(initial=0) < 2 ** 24
    assert np.array_equal(c.result(out), to_bf16(dx[c.held]))
    # on through the activation
    pb = to_bf16(rng.standard_normal((c.rows, 2 * H)) * 2)
    out = c.out(2 * H)
    pre = c.poisoned(pb)
    moe.moe_expert_gemm_backward_x(c.desc, c.lay, c.poisoned(db), dev_bf16(wb, DEV), pre=pre, out=out, **c.kw)
    p = bf16_values(pb)[c.held]
    g, u, dh = p[:, :H], p[:, H:], dx[c.held]
    want = np.concatenate([dh * u * ref64.silu_slope(g), dh * ref64.silu(g)], 1)
    bound = np.concatenate([np.abs(dh * u) * slope_bound(g), np.abs(dh) * silu_bound(g, np.ones_like(g))], 1)
    within(c.result(out), want, bound)
    # the same values of pre in fp32
    pre32, out32 = torch.where(torch.from_numpy(c.held).to(DEV)[:, None], pre.float(), float("nan")), c.out(2 * H)
    moe.moe_expert_gemm_backward_x(c.desc, c.lay, c.poisoned(db), dev_bf16(wb, DEV), pre=pre32, out=out32, **c.kw)
    assert torch.equal(out, out32)
    p = rng.standard_normal((c.rows, 2 * H)).astype(np.float32) * 2
    moe.moe_expert_gemm_backward_x(c.desc, c.lay, c.poisoned(db), dev_bf16(wb, DEV), pre=torch.from_numpy(p).to(DEV), out=out32, **c.kw)
    p = p[c.held].astype(np.float64)
    g, u = p[:, :H], p[:, H:]
    want = np.concatenate([dh * u * ref64.silu_slope(g), dh * ref64.silu(g)], 1)
    bound = np.concatenate([np.abs(dh * u) * slope_bound(g), np.abs(dh) * silu_bound(g, np.ones_like(g))], 1)
    within(c.result(out32), want, bound)
    # into pre itself
    moe.moe_expert_gemm_backward_x(c.desc, c.lay, c.poisoned(db), dev_bf16(wb, DEV), pre=pre, out=pre, **c.kw)
    assert np.array_equal(host_bits(pre)[c.held], c.result(out))


def check_backward_w(moe, c, rng, H, N):
    db, d = whole(rng, (c.rows, N))
    xb, x = whole(rng, (c.rows, H))
    want, size = ref64.product_dw(d, x, c.of_row, c.E)
    assert size.max(initial=0) < 2 ** 24
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((c.E, N, H), 7.0, dtype=dtype, device=DEV)
        moe.moe_expert_gemm_backward_w(c.desc, c.lay, c.poisoned(db), c.poisoned(xb), out=out, **c.kw)
        if dtype is torch.float32:
            assert np.array_equal(out.cpu().numpy().astype(np.float64), want)
        else:
            assert np.array_equal(host_bits(out), to_bf16(want))


def check_int8(moe, c, rng, H, N, act):
    H = (H + 15) // 16 * 16
    swiglu = act == moe.MOE_ACT_SWIGLU
    M = 2 * N if swiglu else N
    x, w = rng.integers(-128, 128, (c.rows, H)).astype(np.int8), rng.integers(-128, 128, (c.E, M, H)).astype(np.int8)
    # scales that give sums of a few units
    xs = (rng.random(c.rows) + 0.5).astype(np.float32)
    ws = ((rng.random((c.E, M)) + 0.5) * 4.0 / (H ** 0.5 * 5461)).astype(np.float32)
    out = c.out(N)
    poison = np.where(c.held, xs, np.float32(np.nan))
    moe.moe_expert_gemm_i8(c.desc, c.lay, dev(x), dev(poison), dev(w), dev(ws), act=act, out=out, **c.kw)
    y = ref64.product(x.astype(np.float64), w.astype(np.float64), c.of_row)[0]
    y = (y * xs[:, None].astype(np.float64) * ws.astype(np.float64)[np.maximum(c.of_row, 0)])[c.held]
    # the sum becomes fp32, then two products: half a unit each
    err = 1.5 * U * np.abs(y) + 2.0 ** -126
    if swiglu:
        g, u = y[:, :N], y[:, N:]
        within(c.result(out), ref64.silu(g) * u, silu_bound(g, u, err[:, :N], err[:, N:]))
    else:
        within(c.result(out), y, err)


@shapes
def test_forward(moe, S, K, E, R, H, N, mode, pad):
    rng = np.random.default_rng(S * 7 + H + N)
    check_forward(moe, Case(moe, rng, S, K, E, R, mode, pad), rng, H, N)


@shapes
def test_gated(moe, S, K, E, R, H, N, mode, pad):
    rng = np.random.default_rng(S * 7 + H + N + 1)
    check_gated(moe, Case(moe, rng, S, K, E, R, mode, pad), rng, H, N)


@shapes
def test_backward_x(moe, S, K, E, R, H, N, mode, pad):
    rng = np.random.default_rng(S * 7 + H + N + 2)
    check_backward_x(moe, Case(moe, rng, S, K, E, R, mode, pad), rng, H, N)


@shapes
def test_backward_w(moe, S, K, E, R, H, N, mode, pad):
    rng = np.random.default_rng(S * 7 + H + N + 3)
    check_backward_w(moe, Case(moe, rng, S, K, E, R, mode, pad), rng, H, N)


@pytest.mark.parametrize("act", [0, 1])
@shapes
def test_int8(moe, S, K, E, R, H, N, mode, pad, act):
    rng = np.random.default_rng(S * 7 + H + N + 4)
    check_int8(moe, Case(moe, rng, S, K, E, R, mode, pad), rng, H, N, act)


@pytest.mark.parametrize("S,K,E,R,B,H,N", [(40, 2, 8, 4, 2, 256, 40), (600, 4, 16, 4, 6, 136, 104), (700, 2, 24, 2, 0, 128, 64),
                                           (9000, 4, 12, 3, 8, 256, 72), (500, 2, 1024, 8, 64, 64, 16)])
def test_balanced(moe, S, K, E, R, B, H, N):
    """Rows of a replica slot use the weights of the expert in it, and add to that expert's gradient."""
    rng = np.random.default_rng(S)
    c = Case(moe, rng, S, K, E, R, slots=B)
    check_forward(moe, c, rng, H, N)
    check_gated(moe, c, rng, H, N)
    check_backward_x(moe, c, rng, H, N)
    check_backward_w(moe, c, rng, H, N)
    check_int8(moe, c, rng, H, N, moe.MOE_ACT_NONE)


@pytest.mark.parametrize("S", [0, 12])
def test_no_row_at_all(moe, S):
    """No expert has a row: nothing is written but the weights' gradient, which is zero."""
    idx = np.full((S, 2), -1, np.int32)
    desc = moe.LayoutDesc(S, 2, 4, 2, moe.MOE_PAD_MULTIPLE, 4)
    lay = moe.moe_layout(desc, dev(idx))
    rows = moe.moe_max_recv_rows(desc)
    x = torch.full((rows, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    w = torch.ones((4, 64, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.full((rows, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_gemm(desc, lay, x, w, out=out)
    moe.moe_expert_gemm_backward_x(desc, lay, x, w, out=out)
    moe.moe_expert_gemm_i8(desc, lay, torch.ones((rows, 64), dtype=torch.int8, device=DEV), torch.ones(rows, device=DEV),
                           torch.ones((4, 64, 64), dtype=torch.int8, device=DEV), torch.ones((4, 64), device=DEV), out=out)
    assert (out == 7.0).all()
    for dtype in (torch.float32, torch.bfloat16):
        dw = torch.full((4, 64, 64), float("nan"), dtype=dtype, device=DEV)
        moe.moe_expert_gemm_backward_w(desc, lay, x, x, out=dw)
        assert (dw == 0).all()


@pytest.mark.parametrize("S", [3, 150, 2000])
def test_any_value(moe, S):
    """N(0,1) values, and a NaN in one row and one weight stay where they belong."""
    rng = np.random.default_rng(S)
    K, E, H, N = 2, 4, 1160, 104
    c = Case(moe, rng, S, K, E, 2)
    xb, wb, db = normal_bf16_bits(rng, (c.rows, H)), normal_bf16_bits(rng, (E, N, H)), normal_bf16_bits(rng, (c.rows, N))
    x, w, d = bf16_values(xb), bf16_values(wb), bf16_values(db)
    X, W, D = c.poisoned(xb), dev_bf16(wb, DEV), c.poisoned(db)
    out = c.out(N)
    moe.moe_expert_gemm(c.desc, c.lay, X, W, out=out)
    y, size = ref64.product(x, w, c.of_row)
    within(c.result(out), y[c.held], ((H / 32 + 16) * U * size)[c.held])
    out = c.out(H)
    moe.moe_expert_gemm_backward_x(c.desc, c.lay, D, W, out=out)
    y, size = ref64.product(d, w.transpose(0, 2, 1), c.of_row)
    within(c.result(out), y[c.held], ((N / 32 + 16) * U * size)[c.held])
    dw = moe.moe_expert_gemm_backward_w(c.desc, c.lay, D, X, dtype=torch.float32).cpu().numpy()
    want, size = ref64.product_dw(d, x, c.of_row, E)
    assert (np.abs(dw - want) <= (S * K / 32 + 16) * U * size).all()
    e = c.of_row[c.held][0]
    row = int(np.nonzero(c.held)[0][0])
    xb[row, 7] = 0x7FC0
    out = c.out(N)
    moe.moe_expert_gemm(c.desc, c.lay, c.poisoned(xb), W, out=out)
    nan = np.isnan(bf16_values(host_bits(out)))[:c.rows]
    assert nan[row].all() and nan.sum() == N
    dw = moe.moe_expert_gemm_backward_w(c.desc, c.lay, D, c.poisoned(xb), dtype=torch.float32).cpu().numpy()
    assert np.isnan(dw[e, :, 7]).all() and np.isnan(dw).sum() == N
    wb[e, 5, 3] = 0x7F80
    out = c.out(N)
    xb[row, 7] = 0x3F80
    moe.moe_expert_gemm(c.desc, c.lay, c.poisoned(xb), dev_bf16(wb, DEV), out=out)
    bad = ~np.isfinite(bf16_values(host_bits(out)))[:c.rows]
    assert bad[c.of_row == e][:, 5].all() and bad.sum() == (c.of_row == e).sum()
    out = c.out(H)
    moe.moe_expert_gemm_backward_x(c.desc, c.lay, D, dev_bf16(wb, DEV), out=out)
    bad = ~np.isfinite(bf16_values(host_bits(out)))[:c.rows]
    assert bad[c.of_row == e][:, 3].all() and bad.sum() == (c.of_row == e).sum()


def test_int8_largest_sums(moe):
    """The longest rows at the codes' limits: the sums stay in 32 bits."""
    H = 131056
    desc = moe.LayoutDesc(2, 1, 1, 1)
    lay = moe.moe_layout(desc, torch.zeros((2, 1), dtype=torch.int32, device=DEV))
    x = torch.full((2, H), -128, dtype=torch.int8, device=DEV)
    w = torch.full((1, 16, H), -128, dtype=torch.int8, device=DEV)
    w[0, 8:] = 127
    scale = torch.ones(16, device=DEV)
    out = moe.moe_expert_gemm_i8(desc, lay, x, scale, w, scale.view(1, 16))
    want = torch.tensor([128.0 * 128 * H, -128.0 * 127 * H], dtype=torch.float64).to(torch.bfloat16).repeat_interleave(8)
    assert torch.equal(out.cpu(), want.expand(2, 16))


def moved_to_host(t):
    return t.detach().double().cpu()


def layer64(idx, tw, hidden, w_in, w_out, shared):
    """The whole layer in 64 bits on the host, token by token, of torch tensors."""
    S, K = idx.shape
    N = w_out.shape[2]
    out = []
    for t in range(S):
        y = shared[t]
        for k in range(K):
            e = int(idx[t, k])
            if e >= 0:
                v = w_in[e] @ hidden[t]
                y = y + tw[t, k] * (w_out[e] @ (torch.nn.functional.silu(v[:N]) * v[N:]))
        out.append(y)
    return torch.stack(out)


@pytest.mark.parametrize("mode,pad,slots", [(PAD_NONE, 0, None), (PAD_MULTIPLE, 16, None), (PAD_NONE, 0, 3)])
def test_layer_and_its_gradients(moe, mode, pad, slots):
    """dispatch, expert_ffn and combine in a row, forward and backward, against the formulas in 64 bits.  Rounded to
    bf16 on the way: h, pre, d_pre, the rows in between; each is off by 2^-8 of itself at most, so a sum over n such
    terms by 2^-8 of their norm, and the gradients by a few of those."""
    rng = np.random.default_rng(11)
    S, K, E, R, H, N = 50, 3, 8, 2, 72, 40
    c = Case(moe, rng, S, K, E, R, mode, pad, slots)
    torch.manual_seed(3)

    def leaf(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, device=DEV) * scale).to(dtype).requires_grad_()

    hidden, w_in, w_out = leaf(S, H), leaf(E, 2 * N, H, scale=H ** -0.5), leaf(E, H, N, scale=N ** -0.5)
    shared = leaf(S, H)
    tw = torch.rand((S, K), device=DEV).requires_grad_()
    rows = moe.dispatch(c.desc, c.lay, hidden)
    y = moe.expert_ffn(c.desc, c.lay, rows, w_in, w_out, **c.kw)
    out = moe.combine(c.desc, c.lay, y, tw, shared)
    assert not bool(torch.isnan(rows).any() | torch.isnan(y).any())
    weight = torch.randn((S, H), device=DEV).to(torch.bfloat16)
    leaves = (hidden, w_in, w_out, tw, shared)
    grads = torch.autograd.grad(out, leaves, weight)
    host = [moved_to_host(t).requires_grad_() for t in leaves]
    want = layer64(c.idx, host[3], host[0], host[1], host[2], host[4])
    want_grads = torch.autograd.grad(want, host, moved_to_host(weight))
    for got, ref, steps in zip((out, *grads), (want, *want_grads), (3, 6, 6, 6, 3, 0)):
        ref = ref.detach()
        off = (moved_to_host(got) - ref).norm() / ref.norm()
        assert off <= steps * 2.0 ** -8, off


def test_gradients_against_differences(moe):
    """d loss / d weights along a direction, against the loss at two points: of a product of whole numbers, linear in
    the weights, so that the difference is exact."""
    rng = np.random.default_rng(5)
    S, K, E, H, N = 60, 2, 5, 64, 24
    c = Case(moe, rng, S, K, E, 1, PAD_MULTIPLE, 8)
    xb, _ = whole(rng, (c.rows, H))
    wb, w = whole(rng, (E, N, H))
    db, d = whole(rng, (c.rows, N))
    _, step = whole(rng, (E, N, H), most=1)

    def loss(weights):
        out = torch.zeros((c.rows, N), dtype=torch.bfloat16, device=DEV)
        moe.moe_expert_gemm(c.desc, c.lay, dev_bf16(xb, DEV), dev_bf16(to_bits(weights), DEV), out=out)
        return float((bf16_values(host_bits(out)) * d)[c.held].sum()), np.abs(bf16_values(host_bits(out)) * d)[c.held].sum()

    up, size_up = loss(w + step)
    down, size_down = loss(w - step)
    dw = moe.moe_expert_gemm_backward_w(c.desc, c.lay, dev_bf16(db, DEV), dev_bf16(xb, DEV), dtype=torch.float32).cpu().numpy()
    # each output is rounded to bf16 once: half a step of it at most
    assert abs((up - down) / 2 - float((dw * step).sum())) <= 2.0 ** -8 * (size_up + size_down) / 2


def test_autograd_functions_refuse_capture(moe):
    desc = moe.LayoutDesc(4, 1, 2, 1)
    lay = moe.moe_layout(desc, torch.zeros((4, 1), dtype=torch.int32, device=DEV))
    x = torch.zeros((4, 16), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((2, 32, 16), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros((2, 16, 16), dtype=torch.bfloat16, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in (lambda: moe.dispatch(desc, lay, x), lambda: moe.expert_ffn(desc, lay, x, w, v), lambda: moe.combine(desc, lay, x)):
            with pytest.raises(RuntimeError, match="captured"):
                call()
        y = x + 1
    g.replay()
    torch.cuda.synchronize()
    assert (y == 1).all()


def test_graph_replay(moe):
    """The calls in a captured graph, replayed with new inputs between eager work."""
    rng = np.random.default_rng(21)
    S, K, E, H, N = 70, 2, 6, 128, 48
    c = Case(moe, rng, S, K, E, 2, PAD_MULTIPLE, 8)
    x, d = (torch.zeros((c.rows, n), dtype=torch.bfloat16, device=DEV) for n in (H, H))
    w_in, w_out = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((E, 2 * N, H), (E, H, N)))
    pre, h = torch.zeros((c.rows, 2 * N), dtype=torch.bfloat16, device=DEV), torch.zeros((c.rows, N), dtype=torch.bfloat16, device=DEV)
    y, dpre, dx = torch.zeros_like(x), torch.zeros_like(pre), torch.zeros_like(x)
    dw_in, dw_out = torch.zeros_like(w_in), torch.zeros_like(w_out)
    codes, scales = torch.zeros((c.rows, H), dtype=torch.int8, device=DEV), torch.zeros(c.rows, device=DEV)
    wq, ws = torch.zeros((E, N, H), dtype=torch.int8, device=DEV), torch.zeros((E, N), device=DEV)
    y8 = torch.zeros((c.rows, N), dtype=torch.bfloat16, device=DEV)
    dyc, dwc = torch.zeros_like(x), torch.zeros((S, K), device=DEV)
    tok, tw = torch.zeros((S, H), dtype=torch.bfloat16, device=DEV), torch.zeros((S, K), device=DEV)
    back = torch.zeros_like(x)
    outs = (pre, h, y, dpre, dx, dw_in, dw_out, codes, scales, y8, dyc, dwc, back)

    def step():
        moe.moe_expert_gemm(c.desc, c.lay, x, w_in, act=moe.MOE_ACT_SWIGLU, out=h, pre=pre)
        moe.moe_expert_gemm(c.desc, c.lay, h, w_out, out=y)
        moe.moe_expert_gemm_backward_x(c.desc, c.lay, d, w_out, pre=pre, out=dpre)
        moe.moe_expert_gemm_backward_w(c.desc, c.lay, d, h, out=dw_out)
        moe.moe_expert_gemm_backward_x(c.desc, c.lay, dpre, w_in, out=dx)
        moe.moe_expert_gemm_backward_w(c.desc, c.lay, dpre, x, out=dw_in)
        moe.moe_quantize_i8(x, codes, scales, layout=c.lay)
        moe.moe_expert_gemm_i8(c.desc, c.lay, codes, scales, wq, ws, out=y8)
        moe.moe_combine_backward(c.desc, c.lay, tok, y, tw, d_expert_out=dyc, d_w=dwc)
        moe.moe_dequantize_i8(codes, scales, out=back, layout=c.lay)

    def fill(seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        for t in (x, d, w_in, w_out, tok):
            t.normal_(0, 0.3, generator=g)
        wq.random_(-127, 128, generator=g)
        ws.uniform_(0.001, 0.002, generator=g)
        tw.uniform_(0, 1, generator=g)

    fill(0)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2, 3):
        fill(seed)
        for t in outs:
            t.zero_()
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
