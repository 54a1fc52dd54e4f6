"""The experts' products, their gradients, the 8-bit rows and combine's gradient over the range that their callers may
draw from: shapes at random, segments of every length around a tile's, arrays past 4 GiB, several streams, an expert
chosen twice."""
from __future__ import annotations

import pickle

import numpy as np
import pytest
import torch

import test_gpu_expert_products as products
from expert_products_reference import combine_backward, quantize_i8
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


def every_product(moe, c, rng, H, N):
    products.check_forward(moe, c, rng, H, N)
    products.check_gated(moe, c, rng, H, N)
    products.check_backward_x(moe, c, rng, H, N)
    products.check_backward_w(moe, c, rng, H, N)
    products.check_int8(moe, c, rng, H, N, moe.MOE_ACT_NONE)
    products.check_int8(moe, c, rng, H, N, moe.MOE_ACT_SWIGLU)


@pytest.mark.parametrize("seed", range(16))
def test_drawn(moe, seed):
    rng = np.random.default_rng(100 + seed)
    R = int(rng.integers(1, 5))
    E = R * int(2 ** rng.uniform(0, 6))
    S, K = int(2 ** rng.uniform(0, 11)), int(rng.integers(1, min(E, 8) + 1))
    H, N = 8 * int(2 ** rng.uniform(0, 6.5)), 8 * int(2 ** rng.uniform(0, 6.5))
    if seed % 4 == 3 and K < E:
        c = products.Case(moe, rng, S, 1, E, R, slots=int(rng.integers(1, 4)))
    else:
        mode = (PAD_NONE, PAD_MULTIPLE, PAD_CAPACITY)[seed % 3]
        c = products.Case(moe, rng, S, K, E, R, mode, 0 if mode == PAD_NONE else int(rng.integers(1, 40)))
    every_product(moe, c, rng, H, N)


class Counted(products.Case):
    """Segments of the given lengths."""

    def __init__(self, moe, rng, counts):
        self.counts = counts
        super().__init__(moe, rng, sum(counts), 1, len(counts), 1)


@pytest.mark.parametrize("counts", [
    [1, 15, 16, 17, 31, 32, 33, 0], [63, 64, 65, 127, 128, 129], [255, 256, 257, 0, 1, 511, 512, 513], [2, 700, 30, 1, 1, 1],
], ids=str)
@pytest.mark.parametrize("H,N", [(256, 520), (1288, 72)])
def test_segments_around_a_tile(moe, monkeypatch, counts, H, N):
    rng = np.random.default_rng(sum(counts) + H)
    idx = rng.permutation(np.repeat(np.arange(len(counts)), counts)).astype(np.int32).reshape(-1, 1)
    monkeypatch.setattr(products, "routing", lambda *a: idx)
    every_product(moe, Counted(moe, rng, counts), rng, H, N)


def test_expert_chosen_twice(moe, monkeypatch):
    """A token may name one expert more than once: it has a row for each."""
    rng = np.random.default_rng(6)
    idx = rng.integers(0, 3, (90, 4)).astype(np.int32)
    monkeypatch.setattr(products, "routing", lambda *a: idx)
    c = products.Case(moe, rng, 90, 4, 3, 1, PAD_MULTIPLE, 16)
    every_product(moe, c, rng, 136, 72)
    hid, y, d = (dev_bf16(normal_bf16_bits(rng, (n, 128)), DEV) for n in (90, c.rows, 90))
    tw = dev(rng.random((90, 4)).astype(np.float32))
    codes, scales, _ = moe.moe_dispatch_i8(c.desc, c.lay, hid)
    wc, ws = quantize_i8(bf16_values(host_bits(hid)))
    src = c.lay.src.cpu().numpy()
    assert np.array_equal(codes.cpu().numpy()[c.held], wc[src[c.held] // 4])
    assert np.array_equal(scales.cpu().numpy()[c.held], ws[src[c.held] // 4])
    d_y, d_w = moe.moe_combine_backward(c.desc, c.lay, d, y, tw)
    pos = c.lay.pos.cpu().numpy().reshape(90, 4)
    want_y, want_w, size = combine_backward(bf16_values(host_bits(d)), bf16_values(host_bits(y)), tw.cpu().numpy().astype(np.float64), pos, c.rows)
    assert np.array_equal(host_bits(d_y)[c.held], to_bf16(want_y[c.held].astype(np.float32)))
    assert (np.abs(d_w.cpu().numpy() - want_w) <= 130 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("S,K,E,H,mode,pad", [(700, 8, 32, 7168, PAD_NONE, 0), (2600, 3, 6, 4104, PAD_MULTIPLE, 64),
                                              (170, 16, 20, 16376, PAD_CAPACITY, 130)])
def test_combine_backward_of_large_batches(moe, S, K, E, H, mode, pad):
    rng = np.random.default_rng(S)
    idx = rng.integers(-1, E, (S, K)).astype(np.int32)
    desc = moe.LayoutDesc(S, K, E, 1, mode, pad)
    lay = moe.moe_layout(desc, dev(idx))
    pos, rows = lay.pos.cpu().numpy().reshape(S, K), moe.moe_max_recv_rows(desc)
    held = lay.src.cpu().numpy() >= 0
    db, yb = normal_bf16_bits(rng, (S, H)), normal_bf16_bits(rng, (rows, H))
    w = rng.random((S, K)).astype(np.float32)
    d, y = dev_bf16(db, DEV), dev_bf16(np.where(held[:, None], yb, POISON_BF16).astype(np.uint16), DEV)
    want_y, want_w, size = combine_backward(bf16_values(db), bf16_values(yb), w.astype(np.float64), pos, rows)
    out = torch.full((rows + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)
    _, d_w = moe.moe_combine_backward(desc, lay, d, y, dev(w), d_expert_out=out)
    bits = host_bits(out)
    assert (bf16_values(bits)[:rows][~held] == 7.0).all() and (bf16_values(bits)[rows:] == 7.0).all()
    assert np.array_equal(bits[:rows][held], to_bf16(want_y[held].astype(np.float32)))
    assert (np.abs(d_w.cpu().numpy() - want_w) <= (H + 2) * 2.0 ** -24 * size).all()
    own = y.clone()
    _, again = moe.moe_combine_backward(desc, lay, d, own, dev(w), d_expert_out=own)
    assert torch.equal(again, d_w)
    assert np.array_equal(host_bits(own)[held], bits[:rows][held]) and np.array_equal(host_bits(own)[~held], host_bits(y)[~held])


def test_quantize_every_ratio(moe):
    """Every mantissa of a row's maximum with every value of the nine exponents below: each code that a ratio of two
    bf16 numbers can have, at both ends of the exponents and in the middle."""
    for exponent in (9, 10, 127, 254):
        top = (exponent << 7) + np.arange(128)
        below = np.arange((exponent - 9) << 7, (exponent << 7) + 128)
        bits = np.zeros((128, below.size * 2 + 16), np.uint16)
        bits[:, 16:] = np.concatenate([below, below | 0x8000])[None]
        mine = (bits & 0x7FFF) > top[:, None]
        bits[mine] = 0
        bits[:, 0] = top
        codes, scales = moe.moe_quantize_i8(dev_bf16(bits, DEV))
        wc, ws = quantize_i8(bf16_values(bits))
        assert np.array_equal(scales.cpu().numpy(), ws)
        assert np.array_equal(codes.cpu().numpy(), wc)


def few(shape, seed, most=2, dtype=torch.bfloat16):
    """Whole numbers up to `most`, made on the device: sums of a few thousand of their products are exact."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV, dtype=torch.int8).to(dtype)


def rows_of_layout(lay, e):
    o, n = int(lay.expert_offset[e]), int(lay.tokens_per_expert[e])
    return slice(o, o + n)


def some(rows):
    """First and last rows of a segment."""
    return [slice(rows.start, min(rows.start + 40, rows.stop)), slice(max(rows.stop - 40, rows.start), rows.stop)]


def test_rows_past_4_gib(moe):
    S, K, E, H, N = 560000, 4, 6, 1024, 64
    assert S * K * H * 2 > 1 << 32
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    idx = torch.rand((S, E), generator=g, device=DEV).topk(K, 1).indices.to(torch.int32)
    desc = moe.LayoutDesc(S, K, E, 2)
    lay = moe.moe_layout(desc, idx)
    x, w = few((S * K, H), 2), few((E, N, H), 3)
    y = moe.moe_expert_gemm(desc, lay, x, w)
    d = few((S * K, N), 4)
    dx = moe.moe_expert_gemm_backward_x(desc, lay, d, w)
    dw = moe.moe_expert_gemm_backward_w(desc, lay, d, x, dtype=torch.float32)
    codes, scale, ones = x.to(torch.int8), torch.ones(S * K, device=DEV), torch.ones((E, N), device=DEV)
    y8 = moe.moe_expert_gemm_i8(desc, lay, codes, scale, w.to(torch.int8), ones)
    assert torch.equal(y8, y)
    # wide results: [rows, 1024] from narrow rows, and both halves of a gated product and of its gradient
    wide = few((E, H, N), 5)
    z = moe.moe_expert_gemm(desc, lay, d, wide)
    pre = torch.empty((S * K, H), device=DEV)
    h = moe.moe_expert_gemm(desc, lay, d, wide, act=moe.MOE_ACT_SWIGLU, pre=pre)
    d_pre = moe.moe_expert_gemm_backward_x(desc, lay, d, few((E, N, H // 2), 6), pre=pre)
    for e in range(E):
        seg = rows_of_layout(lay, e)
        for part in some(seg):
            assert torch.equal(y[part].float(), (x[part].float() @ w[e].float().T).bfloat16().float())
            assert torch.equal(dx[part].float(), (d[part].float() @ w[e].float()).bfloat16().float())
            want = d[part].float() @ wide[e].float().T
            assert torch.equal(z[part].float(), want.bfloat16().float()) and torch.equal(pre[part], want)
            gate, up = want.double().split(H // 2, 1)
            s = torch.sigmoid(gate)
            assert torch.allclose(h[part].double(), gate * s * up, rtol=2.0 ** -8 + 2.0 ** -14, atol=2.0 ** -20)
            dh = (d[part].float() @ few((E, N, H // 2), 6)[e].float()).double()
            want = torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], 1)
            # s is off by 6 units of 2^-23 and |g| times that where g < 0, where s falls faster than |g| rises:
            # s * (1 + g(1 - s)) by (8 + 8|g|) units at most; then half a step of bf16
            slack = torch.cat([(1 + gate.abs()) * 2.0 ** -19 * (dh * up).abs(), torch.zeros_like(gate)], 1)
            assert ((d_pre[part].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * want.abs() + slack + 2.0 ** -20).all()
        want = torch.zeros((N, H), dtype=torch.float64, device=DEV)
        for at in range(seg.start, seg.stop, 100000):
            part = slice(at, min(at + 100000, seg.stop))
            want += (d[part].float().T @ x[part].float()).double()
        # whole numbers: exact as long as 32 bits hold every partial sum
        assert float(want.abs().max()) < 2 ** 24 and torch.equal(dw[e].double(), want)


@pytest.mark.parametrize("S", [24, 3000])
def test_weights_past_4_gib(moe, S):
    """Few rows, which the streaming kernel takes, and many."""
    K, E, M, H = 2, 40, 8192, 8192
    assert E * M * H * 2 > 1 << 32
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    idx = torch.randint(0, E, (S, K), generator=g, device=DEV, dtype=torch.int32)
    idx[0, 0], idx[0, 1] = E - 1, 0
    desc = moe.LayoutDesc(S, K, E, 1)
    lay = moe.moe_layout(desc, idx)
    x, w = few((S * K, H), 2, 1), few((E, M, H), 3, 1)
    y, h = moe.moe_expert_gemm(desc, lay, x, w), moe.moe_expert_gemm(desc, lay, x, w, act=moe.MOE_ACT_SWIGLU)
    dx = moe.moe_expert_gemm_backward_x(desc, lay, few((S * K, M), 4, 1), w)
    y8 = moe.moe_expert_gemm_i8(desc, lay, x.to(torch.int8), torch.ones(S * K, device=DEV), w.to(torch.int8), torch.ones((E, M), device=DEV))
    assert torch.equal(y8, y)
    d = few((S * K, M), 4, 1)
    for e in (0, 1, E // 2, E - 1):
        for part in some(rows_of_layout(lay, e)):
            want = x[part].float() @ w[e].float().T
            assert torch.equal(y[part], want.bfloat16())
            gate, up = want.double().split(M // 2, 1)
            assert torch.allclose(h[part].double(), gate * torch.sigmoid(gate) * up, rtol=2.0 ** -8 + 2.0 ** -13, atol=2.0 ** -20)
            assert torch.equal(dx[part], (d[part].float() @ w[e].float()).bfloat16())
    del w, y8
    for dtype in (torch.bfloat16, torch.float32):
        dw = moe.moe_expert_gemm_backward_w(desc, lay, d, x, dtype=dtype)
        for e in (0, 1, E // 2, E - 1):
            seg = rows_of_layout(lay, e)
            assert torch.equal(dw[e], (d[seg].float().T @ x[seg].float()).to(dtype))
        del dw


def test_8_bit_rows_past_4_gib(moe):
    n, reps, K, E, H = 500, 160, 8, 16, 7168
    S = n * reps
    assert S * K * H > 1 << 32
    rng = np.random.default_rng(2)
    bits = normal_bf16_bits(rng, (n, H))
    hid = dev_bf16(bits, DEV).repeat(reps, 1)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(S)]).astype(np.int32)).to(DEV)
    desc = moe.LayoutDesc(S, K, E, 2)
    lay = moe.moe_layout(desc, idx)
    codes, scales, _ = moe.moe_dispatch_i8(desc, lay, hid)
    wc, ws = quantize_i8(bf16_values(bits))
    out = moe.moe_dequantize_i8(codes, scales, layout=lay)
    again = moe.moe_quantize_i8(out, layout=lay)
    tw = dev(rng.random((S, K)).astype(np.float32))
    d_y, d_w = moe.moe_combine_backward(desc, lay, hid, out, tw)
    rows = S * K
    for first in (0, rows // 2, rows - 300):
        part = slice(first, first + 300)
        src = lay.src[part].cpu().numpy()
        token = src // K % n
        assert np.array_equal(codes[part].cpu().numpy(), wc[token]) and np.array_equal(scales[part].cpu().numpy(), ws[token])
        assert np.array_equal(host_bits(out[part]), to_bf16(wc[token].astype(np.float32) * ws[token][:, None]))
        c, s = quantize_i8(bf16_values(host_bits(out[part])))
        assert np.array_equal(again[0][part].cpu().numpy(), c) and np.array_equal(again[1][part].cpu().numpy(), s)
        w = tw.cpu().numpy().reshape(-1)[src]
        assert np.array_equal(host_bits(d_y[part]), to_bf16(w[:, None] * bf16_values(bits)[token].astype(np.float32)))
        terms = bf16_values(bits)[token] * bf16_values(host_bits(out[part]))
        off = np.abs(d_w.cpu().numpy().reshape(-1)[src] - terms.sum(1))
        assert (off <= (H + 2) * 2.0 ** -24 * np.abs(terms).sum(1)).all()


def test_two_streams_at_once(moe):
    """Two batches of calls on streams of their own, one of them named in the call, equal the same calls in turn."""
    rng = np.random.default_rng(12)
    jobs = []
    for S, E in ((300, 6), (2000, 4)):
        c = products.Case(moe, rng, S, 2, E, 1)
        x, w, v = (dev_bf16(normal_bf16_bits(rng, s), DEV) for s in ((c.rows, 512), (E, 2 * 264, 512), (E, 512, 264)))
        d, tw = dev_bf16(normal_bf16_bits(rng, (S, 512)), DEV), dev(rng.random((S, 2)).astype(np.float32))
        jobs.append((c, x, w, v, d, tw))

    def chain(job, stream=None):
        c, x, w, v, d, tw = job
        pre = torch.empty((c.rows, 2 * 264), device=DEV)
        h = moe.moe_expert_gemm(c.desc, c.lay, x, w, act=moe.MOE_ACT_SWIGLU, pre=pre, stream=stream)
        y = moe.moe_expert_gemm(c.desc, c.lay, h, v, stream=stream)
        dy, dw = moe.moe_combine_backward(c.desc, c.lay, d, y, tw, stream=stream)
        d_pre = moe.moe_expert_gemm_backward_x(c.desc, c.lay, dy, v, pre=pre, stream=stream)
        d_in = moe.moe_expert_gemm_backward_w(c.desc, c.lay, d_pre, x, stream=stream)
        codes, scales = moe.moe_quantize_i8(y, layout=c.lay, stream=stream)
        return h, y, dy, d_pre, codes, scales, dw, d_in

    want = [[t.clone() for t in chain(job)] for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        got = []
        with torch.cuda.stream(streams[0]):
            got.append(chain(jobs[0]))
        with torch.cuda.stream(streams[1]):
            got.append(chain(jobs[1], streams[1]))
        torch.cuda.synchronize()
        for job, a, b in zip(jobs, got, want):
            held = dev(job[0].held)                            # rows without an entry hold anything
            assert all(torch.equal(p[held], q[held]) for p, q in zip(a[:6], b[:6]))
            assert torch.equal(a[6], b[6]) and torch.equal(a[7], b[7])


def test_descriptor_after_use_is_copied(moe):
    rng = np.random.default_rng(4)
    c = products.Case(moe, rng, 20, 2, 4, 1, PAD_MULTIPLE, 8)
    x, w = dev_bf16(normal_bf16_bits(rng, (c.rows, 64)), DEV), dev_bf16(normal_bf16_bits(rng, (4, 24, 64)), DEV)
    want = moe.moe_expert_gemm(c.desc, c.lay, x, w)
    copy = pickle.loads(pickle.dumps(c.desc))
    assert copy == c.desc
    got = moe.moe_expert_gemm(copy, c.lay, x, w)
    held = dev(c.held)
    assert torch.equal(got[held], want[held])


def test_what_is_kept_of_the_activation(moe):
    """expert_ffn keeps its activation's arguments in fp32, or in bf16: the rounding alone lies between the gradients."""
    rng = np.random.default_rng(9)
    c = products.Case(moe, rng, 64, 2, 4, 1)
    torch.manual_seed(2)
    grads = {}
    x = torch.randn((c.rows, 96), device=DEV).bfloat16().requires_grad_()
    w_in = (torch.randn((4, 2 * 72, 96), device=DEV) * 0.1).bfloat16().requires_grad_()
    w_out = (torch.randn((4, 96, 72), device=DEV) * 0.1).bfloat16().requires_grad_()
    d = torch.randn((c.rows, 96), device=DEV).bfloat16()
    for dtype in (torch.float32, torch.bfloat16):
        y = moe.expert_ffn(c.desc, c.lay, x, w_in, w_out, pre_dtype=dtype)
        grads[dtype] = (y.detach(), *torch.autograd.grad(y, (x, w_in, w_out), d))
    a, b = grads[torch.float32], grads[torch.bfloat16]
    assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])
    # each element of pre is off by 2^-8 at most, d_pre by that and the slope's change, and is rounded once itself
    for p, q in zip(a[1:3], b[1:3]):
        assert 0 < float((p.double() - q.double()).norm()) <= 5 * 2.0 ** -8 * float(p.double().norm())
    # the formula from the fp32 values
    e = torch.from_numpy(c.of_row).to(DEV)
    xs, wi, wo = (t.detach().double().requires_grad_() for t in (x, w_in, w_out))
    out = torch.zeros((c.rows, 96), dtype=torch.float64, device=DEV)
    for k in range(4):
        at = torch.nonzero(e == k)[:, 0]
        gate, up = (xs[at] @ wi[k].T).split(72, 1)
        out = out.index_put((at,), (torch.nn.functional.silu(gate) * up) @ wo[k].T)
    want = torch.autograd.grad(out, (xs, wi, wo), d.double())
    # h or d_pre, and the result: each rounded once
    for got, ref in zip(a[1:], want):
        assert float((got.double() - ref).norm()) <= 2 * 2.0 ** -8 * float(ref.norm())
    # nothing is kept where no gradient needs it
    assert torch.equal(moe.expert_ffn(c.desc, c.lay, x.detach(), w_in.detach(), w_out), a[0])
    y = moe.expert_ffn(c.desc, c.lay, x.detach(), w_in.detach(), w_out)
    assert torch.equal(torch.autograd.grad(y, w_out, d)[0], a[3])
    with torch.no_grad():
        before = torch.cuda.memory_allocated()
        y = moe.expert_ffn(c.desc, c.lay, x, w_in, w_out)
        assert torch.equal(y, a[0]) and not y.requires_grad
        assert torch.cuda.memory_allocated() - before <= c.rows * 96 * 2 + 2048
    with pytest.raises(TypeError):
        moe.expert_ffn(c.desc, c.lay, x, w_in, w_out, pre_dtype=torch.float16)
