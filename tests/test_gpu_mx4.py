"""MXFP4 conversions, dispatch and expert products on the GPU.

Conversions and the dispatch are compared bit for bit.  Products of test data
whose scales lie within a factor of two are exact in fp32 in any order (each
product is a multiple of a power of two and their sum stays under 2^24 of
them), so the bf16 result has to equal the rounded exact one, bit for bit.
With arbitrary scales a sum's error is bounded by one unit (2^-23) of the sum
of absolute products for each instruction (H/128 of them), each of the few joins
of partial sums, and the terms an instruction aligns to its largest (8 more for
safety in the instruction's own tree): (H/128 + 16) * 2^-23 * size.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from parity_helpers import dev_bf16, host_bits
from router_mx4_reference import bf16_values, expert_product, mx4_quantize, mx4_values, to_bf16
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


# ---------------------------------------------------------------------------
# conversions
# ---------------------------------------------------------------------------

def quantize_check(moe, bits):
    codes, scales = moe.moe_quantize_mx4(dev_bf16(bits, DEV))
    want_c, want_s = mx4_quantize(bf16_values(bits))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    back = moe.moe_dequantize_mx4(codes, scales)
    v = mx4_values(want_c, want_s)
    got = bf16_values(host_bits(back))
    assert np.array_equal(np.isnan(got), np.isnan(v))
    assert np.array_equal(got[~np.isnan(v)], v[~np.isnan(v)])


@pytest.mark.parametrize("rows,H", [(1, 128), (3, 128), (1, 2048), (7, 384), (5, 2176), (33, 7168), (257, 640)])
def test_quantize(moe, rows, H):
    quantize_check(moe, normal_bf16_bits(np.random.default_rng(rows * H), (rows, H)))


def test_quantize_every_value_at_every_scale(moe):
    """Every finite bf16 value below a block maximum of each exponent, subnormal ones included: rounding ties,
    saturation above 6, signed zeros, the lowest scale."""
    exps = np.arange(0, 255)
    rows = []
    for e in exps:
        top = (e << 7) | 0x7F                            # the largest value of this exponent
        lo = max(0, ((e - 6) << 7))                      # below that everything rounds to 0
        v = np.arange(lo, top + 1, dtype=np.uint16)
        v = np.concatenate([v, v | 0x8000, [0, 0x8000]])
        v = np.concatenate([v, np.zeros(-len(v) % 31, np.uint16)]).reshape(-1, 31)
        rows.append(np.concatenate([np.full((len(v), 1), top, np.uint16), v], 1))
    blocks = np.concatenate(rows)
    blocks = np.concatenate([blocks, np.zeros((-len(blocks) % 4, 32), np.uint16)]).astype(np.uint16)
    quantize_check(moe, blocks.reshape(-1, 128))


def test_quantize_maxima_of_every_mantissa(moe):
    top = np.arange(0, 0x7F80, dtype=np.uint16)          # every finite magnitude as a block's maximum
    blocks = np.zeros((top.size, 32), np.uint16)
    blocks[:, 5] = top | 0x8000
    blocks[:, 9] = np.maximum(top.astype(np.int32) - 0x81, 0).astype(np.uint16)
    quantize_check(moe, blocks.reshape(-1, 128))


def test_quantize_broken_blocks(moe):
    bits = normal_bf16_bits(np.random.default_rng(2), (4, 256))
    bits[0, 5], bits[1, 63], bits[2, 255], bits[3, 128] = 0x7F80, 0xFF80, 0x7FC0, 0xFFFF
    quantize_check(moe, bits)


def test_quantize_rows_in_use(moe):
    """With a layout only the rows that hold an entry are read (others are NaN here) and written."""
    desc = moe.LayoutDesc(9, 2, 4, 2, moe.MOE_PAD_CAPACITY, 7)
    idx = np.random.default_rng(4).integers(0, 4, (9, 2)).astype(np.int32)
    lay = moe.moe_layout(desc, dev(idx))
    used = lay.src.cpu().numpy() >= 0
    for H in (128, 384, 2176):
        bits = normal_bf16_bits(np.random.default_rng(H), (28, H))
        poisoned = np.where(used[:, None], bits, 0x7FA5).astype(np.uint16)
        codes = torch.full((28, H // 2), 0x5A, dtype=torch.uint8, device=DEV)
        scales = torch.full((28, H // 32), 0x5B, dtype=torch.uint8, device=DEV)
        moe.moe_quantize_mx4(dev_bf16(poisoned, DEV), codes, scales, layout=lay)
        wc, ws = mx4_quantize(bf16_values(bits))
        assert np.array_equal(codes.cpu().numpy(), np.where(used[:, None], wc, 0x5A))
        assert np.array_equal(scales.cpu().numpy(), np.where(used[:, None], ws, 0x5B))
        out = torch.full((28, H), 7.0, dtype=torch.bfloat16, device=DEV)
        moe.moe_dequantize_mx4(codes, scales, out=out, layout=lay)
        assert np.array_equal(bf16_values(host_bits(out)), np.where(used[:, None], mx4_values(wc, ws), 7.0))


@pytest.mark.parametrize("H", [1920, 2048, 7168, 8320, 16640])
@pytest.mark.parametrize("S,E,rows", [(61, 9, 31), (3, 16, 1), (0, 4, 5)])
def test_conversions_of_long_rows_in_use(moe, H, S, E, rows):
    """Rows of less than, exactly and many times a wave's channels; rows that are no multiple of the XCDs; a layout
    without an entry."""
    desc = moe.LayoutDesc(S, 2, E, 1, moe.MOE_PAD_CAPACITY, rows)
    rng = np.random.default_rng(H + S)
    lay = moe.moe_layout(desc, dev(rng.integers(0, E, (S, 2)).astype(np.int32)))
    n = E * rows
    used = lay.src.cpu().numpy()[:n] >= 0
    assert used.any() == (S > 0)
    bits = normal_bf16_bits(rng, (n, H))
    codes = torch.full((n, H // 2), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((n, H // 32), 0x5B, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_mx4(dev_bf16(np.where(used[:, None], bits, 0x7FA5).astype(np.uint16), DEV), codes, scales, layout=lay)
    wc, ws = mx4_quantize(bf16_values(bits))
    assert np.array_equal(codes.cpu().numpy(), np.where(used[:, None], wc, 0x5A))
    assert np.array_equal(scales.cpu().numpy(), np.where(used[:, None], ws, 0x5B))
    out = torch.full((n, H), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_dequantize_mx4(codes, scales, out=out, layout=lay)
    assert np.array_equal(bf16_values(host_bits(out)), np.where(used[:, None], mx4_values(wc, ws), 7.0))


def test_quantize_past_4_gib(moe):
    """The last rows of an array whose bytes pass 2^32 (rows repeat, so the reference is small)."""
    H, rows = 7168, 310_000
    bits = normal_bf16_bits(np.random.default_rng(6), (1000, H))
    x = dev_bf16(bits, DEV).repeat(310, 1)
    assert x.numel() * 2 > 1 << 32
    codes, scales = moe.moe_quantize_mx4(x)
    wc, ws = mx4_quantize(bf16_values(bits))
    for r in (0, 149, 299, 309):
        assert np.array_equal(codes[r * 1000:(r + 1) * 1000].cpu().numpy(), wc)
        assert np.array_equal(scales[r * 1000:(r + 1) * 1000].cpu().numpy(), ws)
    x.fill_(0.0)
    moe.moe_dequantize_mx4(codes, scales, out=x)
    v = mx4_values(wc, ws)
    for r in (0, 299, 309):
        assert np.array_equal(bf16_values(host_bits(x[r * 1000:(r + 1) * 1000])), v)


# ---------------------------------------------------------------------------
# dispatch
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("S,K,E,R,H,mode,pad", [
    (1, 1, 1, 1, 128, PAD_NONE, 0), (1, 8, 8, 2, 7168, PAD_NONE, 0), (130, 8, 64, 8, 7168, PAD_CAPACITY, 12),
    (77, 3, 12, 4, 2176, PAD_MULTIPLE, 16), (300, 16, 40, 5, 384, PAD_NONE, 0), (64, 5, 9, 3, 2048, PAD_MULTIPLE, 100),
])
def test_dispatch(moe, S, K, E, R, H, mode, pad):
    rng = np.random.default_rng(S * K + H)
    idx = rng.integers(-1, E, (S, K)).astype(np.int32)   # some ids are not experts; repeats allowed
    hid = normal_bf16_bits(rng, (S, H))
    hid[S // 2, 3] = 0x7FC0
    tw = rng.random((S, K)).astype(np.float32)
    desc = moe.LayoutDesc(S, K, E, R, mode, pad)
    lay = moe.moe_layout(desc, dev(idx))
    rows = moe.moe_max_recv_rows(desc)
    recv = torch.full((rows + 1, H // 2), 0x5A, dtype=torch.uint8, device=DEV)
    sc = torch.full((rows + 1, H // 32), 0x5B, dtype=torch.uint8, device=DEV)
    rw = torch.full((rows + 1,), -7.0, device=DEV)
    moe.moe_dispatch_mx4(desc, lay, dev_bf16(hid, DEV), dev(tw), recv, sc, rw)
    ref = oracle.layout(idx, E, R, mode, pad)
    wc, ws = mx4_quantize(bf16_values(hid))
    want_c, want_s = np.full((rows + 1, H // 2), 0x5A, np.uint8), np.full((rows + 1, H // 32), 0x5B, np.uint8)
    want_w = np.full(rows + 1, -7.0, np.float32)
    held = np.nonzero(ref.src >= 0)[0]
    want_c[held], want_s[held] = wc[ref.src[held] // K], ws[ref.src[held] // K]
    want_w[held] = tw.reshape(-1)[ref.src[held]]
    assert np.array_equal(recv.cpu().numpy(), want_c)
    assert np.array_equal(sc.cpu().numpy(), want_s)
    assert np.array_equal(rw.cpu().numpy(), want_w)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def mx4_random(rng, shape, H, lo, hi):
    """Packed rows of arbitrary codes with scale bytes in [lo, hi]."""
    return (rng.integers(0, 256, (*shape, H // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (*shape, H // 32)).astype(np.uint8))


def expert_of_rows(ref, E, rows):
    out = np.full(rows, -1)
    for e in range(E):
        o = ref.expert_offset[e]
        out[o:o + ref.tokens_per_expert[e]] = e
    return out


def product_check(moe, desc, lay, of_row, xc, xs, wc, ws, act, exact, balance=None, slots=0, stream=None):
    """One call against the reference; rows without an entry hold NaN scales and must keep their output."""
    rows = len(of_row)
    H, M = xc.shape[1] * 2, wc.shape[1]
    swiglu = act == moe.MOE_ACT_SWIGLU
    N = M // 2 if swiglu else M
    xs = np.where(of_row[:, None] < 0, 255, xs).astype(np.uint8)
    out = torch.full((rows + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_gemm_mx4(desc, lay, dev(xc), dev(xs), dev(wc), dev(ws), act, out=out, balance=balance,
                            slots_per_rank=slots, stream=stream)
    torch.cuda.synchronize()
    got_bits = host_bits(out)
    got = bf16_values(got_bits)
    held = of_row >= 0
    assert (got[:rows][~held] == 7.0).all() and (got[rows] == 7.0).all(), "a row without an entry was written"
    y, parts, size = expert_product(mx4_values(xc, xs), mx4_values(wc, ws), of_row, swiglu)
    y, parts, size, got = y[held], parts[held], size[held], got[:rows][held]
    if not held.any():
        return
    if exact and not swiglu:
        assert size.max() * 16 < 2 ** 24, "the data is not exact in fp32"
        assert np.array_equal(got_bits[:rows][held], to_bf16(y))
        return
    err = (0.0 if exact else (H / 128 + 16) * 2.0 ** -23) * size
    if swiglu:
        # silu'(g) lies within [-0.1, 1.1]; five roundings and an exponential that is within 2 units and whose
        # argument |g| carries its own relative rounding: (8 + |g|) units of the result
        g, u = parts[:, :N], parts[:, N:]
        s = np.abs(g / (1 + np.exp(-g)))
        err = 1.1 * err[:, :N] * np.abs(u) + (s + 1.1 * err[:, :N]) * err[:, N:] + (8 + np.abs(g)) * 2.0 ** -23 * np.abs(y)
    bound = err + 2.0 ** -8 * (np.abs(y) + err) + 2.0 ** -126
    off = np.abs(got - y)
    assert np.all(off <= bound), f"off by {np.max(off / bound):.3g} of the bound"


PRODUCTS = [
    # S, K, E, R, H, N, pad mode, pad rows
    (1, 1, 1, 1, 128, 8, PAD_NONE, 0),
    (1, 4, 8, 2, 256, 64, PAD_NONE, 0),
    (1, 8, 16, 1, 1024, 136, PAD_CAPACITY, 4),
    (5, 2, 4, 2, 640, 40, PAD_MULTIPLE, 16),
    (64, 2, 8, 2, 512, 96, PAD_NONE, 0),
    (100, 4, 6, 3, 384, 264, PAD_MULTIPLE, 100),
    (256, 2, 3, 1, 896, 72, PAD_CAPACITY, 130),
    (400, 3, 2, 1, 256, 520, PAD_NONE, 0),
    (33, 16, 80, 8, 256, 24, PAD_NONE, 0),
    (700, 1, 5, 5, 128, 200, PAD_MULTIPLE, 64),
    (1500, 4, 6, 2, 768, 384, PAD_NONE, 0),
    (2000, 2, 300, 4, 512, 272, PAD_MULTIPLE, 8),
    # more tiles than one round of workgroups, and a last round of few
    (30000, 1, 10, 1, 128, 520, PAD_NONE, 0),
    (9000, 3, 7, 1, 256, 776, PAD_NONE, 0),
]


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("S,K,E,R,H,N,mode,pad", PRODUCTS, ids=[f"{p[0]}x{p[1]}e{p[2]}h{p[4]}n{p[5]}" for p in PRODUCTS])
def test_product(moe, S, K, E, R, H, N, mode, pad, act):
    """Ragged segments of every length, some experts without a row, ids that are no expert."""
    rng = np.random.default_rng(S * 7 + H + N)
    p = rng.random(E) ** 3 + 1e-4                        # a few experts get most rows
    idx = rng.choice(E, (S, K), p=p / p.sum()).astype(np.int32)
    idx[rng.random((S, K)) < 0.05] = -1
    desc = moe.LayoutDesc(S, K, E, R, mode, pad)
    lay = moe.moe_layout(desc, dev(idx))
    ref = oracle.layout(idx, E, R, mode, pad)
    rows = len(ref.src)
    swiglu = act == "swiglu"
    code = moe.MOE_ACT_SWIGLU if swiglu else moe.MOE_ACT_NONE
    # scales within a factor of two: every sum is exact (SWIGLU: of a size that silu can tell apart)
    xc, xs = mx4_random(rng, (rows,), H, 127, 128)
    wc, ws = mx4_random(rng, (E, N * (2 if swiglu else 1)), H, 120 if swiglu else 127, 121 if swiglu else 128)
    if swiglu:
        assert H * 144 <= 1 << 24
    product_check(moe, desc, lay, expert_of_rows(ref, E, rows), xc, xs, wc, ws, code, exact=True)


@pytest.mark.parametrize("S", [3, 300, 2000])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_product_any_scale(moe, S, act):
    """Scales over eleven binary orders, and a block of NaN in one row and in one weight row."""
    rng = np.random.default_rng(S)
    K, E, R, H, N = 2, 4, 2, 1152, 104
    idx = rng.integers(0, E, (S, K)).astype(np.int32)
    desc = moe.LayoutDesc(S, K, E, R)
    lay = moe.moe_layout(desc, dev(idx))
    ref = oracle.layout(idx, E, R, PAD_NONE, 0)
    rows = S * K
    M = 2 * N if act == "swiglu" else N
    code = moe.MOE_ACT_SWIGLU if act == "swiglu" else moe.MOE_ACT_NONE
    xc, xs = mx4_random(rng, (rows,), H, 120, 130)
    wc, ws = mx4_random(rng, (E, M), H, 113, 123)
    of_row = expert_of_rows(ref, E, rows)
    product_check(moe, desc, lay, of_row, xc, xs, wc, ws, code, exact=False)
    xs[2, 7], xc[2, 7 * 16:8 * 16] = 255, 0
    out = moe.moe_expert_gemm_mx4(desc, lay, dev(xc), dev(xs), dev(wc), dev(ws), code)
    nan = np.isnan(bf16_values(host_bits(out)))
    assert nan[2].all() and not nan[np.arange(rows) != 2].any()
    xs[2, 7] = 127
    e = of_row[1]
    ws[e, 17, 3], wc[e, 17, 3 * 16:4 * 16] = 255, 0
    out = moe.moe_expert_gemm_mx4(desc, lay, dev(xc), dev(xs), dev(wc), dev(ws), code)
    nan = np.isnan(bf16_values(host_bits(out)))
    assert nan[of_row == e][:, 17].all() and nan.sum() == (of_row == e).sum()


@pytest.mark.parametrize("S,K,E,R,B,H,N", [(40, 2, 8, 4, 2, 256, 40), (600, 4, 16, 4, 6, 384, 136), (700, 2, 24, 2, 0, 128, 64),
                                           (9000, 4, 12, 3, 8, 256, 72), (500, 2, 1024, 8, 64, 128, 16),
                                           (9000, 8, 1024, 8, 64, 384, 264)])
def test_product_balanced(moe, S, K, E, R, B, H, N):
    """Rows of a replica slot use the weights of the expert in it."""
    rng = np.random.default_rng(S)
    p = 1.0 / np.arange(1, E + 1) ** 1.5
    idx = rng.choice(E, (S, K), p=p / p.sum()).astype(np.int32)
    desc = moe.LayoutDesc(S, K, E, R)
    lay, bal = moe.moe_layout_balanced(desc, B, dev(idx))
    src = lay.src.cpu().numpy()
    of_row = np.where(src >= 0, idx.reshape(-1)[np.maximum(src, 0)], -1)
    xc, xs = mx4_random(rng, (S * K,), H, 127, 128)
    wc, ws = mx4_random(rng, (E, N), H, 127, 128)
    product_check(moe, desc, lay, of_row, xc, xs, wc, ws, moe.MOE_ACT_NONE, True, balance=bal, slots=B)


def test_product_no_row_at_all(moe):
    idx = np.full((12, 2), -1, np.int32)
    desc = moe.LayoutDesc(12, 2, 4, 2)
    lay = moe.moe_layout(desc, dev(idx))
    rng = np.random.default_rng(1)
    xc, xs = mx4_random(rng, (24,), 256, 127, 128)
    wc, ws = mx4_random(rng, (4, 16), 256, 127, 128)
    product_check(moe, desc, lay, np.full(24, -1), xc, xs, wc, ws, moe.MOE_ACT_NONE, True)


def test_product_offsets_past_4_gib(moe):
    """Weights and outputs whose bytes pass 2^32: the last expert, and the last rows."""
    E, H, N = 40, 7168, 32768                            # 4.7 GB of weights
    assert E * N * H // 2 > 1 << 32
    rng = np.random.default_rng(5)
    S = 70000
    idx = np.full((S, 1), E - 1, np.int32)
    idx[:3, 0] = [0, E - 2, -1]
    desc = moe.LayoutDesc(S, 1, E, 1)
    lay = moe.moe_layout(desc, dev(idx))
    xc, xs = mx4_random(rng, (64,), H, 127, 127)
    reps = -(-S // 64)
    X, XS = dev(xc).repeat(reps, 1)[:S].contiguous(), dev(xs).repeat(reps, 1)[:S].contiguous()
    wc, ws = mx4_random(rng, (512,), H, 120, 120)
    W = dev(wc).repeat(E * N // 512, 1).view(E, N, H // 2)
    WS = dev(ws).repeat(E * N // 512, 1).view(E, N, H // 32)
    WS[E - 1].add_(1)                                    # the last expert's weights are twice the others'
    out = moe.moe_expert_gemm_mx4(desc, lay, X, XS, W, WS)
    assert out.numel() * 2 > 1 << 32
    y = mx4_values(xc, xs) @ mx4_values(wc, ws).T        # [64,512]; sums of at most 7168 * 36 quarters: exact
    for r in (0, 1, 2, 40000, S - 2):
        want = y[r % 64] * (1.0 if r < 2 else 2.0)
        got = host_bits(out[r]).reshape(-1, 512)
        assert np.array_equal(got, np.broadcast_to(to_bf16(want), got.shape)), r


def test_product_on_streams_and_in_a_graph(moe):
    rng = np.random.default_rng(9)
    S, K, E, H, N = 200, 2, 6, 512, 136
    desc = moe.LayoutDesc(S, K, E, 2)
    idx = dev(rng.integers(0, E, (S, K)).astype(np.int32))
    xc, xs = (dev(a) for a in mx4_random(rng, (S * K,), H, 120, 130))
    wc, ws = (dev(a) for a in mx4_random(rng, (E, 2 * N), H, 115, 121))
    lay = moe.moe_layout(desc, idx)
    want = moe.moe_expert_gemm_mx4(desc, lay, xc, xs, wc, ws, moe.MOE_ACT_SWIGLU)
    torch.cuda.synchronize()
    got = [moe.moe_expert_gemm_mx4(desc, lay, xc, xs, wc, ws, moe.MOE_ACT_SWIGLU, stream=s)
           for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    with moe.CULimitedStream(64) as cu:
        got.append(moe.moe_expert_gemm_mx4(desc, lay, xc, xs, wc, ws, moe.MOE_ACT_SWIGLU, stream=cu.stream))
        torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_layout(desc, idx, lay)
        moe.moe_expert_gemm_mx4(desc, lay, xc, xs, wc, ws, moe.MOE_ACT_SWIGLU, out=out)
    for k in range(4):                                   # new routing between replays
        idx.copy_(torch.from_numpy(rng.integers(0, E, (S, K)).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        eager = moe.moe_expert_gemm_mx4(desc, moe.moe_layout(desc, idx), xc, xs, wc, ws, moe.MOE_ACT_SWIGLU)
        assert torch.equal(out, eager)


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("case", ["plain", "capacity", "balanced"])
def test_layer(moe, case):
    """Router, dispatch, gate and up products with SwiGLU, quantise, down product, combine, through Buffer; every
    step against its reference on the step's own inputs."""
    S, H, K, E, R, F = 150, 512, 4, 16, 4, 256
    rng = np.random.default_rng(77)
    kw = dict(plain={}, capacity=dict(pad_mode=PAD_CAPACITY, pad_rows=60), balanced=dict(balance_slots=4))[case]
    buf = moe.Buffer(S=S, H=H, K=K, E=E, R=R, mx4=True, device=DEV, **kw)
    hid = normal_bf16_bits(rng, (S, H))
    z = rng.standard_normal((S, E)).astype(np.float32)
    z[:, 0] += 1.5                                       # a hot expert
    mask = np.ones(S, bool)
    mask[140:] = False                                   # the batch's padding
    rd = moe.RouterDesc(S, E, K, n_groups=4, topk_groups=3)
    r = moe.moe_router(rd, dev(z), dev(mask), loss=False)
    recv, recv_w, _, scales = buf.dispatch(dev_bf16(hid, DEV), r.topk_w, r.topk_idx)
    wb = normal_bf16_bits(rng, (E * 2 * F, H)).reshape(E, 2 * F, H)
    db = normal_bf16_bits(rng, (E * H, F)).reshape(E, H, F)
    up = moe.moe_quantize_mx4(dev_bf16(wb, DEV).mul_(2.0 ** -5))
    down = moe.moe_quantize_mx4(dev_bf16(db, DEV).mul_(2.0 ** -4))
    h = buf.expert_gemm(*up, act=moe.MOE_ACT_SWIGLU)
    h4 = moe.moe_quantize_mx4(h, layout=buf.layout)
    y = buf.expert_gemm(*down, x=h4[0], x_scales=h4[1])
    out = buf.combine(y, r.topk_w)
    torch.cuda.synchronize()

    ref = router_rows(z, K, mask)
    idx = r.topk_idx.cpu().numpy()
    assert np.array_equal(idx, ref)
    src = buf.layout.src.cpu().numpy()
    held = src >= 0
    assert held.sum() == 140 * K or case == "capacity"
    of_row = np.where(held, idx.reshape(-1)[np.maximum(src, 0)], -1)
    wc, ws = mx4_quantize(bf16_values(hid))
    assert np.array_equal(recv.cpu().numpy()[held], wc[src[held] // K])
    assert np.array_equal(scales.cpu().numpy()[held], ws[src[held] // K])
    wv = mx4_values(*(t.cpu().numpy().reshape(E * 2 * F, -1) for t in up)).reshape(E, 2 * F, H)
    x = np.zeros((len(src), H))
    x[held] = mx4_values(wc, ws)[src[held] // K]
    want, parts, size = expert_product(x, wv, of_row, True)
    err = (H / 128 + 16) * 2.0 ** -23 * size[held]
    g, u = parts[held][:, :F], parts[held][:, F:]
    s = np.abs(g / (1 + np.exp(-g)))
    e = 1.1 * err[:, :F] * np.abs(u) + (s + 1.1 * err[:, :F]) * err[:, F:] + (8 + np.abs(g)) * 2.0 ** -23 * np.abs(want[held])
    hv = bf16_values(host_bits(h))[held]
    assert np.all(np.abs(hv - want[held]) <= e + 2.0 ** -8 * (np.abs(want[held]) + e))
    hc, hs = mx4_quantize(hv)
    assert np.array_equal(h4[0].cpu().numpy()[held], hc) and np.array_equal(h4[1].cpu().numpy()[held], hs)
    x2 = np.zeros((len(src), F))
    x2[held] = mx4_values(hc, hs)
    dv = mx4_values(*(t.cpu().numpy().reshape(E * H, -1) for t in down)).reshape(E, H, F)
    want, _, size = expert_product(x2, dv, of_row, False)
    yv = host_bits(y)
    e = (F / 128 + 16) * 2.0 ** -23 * size[held]
    assert np.all(np.abs(bf16_values(yv)[held] - want[held]) <= e + 2.0 ** -8 * (np.abs(want[held]) + e))
    ybits = np.where(held[:, None], yv, np.uint16(0)).astype(np.uint16)
    got = host_bits(out)
    assert np.array_equal(got, oracle.combine(ybits, buf.layout.pos.cpu().numpy(), r.topk_w.cpu().numpy()))
    assert not got[140:].any()                           # tokens that do not count


def test_layer_in_graphs(moe):
    """The layer of two micro-batches, each captured into a graph of its own, replayed in turn and at the same time
    with new tokens and weights, eager work between: every replay as the eager calls."""
    S, H, K, E, R, F = 130, 384, 3, 12, 3, 128
    rng = np.random.default_rng(78)
    rd = moe.RouterDesc(S, E, K, n_groups=3, topk_groups=2, seq_len=65, alpha=0.1)
    up = moe.moe_quantize_mx4(dev_bf16(normal_bf16_bits(rng, (E * 2 * F, H)).reshape(E, 2 * F, H), DEV).mul_(2.0 ** -5))
    down = moe.moe_quantize_mx4(dev_bf16(normal_bf16_bits(rng, (E * H, F)).reshape(E, H, F), DEV).mul_(2.0 ** -4))

    def layer(buf, z, hid):
        r = moe.moe_router(rd, z)
        buf.dispatch(hid, r.topk_w, r.topk_idx)
        h = buf.expert_gemm(*up, act=moe.MOE_ACT_SWIGLU)
        h4 = moe.moe_quantize_mx4(h, layout=buf.layout)
        out = buf.combine(buf.expert_gemm(*down, x=h4[0], x_scales=h4[1]), r.topk_w)
        d = moe.moe_router_backward(rd, z, r, d_topk_w=torch.ones_like(r.topk_w), d_loss=torch.ones(1, device=DEV))
        return out, r.topk_idx, r.topk_w, r.expert_count, r.balance_loss, d

    def fresh():
        return dev(rng.standard_normal((S, E)).astype(np.float32)), dev_bf16(normal_bf16_bits(rng, (S, H)), DEV)

    bufs = [moe.Buffer(S=S, H=H, K=K, E=E, R=R, mx4=True, device=DEV) for _ in range(3)]
    ins = [fresh(), fresh()]
    layer(bufs[2], *ins[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b, i in zip(bufs, ins):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(b, *i))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(4):
        want = []
        for i in ins:
            for t, n in zip(i, fresh()):
                t.copy_(n)
            want.append([t.clone() for t in layer(bufs[2], *i)])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):                # at the same time, or one behind the other
            with torch.cuda.stream(s if k % 2 else streams[0]):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w)), k


def router_rows(z, K, mask):
    from router_mx4_reference import router_reference
    return router_reference(z.astype(np.float64), K, n_groups=4, topk_groups=3, mask=mask)["idx"]


def test_python_refusals(moe):
    desc = moe.LayoutDesc(4, 2, 4, 2)
    lay = moe.alloc_layout(desc, torch.device(DEV))
    u8 = dict(dtype=torch.uint8, device=DEV)
    x, xs = torch.zeros((8, 128), **u8), torch.zeros((8, 8), **u8)
    w, ws = torch.zeros((4, 16, 128), **u8), torch.zeros((4, 16, 8), **u8)
    for bad in (dict(x=x[:7]), dict(xs=xs[:, :4].contiguous()), dict(w=w[:3]), dict(ws=ws[:, :8].contiguous()),
                dict(x=torch.zeros((8, 256), **u8)[:, ::2]), dict(out=torch.zeros((7, 16), dtype=torch.bfloat16, device=DEV)),
                dict(balance=moe.alloc_balance(desc, 3, torch.device(DEV)), slots_per_rank=2)):
        kw = dict(x=x, xs=xs, w=w, ws=ws)
        rest = {k: v for k, v in bad.items() if k not in kw}
        kw.update({k: v for k, v in bad.items() if k in kw})
        with pytest.raises(ValueError):
            moe.moe_expert_gemm_mx4(desc, lay, kw["x"], kw["xs"], kw["w"], kw["ws"], **rest)
    with pytest.raises(TypeError):
        moe.moe_expert_gemm_mx4(desc, lay, x.to(torch.int8), xs, w, ws)
    with pytest.raises(moe.MoeError):
        moe.moe_expert_gemm_mx4(desc, lay, x, xs, w[:, :12].contiguous(), ws[:, :12].contiguous())
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_mx4(torch.zeros((2, 96), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        moe.moe_quantize_mx4(torch.zeros((9, 128), dtype=torch.bfloat16, device=DEV), layout=lay)
    with pytest.raises(moe.MoeError):
        moe.Buffer(S=4, H=128, K=2, E=4, R=2, fp8=True, mx4=True, device=DEV)
