"""What the bf16 and 8-bit products, their gradients, the 8-bit rows and combine's gradient refuse, and the sizes they
take.  Every call here returns before anything is enqueued."""
from __future__ import annotations

import ctypes

import pytest
import torch

P = ctypes.c_void_p
FAKE = 1 << 20   # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def moe():
    import os
    from combine_moe_layout_02_amd.build import LIB
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def bufs(moe, **over):
    fields = {n: FAKE + 4096 * i for i, (n, _) in enumerate(moe.moe_layout_bufs._fields_)}
    fields.update(over)
    return moe.moe_layout_bufs(**fields)


CALLS = ("forward", "backward_x", "backward_w", "int8")


def call(moe, which, desc=None, layout=None, bal=None, slots=0, H=64, N=64, act=0, x=FAKE, w=FAKE, out=FAKE, pre=None, xs=FAKE,
         ws=FAKE, dtype=0, pre_type=1):
    L = moe.lib()
    desc = moe.LayoutDesc(64, 2, 8, 2) if desc is None else desc
    layout = bufs(moe) if layout is None else layout
    d = None if desc == "null" else ctypes.byref(desc.c())
    b = None if layout == "null" else ctypes.byref(layout)
    bal = None if bal is None else ctypes.byref(bal)
    if which == "forward":
        return L.moe_expert_gemm(d, b, bal, slots, P(x), H, P(w), N, act, P(pre), pre_type, P(out), None)
    if which == "backward_x":
        return L.moe_expert_gemm_backward_x(d, b, bal, slots, P(x), N, P(w), H, P(pre), pre_type, P(out), None)
    if which == "backward_w":
        return L.moe_expert_gemm_backward_w(d, b, bal, slots, P(x), N, P(w), H, dtype, P(out), None)
    return L.moe_expert_gemm_i8(d, b, bal, slots, P(x), P(xs), H, P(w), P(ws), N, act, P(out), None)


@pytest.mark.parametrize("which", CALLS)
def test_products(moe, which):
    E = moe
    for bad in (dict(desc="null"), dict(layout="null"), dict(x=None), dict(w=None), dict(out=None),
                dict(layout=bufs(moe, tokens_per_expert=None)), dict(layout=bufs(moe, expert_offset=None))):
        assert call(moe, which, **bad) == E.MOE_ERR_NULL, bad
    for bad in (dict(H=0), dict(H=-8), dict(H=60), dict(N=0), dict(N=12), dict(N=(1 << 22) + 8), dict(H=(1 << 22) + 16),
                dict(desc=moe.LayoutDesc(64, 2, 8, 3)), dict(desc=moe.LayoutDesc(-1, 2, 8, 2)), dict(slots=1)):
        assert call(moe, which, **bad) == E.MOE_ERR_SHAPE, bad
    for bad in (dict(x=FAKE + 8), dict(w=FAKE + 4), dict(out=FAKE + 8), dict(layout=bufs(moe, tokens_per_expert=FAKE + 2)),
                dict(layout=bufs(moe, expert_offset=FAKE + 1))):
        assert call(moe, which, **bad) == E.MOE_ERR_ALIGN, bad


@pytest.mark.parametrize("which", CALLS)
def test_balanced_layouts(moe, which):
    bal = moe.moe_balance_bufs(FAKE, FAKE + 4096)
    padded = moe.LayoutDesc(64, 2, 8, 2, moe.MOE_PAD_MULTIPLE, 16)
    for bad in (dict(desc=padded, bal=bal, slots=1), dict(bal=bal, slots=-1), dict(bal=bal, slots=65),
                dict(desc=moe.LayoutDesc(64, 2, 64, 32), bal=bal, slots=17)):
        assert call(moe, which, **bad) == moe.MOE_ERR_SHAPE, bad
    assert call(moe, which, bal=moe.moe_balance_bufs(None, FAKE), slots=1) == moe.MOE_ERR_NULL
    assert call(moe, which, bal=moe.moe_balance_bufs(FAKE, None), slots=1) == moe.MOE_ERR_NULL
    assert call(moe, which, bal=moe.moe_balance_bufs(FAKE + 2, FAKE), slots=1) == moe.MOE_ERR_ALIGN


def test_what_only_some_take(moe):
    assert call(moe, "forward", act=2) == moe.MOE_ERR_SHAPE
    assert call(moe, "int8", act=2) == moe.MOE_ERR_SHAPE
    assert call(moe, "forward", pre=FAKE) == moe.MOE_ERR_SHAPE          # only with the activation
    assert call(moe, "forward", act=1, pre=FAKE + 8) == moe.MOE_ERR_ALIGN
    assert call(moe, "backward_x", pre=FAKE + 8) == moe.MOE_ERR_ALIGN
    assert call(moe, "forward", act=1, pre=FAKE, pre_type=2) == moe.MOE_ERR_SHAPE
    assert call(moe, "backward_x", pre=FAKE, pre_type=-1) == moe.MOE_ERR_SHAPE
    assert call(moe, "backward_x", pre=FAKE, pre_type=0, out=FAKE) == moe.MOE_ERR_SHAPE     # fp32: not into itself
    assert call(moe, "backward_w", dtype=2) == moe.MOE_ERR_SHAPE
    # rows of more than 2^23 bytes of results
    most = 1 << 21
    for which, kw in (("forward", dict(N=most, act=1)), ("int8", dict(N=most, act=1)), ("backward_x", dict(H=most, pre=FAKE)),
                      ("backward_w", dict(H=most, dtype=0))):
        assert call(moe, which, out=None, **kw) == moe.MOE_ERR_NULL
        size = "N" if "N" in kw else "H"
        assert call(moe, which, out=None, **{**kw, size: most + 8}) == moe.MOE_ERR_SHAPE
    for which, kw in (("forward", dict(N=most // 2, act=1)), ("backward_x", dict(H=most // 2))):
        kw.update(pre=FAKE, pre_type=0)
        assert call(moe, which, out=None, **kw) == moe.MOE_ERR_NULL
        size = "N" if "N" in kw else "H"
        assert call(moe, which, out=None, **{**kw, size: most // 2 + 8}) == moe.MOE_ERR_SHAPE
    assert call(moe, "backward_w", H=1 << 22, dtype=1, out=None) == moe.MOE_ERR_NULL
    assert call(moe, "int8", H=72) == moe.MOE_ERR_SHAPE
    assert call(moe, "int8", H=131072) == moe.MOE_ERR_SHAPE             # 131072 * 128 * 128 passes 32 bits
    assert call(moe, "int8", H=131056, x=None) == moe.MOE_ERR_NULL
    assert call(moe, "int8", xs=None) == moe.MOE_ERR_NULL
    assert call(moe, "int8", ws=None) == moe.MOE_ERR_NULL
    assert call(moe, "int8", xs=FAKE + 2) == moe.MOE_ERR_ALIGN


@pytest.mark.parametrize("which", CALLS)
def test_empty_batch(moe, which):
    """Nothing to do, but for the weights' gradient, which has to be written."""
    empty = moe.LayoutDesc(0, 2, 8, 2)
    want = moe.MOE_ERR_NULL if which == "backward_w" else moe.MOE_OK
    assert call(moe, which, desc=empty, x=None, w=None, out=None) == want


@pytest.mark.parametrize("which", CALLS)
@pytest.mark.parametrize("S,K,E", [(1, 1, 1), (1, 8, 256), (256, 1, 256), (1000, 8, 1024), (16, 16, 16), (4096, 8, 64), (1 << 20, 4, 8)])
def test_sizes_taken(moe, which, S, K, E):
    """The sizes that include/moe_ep.h says a launch can always number: the call gets as far as its missing array."""
    desc = moe.LayoutDesc(S, K, E, 1)
    row_tiles = S * K // 16 + min(E, S * K)
    tiles = min(((1 << 23) - 8) // row_tiles, 1 << 17)
    for act in (0, 1) if which in ("forward", "int8") else (0,):
        if which == "backward_w":
            side = int((((1 << 24) - 16) // E) ** 0.5) * 64
            assert call(moe, which, desc=desc, H=min(side, 1 << 22), N=min(side, 1 << 22), out=None) == moe.MOE_ERR_NULL
            continue
        c = tiles * (16 if act else 32)
        for inner in (64, 131056):
            kw = dict(H=c, N=inner) if which == "backward_x" else dict(H=inner, N=c, act=act)
            assert call(moe, which, desc=desc, out=None, **kw) == moe.MOE_ERR_NULL, kw


@pytest.mark.parametrize("H", [16, 2048, 7168, 1 << 22])
def test_int8_rows(moe, H):
    L, most = moe.lib(), (1 << 23) - 8
    for rows, want in ((most, moe.MOE_ERR_NULL), (most + 1, moe.MOE_ERR_SHAPE), (-1, moe.MOE_ERR_SHAPE), (0, moe.MOE_OK)):
        assert L.moe_quantize_i8(None, rows, H, None, None, None, None) == want
        assert L.moe_dequantize_i8(None, None, rows, H, None, None, None) == want
    for bad in (0, 8, H + 8, (1 << 22) + 16):
        assert L.moe_quantize_i8(P(FAKE), 1, bad, None, P(FAKE), P(FAKE), None) == moe.MOE_ERR_SHAPE
        assert L.moe_dequantize_i8(P(FAKE), P(FAKE), 1, bad, None, P(FAKE), None) == moe.MOE_ERR_SHAPE
    for i in range(3):
        a = [P(FAKE)] * 3
        a[i] = P(FAKE + 2)
        assert L.moe_quantize_i8(a[0], 1, H, None, a[1], a[2], None) == moe.MOE_ERR_ALIGN
        assert L.moe_dequantize_i8(a[1], a[2], 1, H, None, a[0], None) == moe.MOE_ERR_ALIGN


def test_dispatch_i8(moe):
    L = moe.lib()
    b = bufs(moe)

    def go(desc=moe.LayoutDesc(64, 2, 8, 2), layout=b, hidden=FAKE, H=64, w=None, recv=FAKE, scales=FAKE, recv_w=None):
        return L.moe_dispatch_i8(None if desc is None else ctypes.byref(desc.c()), None if layout is None else ctypes.byref(layout),
                                 P(hidden), H, P(w), P(recv), P(scales), P(recv_w), None)

    for bad in (dict(desc=None), dict(layout=None), dict(hidden=None), dict(recv=None), dict(scales=None), dict(layout=bufs(moe, pos=None))):
        assert go(**bad) == moe.MOE_ERR_NULL, bad
    for bad in (dict(H=72), dict(H=0), dict(desc=moe.LayoutDesc(64, 2, 8, 3)), dict(desc=moe.LayoutDesc((1 << 23) - 7, 1, 8, 2))):
        assert go(**bad) == moe.MOE_ERR_SHAPE, bad
    for bad in (dict(hidden=FAKE + 8), dict(recv=FAKE + 8), dict(scales=FAKE + 2), dict(w=FAKE + 1), dict(recv_w=FAKE + 2),
                dict(layout=bufs(moe, pos=FAKE + 2))):
        assert go(**bad) == moe.MOE_ERR_ALIGN, bad
    assert go(desc=moe.LayoutDesc(0, 2, 8, 2), hidden=None, recv=None) == moe.MOE_OK
    assert go(desc=moe.LayoutDesc((1 << 23) - 8, 1, 8, 2), hidden=None) == moe.MOE_ERR_NULL


def test_combine_backward(moe):
    L = moe.lib()
    b = bufs(moe)

    def go(desc=moe.LayoutDesc(64, 2, 8, 2), layout=b, d_out=FAKE, H=64, y=FAKE, w=None, d_y=FAKE, d_w=FAKE):
        return L.moe_combine_backward(None if desc is None else ctypes.byref(desc.c()), None if layout is None else ctypes.byref(layout),
                                      P(d_out), H, P(y), P(w), P(d_y), P(d_w), None)

    for bad in (dict(desc=None), dict(layout=None), dict(d_out=None), dict(y=None), dict(d_y=None, d_w=None), dict(layout=bufs(moe, pos=None))):
        assert go(**bad) == moe.MOE_ERR_NULL, bad
    for bad in (dict(H=4), dict(H=12), dict(H=(1 << 22) + 8), dict(desc=moe.LayoutDesc(64, 2, 8, 3)), dict(desc=moe.LayoutDesc(1 << 23, 1, 8, 2))):
        assert go(**bad) == moe.MOE_ERR_SHAPE, bad
    for bad in (dict(d_out=FAKE + 8), dict(y=FAKE + 8), dict(d_y=FAKE + 8), dict(w=FAKE + 2), dict(d_w=FAKE + 2),
                dict(layout=bufs(moe, pos=FAKE + 2))):
        assert go(**bad) == moe.MOE_ERR_ALIGN, bad
    assert go(desc=moe.LayoutDesc(0, 2, 8, 2), d_out=None, y=None) == moe.MOE_OK
    assert go(desc=moe.LayoutDesc((1 << 23) - 1, 1, 8, 2), d_out=None) == moe.MOE_ERR_NULL


def test_host_tensors(moe):
    """The bindings refuse tensors that are not on a device, before the library is called."""
    desc = moe.LayoutDesc(4, 1, 2, 1)
    i32 = dict(dtype=torch.int32)
    lay = moe.Layout(torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros((4, 1), **i32),
                     torch.zeros(4, **i32), torch.zeros(1, **i32))
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    w = torch.zeros((2, 16, 16), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4)
    for go in (lambda: moe.moe_expert_gemm(desc, lay, x, w), lambda: moe.moe_expert_gemm_backward_x(desc, lay, x, w),
               lambda: moe.moe_expert_gemm_backward_w(desc, lay, x, x), lambda: moe.moe_combine_backward(desc, lay, x, x),
               lambda: moe.moe_quantize_i8(x), lambda: moe.moe_dequantize_i8(q, s), lambda: moe.moe_dispatch_i8(desc, lay, x),
               lambda: moe.moe_expert_gemm_i8(desc, lay, q, s, torch.zeros((2, 16, 16), dtype=torch.int8), torch.zeros((2, 16)))):
        with pytest.raises(ValueError, match="device tensor"):
            go()


def test_outputs_over_inputs(moe):
    """An output that is an input's own buffer is refused where the call does not allow it."""
    other = [FAKE + (1 << 20) * i for i in range(1, 8)]
    for which in CALLS:
        for kw in (dict(x=other[0], w=other[1], out=other[0]), dict(x=other[0], w=other[1], out=other[1])):
            assert call(moe, which, xs=other[2], ws=other[3], **kw) == moe.MOE_ERR_SHAPE, (which, kw)
    for same in other[:3]:
        assert call(moe, "forward", act=1, x=other[0], w=other[1], out=other[2], pre=same, pre_type=0) == moe.MOE_ERR_SHAPE
    assert call(moe, "backward_x", x=other[0], w=other[1], out=other[2], pre=other[2], pre_type=0) == moe.MOE_ERR_SHAPE
    L, a, b, c, d = moe.lib(), *other[:4]
    assert L.moe_quantize_i8(P(a), 4, 16, None, P(a), P(b), None) == moe.MOE_ERR_SHAPE
    assert L.moe_dequantize_i8(P(a), P(b), 4, 16, None, P(a), None) == moe.MOE_ERR_SHAPE
    desc, layout = ctypes.byref(moe.LayoutDesc(64, 2, 8, 2).c()), ctypes.byref(bufs(moe))
    assert L.moe_dispatch_i8(desc, layout, P(a), 16, None, P(a), P(b), None, None) == moe.MOE_ERR_SHAPE
    assert L.moe_combine_backward(desc, layout, P(a), 16, P(b), P(c), P(a), P(d), None) == moe.MOE_ERR_SHAPE
    assert L.moe_combine_backward(desc, layout, P(a), 16, P(b), P(c), P(d), P(c), None) == moe.MOE_ERR_SHAPE
