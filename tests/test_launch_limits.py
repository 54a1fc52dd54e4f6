"""The sizes that include/moe_ep.h says every call takes, on the edge of what it says, and the refusal beyond.  A call
that takes a shape gets as far as its next check, a missing array; nothing is enqueued."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE = 1 << 20   # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_02_amd.build import LIB
    import os
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


@pytest.mark.parametrize("chunks", [1, 2, 3, 4, 7])
def test_dispatch_mx4(moe, chunks):
    bufs = moe.moe_layout_bufs(pos=FAKE)

    def call(S):
        d = moe.LayoutDesc(S, 1, 8, 1).c()
        return moe.lib().moe_dispatch_mx4(ctypes.byref(d), ctypes.byref(bufs), None, 2048 * chunks - 1920, None, None, None, None,
                                          None)

    most = ((1 << 26) - 1) // chunks
    assert call(most) == moe.MOE_ERR_NULL
    assert call(most + 1) == moe.MOE_ERR_SHAPE


@pytest.mark.parametrize("H", [128, 384, 7168, 1 << 20])
def test_conversions(moe, H):
    L = moe.lib()
    most = ((1 << 37) - 8192) // H
    for rows, want in ((most, moe.MOE_ERR_NULL), (most + 1, moe.MOE_ERR_SHAPE)):
        assert L.moe_quantize_mx4(None, rows, H, None, None, None, None) == want
        assert L.moe_dequantize_mx4(None, None, rows, H, None, None, None) == want


def test_router_without_the_loss(moe):
    L = moe.lib()
    bufs = moe.moe_router_bufs()
    for S, want in (((1 << 26) - 5, moe.MOE_ERR_NULL), ((1 << 26) - 4, moe.MOE_ERR_SHAPE)):
        d = moe.RouterDesc(S, 8, 1).c()
        assert L.moe_router(ctypes.byref(d), None, 0, None, ctypes.byref(bufs), None, 0, None) == want
        assert L.moe_router_backward(ctypes.byref(d), None, 0, None, None, None, None, P(FAKE), None, None, None) == want


@pytest.mark.parametrize("E", [1, 8, 32, 33, 64, 65, 256, 257, 512, 513, 1000, 1024])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 100, 1000, 4095, 4096, 4097, 5000, 9000, 100000, 1 << 22])
def test_router_with_the_loss(moe, E, T):
    """The workspace's size is 0 for a shape that is refused."""
    cells, parts = -(-E // 32), min(-(-T // 16), 256)
    G = min(((1 << 22) - 1) // max(cells, parts), ((1 << 26) - 5) // T)
    assert G > 0

    def taken(G):
        return moe.moe_router_workspace_bytes(moe.RouterDesc(G * T, E, 1, seq_len=T)) > 0

    assert taken(G)
    # with at most 256 experts and 4096 tokens to a sequence nothing more is taken
    if E <= 256 and T <= 4096 and (G + 1) * max(cells, parts) >= 1 << 22:
        assert not taken(G + 1)


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("S,K,E", [(1, 1, 1), (1, 8, 256), (256, 1, 256), (1000, 8, 1024), (16, 16, 16), (4096, 8, 64), (1 << 20, 4, 8)])
def test_products(moe, S, K, E, act):
    d, bufs = moe.LayoutDesc(S, K, E, 1), moe.moe_layout_bufs()
    row_tiles = S * K // 16 + min(E, S * K)
    weight_tiles = min(((1 << 23) - 8) // row_tiles, 1 << 17)
    N = weight_tiles * (16 if act else 32)
    for H in (128, 7168, 1 << 22):
        assert moe.lib().moe_expert_gemm_mx4(ctypes.byref(d.c()), ctypes.byref(bufs), None, 0, None, None, H, None, None, N, act, None,
                                             None) == moe.MOE_ERR_NULL
