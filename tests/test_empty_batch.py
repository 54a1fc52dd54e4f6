"""A batch without a token: its arrays are empty, and an empty array's address is NULL.  Every call of a layer takes it
and enqueues nothing."""
from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    import os
    from combine_moe_layout_02_amd.build import LIB
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


def test_no_token(moe):
    L = moe.lib()
    d, b = ctypes.byref(moe.LayoutDesc(0, 2, 4, 2).c()), ctypes.byref(moe.moe_layout_bufs())
    assert L.moe_dispatch(d, b, None, 64, None, None, 0, None, None, None, None) == moe.MOE_OK
    assert L.moe_zero_padding(d, b, 64, 0, None, None, None) == moe.MOE_OK
    assert L.moe_dispatch_i8(d, b, None, 64, None, None, None, None, None) == moe.MOE_OK
    assert L.moe_quantize_i8(None, 0, 64, None, None, None, None) == moe.MOE_OK
    assert L.moe_dequantize_i8(None, None, 0, 64, None, None, None) == moe.MOE_OK
    for act in (0, 1):
        assert L.moe_expert_gemm(d, b, None, 0, None, 64, None, 64, act, None, 0, None, None) == moe.MOE_OK
        assert L.moe_expert_gemm_i8(d, b, None, 0, None, None, 64, None, None, 64, act, None, None) == moe.MOE_OK
    assert L.moe_expert_gemm_backward_x(d, b, None, 0, None, 64, None, 64, None, 0, None, None) == moe.MOE_OK
    assert L.moe_combine(d, b, None, 64, None, None, None, None) == moe.MOE_OK
    assert L.moe_combine_backward(d, b, None, 64, None, None, None, None, None) == moe.MOE_OK
