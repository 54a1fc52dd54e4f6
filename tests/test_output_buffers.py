"""An output of the bf16 and 8-bit calls that is the buffer of something the call reads, or of another output, is refused:
every pair of arguments, but for the two that the header allows.  The calls get addresses that nothing lies at, so they are
made only where there is no GPU: one that is not refused ends there at its launch."""
from __future__ import annotations

import ctypes

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would be enqueued")
P = ctypes.c_void_p
S, K, E, H, N = 64, 2, 8, 64, 64


@pytest.fixture(scope="module")
def moe():
    import os
    from combine_moe_layout_02_amd.build import LIB
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


# A call's outputs and what it reads; the arrays of the layout by their field's name.
SEGMENTS = ("tokens_per_expert", "expert_offset")
BALANCED = ("seg_offset", "slot_expert")
CALLS = {
    "forward": (("out",), ("x", "w") + SEGMENTS),
    "forward balanced": (("out",), ("x", "w") + BALANCED),
    "forward kept": (("out", "pre"), ("x", "w") + SEGMENTS),
    "backward_x": (("out",), ("x", "w") + SEGMENTS),
    "backward_x fp32 pre": (("out",), ("x", "w", "pre") + SEGMENTS),
    "backward_x bf16 pre": (("out",), ("x", "w") + SEGMENTS),          # into pre is allowed
    "backward_w": (("out",), ("x", "w") + SEGMENTS),
    "backward_w balanced": (("out",), ("x", "w") + BALANCED),
    "int8": (("out",), ("x", "w", "xs", "ws") + SEGMENTS),
    "quantize": (("out", "scales"), ("x", "src")),
    "dequantize": (("out",), ("x", "xs", "src")),
    "dispatch": (("out", "scales", "recv_w"), ("x", "tw", "pos")),
    "combine_backward": (("out", "d_w"), ("x", "tw", "pos")),                 # the rows into expert_out is allowed
    "combine_backward weights": (("d_w",), ("x", "y", "tw", "pos")),
}
PAIRS = [(name, o, i) for name, (outs, ins) in CALLS.items() for o in outs for i in ins + outs if o != i]


def call(moe, name, at):
    """The call with each argument at its address of `at`."""
    L, d = moe.lib(), ctypes.byref(moe.LayoutDesc(S, K, E, 2).c())
    lay = ctypes.byref(moe.moe_layout_bufs(**{n: at.get(n) for n, _ in moe.moe_layout_bufs._fields_}))
    bal = ctypes.byref(moe.moe_balance_bufs(at["seg_offset"], at["slot_expert"])) if "balanced" in name else None
    slots = 1 if "balanced" in name else 0
    a = {k: P(v) for k, v in at.items()}
    if name.startswith("forward"):
        kept = "kept" in name
        return L.moe_expert_gemm(d, lay, bal, slots, a["x"], H, a["w"], N, int(kept), a["pre"] if kept else None, 0, a["out"], None)
    if name.startswith("backward_x"):
        pre = a["pre"] if "pre" in name else None
        return L.moe_expert_gemm_backward_x(d, lay, bal, slots, a["x"], N, a["w"], H, pre, 1 if "bf16" in name else 0, a["out"], None)
    if name.startswith("backward_w"):
        return L.moe_expert_gemm_backward_w(d, lay, bal, slots, a["x"], N, a["w"], H, 0, a["out"], None)
    if name == "int8":
        return L.moe_expert_gemm_i8(d, lay, bal, slots, a["x"], a["xs"], H, a["w"], a["ws"], N, 0, a["out"], None)
    if name == "quantize":
        return L.moe_quantize_i8(a["x"], 4, H, a["src"], a["out"], a["scales"], None)
    if name == "dequantize":
        return L.moe_dequantize_i8(a["x"], a["xs"], 4, H, a["src"], a["out"], None)
    if name == "dispatch":
        return L.moe_dispatch_i8(d, lay, a["x"], H, a["tw"], a["out"], a["scales"], a["recv_w"], None)
    rows = None if "weights" in name else a["out"]
    return L.moe_combine_backward(d, lay, a["x"], H, a["y"], a["tw"], rows, a["d_w"], None)


def addresses():
    """A 16-byte aligned address for each argument."""
    names = sorted({n for outs, ins in CALLS.values() for n in outs + ins} | {"pre", "y"})
    return {n: (1 << 20) * (i + 1) for i, n in enumerate(names)}


@pytest.mark.parametrize("name,output,other", PAIRS, ids=[f"{n}: {o} is {i}" for n, o, i in PAIRS])
def test_refused(moe, name, output, other):
    at = addresses()
    at[output] = at[other]
    assert call(moe, name, at) == moe.MOE_ERR_SHAPE


@pytest.mark.parametrize("name", CALLS)
def test_allowed_otherwise(moe, name):
    """The same call with buffers of their own is not refused: with no GPU here, it gets as far as its launch."""
    at = addresses()
    assert call(moe, name, at) == moe.MOE_ERR_HIP
    if name == "backward_x bf16 pre":
        at["out"] = at["pre"]
        assert call(moe, name, at) == moe.MOE_ERR_HIP
    if name == "combine_backward":
        at["out"] = at["y"]
        assert call(moe, name, at) == moe.MOE_ERR_HIP
