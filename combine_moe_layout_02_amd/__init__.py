"""MI355X-native MoE expert-parallel layout, dispatch and combine.

Thin ctypes binding over libmoe_ep.so (declared in include/moe_ep.h).  The
Python functions carry the C names and only marshal arguments: torch tensors
supply device memory and the current HIP stream, every step of the path runs
in the library's HIP kernels.  ``router``, ``balance_loss``, ``dispatch``,
``expert_ffn`` and ``combine`` are the same calls as autograd functions.  Importing this package fails loudly when the
library has not been built; there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_ep.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(6)
MOE_PAD_NONE, MOE_PAD_MULTIPLE, MOE_PAD_CAPACITY = 0, 1, 2
MOE_F32, MOE_BF16 = 0, 1
MOE_ACT_NONE, MOE_ACT_SWIGLU = 0, 1
MOE_FLAG_BAD_EXPERT, MOE_FLAG_CAPACITY, MOE_FLAG_UNBALANCED = 1, 2, 4

EXPORTED = ("moe_max_recv_rows", "moe_layout_workspace_bytes", "moe_layout", "moe_dispatch",
            "moe_layout_dispatch", "moe_combine", "moe_layout_balanced_workspace_bytes", "moe_layout_balanced",
            "moe_zero_padding", "moe_stream_create_cu_limited", "moe_stream_create_cu_range", "moe_stream_destroy",
            "moe_status_str", "moe_layout_noalloc", "moe_router_workspace_bytes", "moe_router", "moe_balance_loss",
            "moe_router_backward", "moe_quantize_mx4", "moe_dequantize_mx4", "moe_dispatch_mx4", "moe_expert_gemm_mx4",
            "moe_expert_gemm", "moe_expert_gemm_backward_x", "moe_expert_gemm_backward_w", "moe_combine_backward",
            "moe_quantize_i8", "moe_dequantize_i8", "moe_dispatch_i8", "moe_expert_gemm_i8")


class MoeError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {_lib.moe_status_str(status).decode()}")


class moe_layout_desc(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32),
                ("R", ctypes.c_int32), ("pad_mode", ctypes.c_int32), ("pad_rows", ctypes.c_int32)]


class moe_layout_bufs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("tokens_per_expert", "tokens_per_rank", "expert_offset",
                                               "rank_offset", "pos", "src", "status")]


class moe_balance_bufs(ctypes.Structure):
    _fields_ = [("seg_offset", ctypes.c_void_p), ("slot_expert", ctypes.c_void_p)]


class moe_router_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "E", "K", "n_groups", "topk_groups", "renorm", "seq_len")] + \
               [("alpha", ctypes.c_float)]


class moe_router_bufs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_w", "expert_count", "balance_coef", "balance_loss")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                          "g.build()'` (hipcc, gfx950); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    D = ctypes.POINTER(moe_layout_desc)
    B = ctypes.POINTER(moe_layout_bufs)
    L.moe_max_recv_rows.argtypes = [D]
    L.moe_max_recv_rows.restype = ctypes.c_int64
    L.moe_layout_workspace_bytes.argtypes = [D]
    L.moe_layout_workspace_bytes.restype = ctypes.c_size_t
    L.moe_layout.argtypes = [D, P, B, P, ctypes.c_size_t, P]
    L.moe_layout.restype = ctypes.c_int
    L.moe_dispatch.argtypes = [D, B, P, ctypes.c_int32, P, P, ctypes.c_int32, P, P, P, P]
    L.moe_dispatch.restype = ctypes.c_int
    L.moe_layout_dispatch.argtypes = [D, P, B, P, ctypes.c_size_t, P, ctypes.c_int32, P, ctypes.c_int32,
                                      P, P, P, P]
    L.moe_layout_dispatch.restype = ctypes.c_int
    L.moe_combine.argtypes = [D, B, P, ctypes.c_int32, P, P, P, P]
    L.moe_combine.restype = ctypes.c_int
    L.moe_zero_padding.argtypes = [D, B, ctypes.c_int32, ctypes.c_int32, P, P, P]
    L.moe_zero_padding.restype = ctypes.c_int
    L.moe_layout_balanced_workspace_bytes.argtypes = [D, ctypes.c_int32]
    L.moe_layout_balanced_workspace_bytes.restype = ctypes.c_size_t
    L.moe_layout_balanced.argtypes = [D, ctypes.c_int32, P, B, ctypes.POINTER(moe_balance_bufs), P,
                                      ctypes.c_size_t, P]
    L.moe_layout_balanced.restype = ctypes.c_int
    L.moe_stream_create_cu_limited.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p)]
    L.moe_stream_create_cu_limited.restype = ctypes.c_int
    L.moe_stream_create_cu_range.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p)]
    L.moe_stream_create_cu_range.restype = ctypes.c_int
    L.moe_stream_destroy.argtypes = [P]
    L.moe_stream_destroy.restype = ctypes.c_int
    L.moe_status_str.argtypes = [ctypes.c_int32]
    L.moe_status_str.restype = ctypes.c_char_p
    L.moe_layout_noalloc.argtypes = [D, P, B, P]
    L.moe_layout_noalloc.restype = ctypes.c_int
    I, I64, RD, RB = ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(moe_router_desc), ctypes.POINTER(moe_router_bufs)
    L.moe_router_workspace_bytes.argtypes = [RD]
    L.moe_router_workspace_bytes.restype = ctypes.c_size_t
    L.moe_router.argtypes = [RD, P, I, P, RB, P, ctypes.c_size_t, P]
    L.moe_balance_loss.argtypes = [RD, P, I, P, P, RB, P, ctypes.c_size_t, P]
    L.moe_router_backward.argtypes = [RD, P, I, P, P, P, P, P, P, P, P]
    L.moe_quantize_mx4.argtypes = [P, I64, I, P, P, P, P]
    L.moe_dequantize_mx4.argtypes = [P, P, I64, I, P, P, P]
    L.moe_dispatch_mx4.argtypes = [D, B, P, I, P, P, P, P, P]
    L.moe_expert_gemm_mx4.argtypes = [D, B, ctypes.POINTER(moe_balance_bufs), I, P, P, I, P, P, I, I, P, P]
    BB = ctypes.POINTER(moe_balance_bufs)
    L.moe_expert_gemm.argtypes = [D, B, BB, I, P, I, P, I, I, P, I, P, P]
    L.moe_expert_gemm_backward_x.argtypes = [D, B, BB, I, P, I, P, I, P, I, P, P]
    L.moe_expert_gemm_backward_w.argtypes = [D, B, BB, I, P, I, P, I, I, P, P]
    L.moe_combine_backward.argtypes = [D, B, P, I, P, P, P, P, P]
    L.moe_quantize_i8.argtypes = [P, I64, I, P, P, P, P]
    L.moe_dequantize_i8.argtypes = [P, P, I64, I, P, P, P]
    L.moe_dispatch_i8.argtypes = [D, B, P, I, P, P, P, P, P]
    L.moe_expert_gemm_i8.argtypes = [D, B, BB, I, P, P, I, P, P, I, I, P, P]
    for f in (L.moe_router, L.moe_balance_loss, L.moe_router_backward, L.moe_quantize_mx4, L.moe_dequantize_mx4,
              L.moe_dispatch_mx4, L.moe_expert_gemm_mx4, L.moe_expert_gemm, L.moe_expert_gemm_backward_x,
              L.moe_expert_gemm_backward_w, L.moe_combine_backward, L.moe_quantize_i8, L.moe_dequantize_i8, L.moe_dispatch_i8,
              L.moe_expert_gemm_i8):
        f.restype = ctypes.c_int
    return L


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


# ---------------------------------------------------------------------------
# descriptors
# ---------------------------------------------------------------------------

class _Descriptor:
    """A frozen descriptor; its C struct is built once and is no part of its state."""

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in ("_ref", "_rows")}


@dataclasses.dataclass(frozen=True)
class LayoutDesc(_Descriptor):
    S: int
    K: int
    E: int
    R: int
    pad_mode: int = MOE_PAD_NONE
    pad_rows: int = 0

    def c(self) -> moe_layout_desc:
        return moe_layout_desc(self.S, self.K, self.E, self.R, self.pad_mode, self.pad_rows)


def _made_once(desc):
    """A reference to the descriptor's C struct, which its fields, frozen, cannot outlive."""
    ref = desc.__dict__.get("_ref")
    if ref is None:
        ref = ctypes.byref(desc.c())
        desc.__dict__["_ref"] = ref
    return ref


@dataclasses.dataclass
class Layout:
    """Device tensors of one batch's layout (outputs of moe_layout)."""
    tokens_per_expert: torch.Tensor   # [E] int32
    tokens_per_rank: torch.Tensor     # [R] int32
    expert_offset: torch.Tensor       # [E+1] int32
    rank_offset: torch.Tensor         # [R+1] int32
    pos: torch.Tensor                 # [S,K] int32
    src: torch.Tensor                 # [max_recv] int32
    status: torch.Tensor              # [1] int32
    workspace: Optional[torch.Tensor] = None

    def c(self) -> moe_layout_bufs:
        return moe_layout_bufs(*(_ptr(t) for t in (
            self.tokens_per_expert, self.tokens_per_rank, self.expert_offset, self.rank_offset,
            self.pos, self.src, self.status)))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()   # argtypes make it a void*


# torch's raw current-stream query: measured ~0.1 us per call against ~2 us
# for torch.cuda.current_stream(), which builds a Stream object.  A
# decode-sized call costs only a few microseconds on the GPU, so the host side
# of every call counts.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device) -> int:
    """Raw hipStream_t of `stream`, or of the current stream of `device`."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_current_stream is not None:
        return _raw_current_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _check(t: Optional[torch.Tensor], name: str, dtype, shape=None, device=None):
    if t is None:
        return
    # the usual case in one line
    if t.is_cuda and t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == shape) and \
            (device is None or t.device == device):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


# ---------------------------------------------------------------------------
# the C calls
# ---------------------------------------------------------------------------

def moe_max_recv_rows(desc: LayoutDesc) -> int:
    d = desc.c()
    return int(_lib.moe_max_recv_rows(ctypes.byref(d)))


def moe_layout_workspace_bytes(desc: LayoutDesc) -> int:
    d = desc.c()
    return int(_lib.moe_layout_workspace_bytes(ctypes.byref(d)))


def moe_status_str(status: int) -> str:
    return _lib.moe_status_str(int(status)).decode()


class PingPongBuffer:
    """Two Buffers of one shape used in turn: call i works in buffer i % 2, so
    the results of call i stay valid while call i + 1 runs -- the double
    buffer of DeepEP's low-latency kernels (DeepEP analysis, code notes).
    ``next()`` returns the buffer for the next call; arguments as Buffer."""

    def __init__(self, *args, **kwargs):
        self.buffers = (Buffer(*args, **kwargs), Buffer(*args, **kwargs))
        self._i = 0

    def next(self) -> "Buffer":
        b = self.buffers[self._i]
        self._i ^= 1
        return b


class CULimitedStream:
    """A HIP stream whose kernels run only on CUs [first_cu, first_cu +
    num_cus) (moe_stream_create_cu_range; first_cu = 0 is
    moe_stream_create_cu_limited), usable as a torch stream."""

    def __init__(self, num_cus: int, device="cuda", first_cu: int = 0):
        handle = ctypes.c_void_p()
        rc = _lib.moe_stream_create_cu_range(int(first_cu), int(num_cus), ctypes.byref(handle))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_stream_create_cu_range")
        self.num_cus = num_cus
        self.handle = handle.value
        self.stream = torch.cuda.ExternalStream(self.handle, device=torch.device(device))

    def close(self):
        if self.handle:
            torch.cuda.synchronize()
            _lib.moe_stream_destroy(ctypes.c_void_p(self.handle))
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def alloc_layout(desc: LayoutDesc, device) -> Layout:
    """Device buffers for moe_layout's outputs and its workspace (torch memory)."""
    rows = moe_max_recv_rows(desc)
    if rows < 0:
        raise MoeError(MOE_ERR_SHAPE, "alloc_layout")
    i32 = dict(dtype=torch.int32, device=device)
    ws = moe_layout_workspace_bytes(desc)
    return Layout(
        tokens_per_expert=torch.empty(desc.E, **i32), tokens_per_rank=torch.empty(desc.R, **i32),
        expert_offset=torch.empty(desc.E + 1, **i32), rank_offset=torch.empty(desc.R + 1, **i32),
        pos=torch.empty((desc.S, desc.K), **i32), src=torch.empty(rows, **i32),
        status=torch.empty(1, **i32),
        workspace=torch.empty(ws, dtype=torch.uint8, device=device) if ws else None)


def moe_layout(desc: LayoutDesc, topk_idx: torch.Tensor, layout: Optional[Layout] = None,
               stream=None) -> Layout:
    dev = topk_idx.device
    _check(topk_idx, "topk_idx", torch.int32, (desc.S, desc.K))
    if layout is None:
        layout = alloc_layout(desc, dev)
    ws = layout.workspace
    d, b = desc.c(), layout.c()
    rc = _lib.moe_layout(ctypes.byref(d), _ptr(topk_idx), ctypes.byref(b), _ptr(ws),
                         0 if ws is None else ws.numel(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_layout")
    return layout


def moe_layout_noalloc(desc: LayoutDesc, topk_idx: torch.Tensor, layout: Layout, stream=None) -> Layout:
    """moe_layout with the library's own per-GPU scratch instead of a
    workspace: the C call allocates nothing (the output tensors of `layout`
    are the caller's; its workspace, if any, is not used)."""
    dev = topk_idx.device
    _check(topk_idx, "topk_idx", torch.int32, (desc.S, desc.K))
    d, b = desc.c(), layout.c()
    rc = _lib.moe_layout_noalloc(ctypes.byref(d), _ptr(topk_idx), ctypes.byref(b), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_layout_noalloc")
    return layout


def moe_dispatch(desc: LayoutDesc, layout: Layout, hidden: torch.Tensor, topk_idx=None, topk_w=None,
                 fp8: bool = False, recv=None, recv_scales=None, recv_w=None, stream=None):
    """Returns (recv, recv_scales or None, recv_w or None).  recv is bf16
    [max_recv,H], or uint8 E4M3FN codes [max_recv,H] when fp8."""
    dev = hidden.device
    S, H = hidden.shape
    rows = moe_max_recv_rows(desc)
    _check(hidden, "hidden", torch.bfloat16, (desc.S, H))
    _check(topk_w, "topk_w", torch.float32, (desc.S, desc.K))
    if recv is None:
        recv = torch.empty((rows, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    if fp8 and recv_scales is None:
        recv_scales = torch.empty((rows, H // 128), dtype=torch.float32, device=dev)
    if recv_w is None and topk_w is not None:
        recv_w = torch.empty(rows, dtype=torch.float32, device=dev)
    _check(recv, "recv", (torch.uint8, torch.float8_e4m3fn) if fp8 else torch.bfloat16)
    if recv.shape[0] < rows or recv.shape[-1] != H:
        raise ValueError("recv must hold moe_max_recv_rows rows of H channels")
    if fp8:
        _check(recv_scales, "recv_scales", torch.float32)
        if recv_scales.shape[0] < rows or recv_scales.shape[-1] != H // 128:
            raise ValueError("recv_scales must be [max_recv, H/128]")
    _check(recv_w, "recv_w", torch.float32)
    d, b = desc.c(), layout.c()
    rc = _lib.moe_dispatch(ctypes.byref(d), ctypes.byref(b), _ptr(hidden), H, _ptr(topk_idx), _ptr(topk_w),
                           1 if fp8 else 0, _ptr(recv), _ptr(recv_scales if fp8 else None), _ptr(recv_w),
                           _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_dispatch")
    return recv, (recv_scales if fp8 else None), recv_w


def moe_layout_balanced_workspace_bytes(desc: LayoutDesc, slots_per_rank: int) -> int:
    d = desc.c()
    return int(_lib.moe_layout_balanced_workspace_bytes(ctypes.byref(d), int(slots_per_rank)))


@dataclasses.dataclass
class Balance:
    """Device outputs of moe_layout_balanced beyond the layout."""
    seg_offset: torch.Tensor    # [R*(E/R+B)+1] int32
    slot_expert: torch.Tensor   # [R*B] int32
    workspace: Optional[torch.Tensor]   # scratch (uint8), None when none is needed

    def c(self) -> moe_balance_bufs:
        return moe_balance_bufs(self.seg_offset.data_ptr(), self.slot_expert.data_ptr())


def alloc_balance(desc: LayoutDesc, slots_per_rank: int, device) -> Balance:
    epr = desc.E // desc.R
    ws = moe_layout_balanced_workspace_bytes(desc, slots_per_rank)
    return Balance(torch.empty(desc.R * (epr + slots_per_rank) + 1, dtype=torch.int32, device=device),
                   torch.empty(max(desc.R * slots_per_rank, 1), dtype=torch.int32, device=device),
                   torch.empty(ws, dtype=torch.uint8, device=device) if ws else None)


def moe_layout_balanced(desc: LayoutDesc, slots_per_rank: int, topk_idx: torch.Tensor,
                        layout: Optional[Layout] = None, balance: Optional[Balance] = None, stream=None):
    """Balanced layout (equal rows per rank through redundant-expert slots).
    Returns (layout, balance)."""
    dev = topk_idx.device
    _check(topk_idx, "topk_idx", torch.int32, (desc.S, desc.K))
    if layout is None:
        layout = alloc_layout(desc, dev)
    if balance is None:
        balance = alloc_balance(desc, slots_per_rank, dev)
    d, b, bb = desc.c(), layout.c(), balance.c()
    rc = _lib.moe_layout_balanced(ctypes.byref(d), int(slots_per_rank), _ptr(topk_idx), ctypes.byref(b),
                                  ctypes.byref(bb), _ptr(balance.workspace),
                                  0 if balance.workspace is None else balance.workspace.numel(),
                                  _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_layout_balanced")
    return layout, balance


def moe_layout_dispatch(desc: LayoutDesc, topk_idx: torch.Tensor, hidden: torch.Tensor, topk_w=None,
                        fp8: bool = False, layout: Optional[Layout] = None, recv=None, recv_scales=None,
                        recv_w=None, stream=None):
    """moe_layout + moe_dispatch in one call (one launch for S*K <= 4096 and S <= 512).
    Returns (layout, recv, recv_scales or None, recv_w or None)."""
    dev = hidden.device
    H = hidden.shape[1]
    rows = moe_max_recv_rows(desc)
    _check(topk_idx, "topk_idx", torch.int32, (desc.S, desc.K))
    _check(hidden, "hidden", torch.bfloat16, (desc.S, H))
    _check(topk_w, "topk_w", torch.float32, (desc.S, desc.K))
    if layout is None:
        layout = alloc_layout(desc, dev)
    if recv is None:
        recv = torch.empty((rows, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    if fp8 and recv_scales is None:
        recv_scales = torch.empty((rows, H // 128), dtype=torch.float32, device=dev)
    if recv_w is None and topk_w is not None:
        recv_w = torch.empty(rows, dtype=torch.float32, device=dev)
    _check(recv, "recv", (torch.uint8, torch.float8_e4m3fn) if fp8 else torch.bfloat16)
    if recv.shape[0] < rows or recv.shape[-1] != H:
        raise ValueError("recv must hold moe_max_recv_rows rows of H channels")
    if fp8:
        _check(recv_scales, "recv_scales", torch.float32)
        if recv_scales.shape[0] < rows or recv_scales.shape[-1] != H // 128:
            raise ValueError("recv_scales must be [max_recv, H/128]")
    _check(recv_w, "recv_w", torch.float32)
    ws = layout.workspace
    d, b = desc.c(), layout.c()
    rc = _lib.moe_layout_dispatch(ctypes.byref(d), _ptr(topk_idx), ctypes.byref(b), _ptr(ws),
                                  0 if ws is None else ws.numel(), _ptr(hidden), H, _ptr(topk_w),
                                  1 if fp8 else 0, _ptr(recv), _ptr(recv_scales if fp8 else None), _ptr(recv_w),
                                  _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_layout_dispatch")
    return layout, recv, (recv_scales if fp8 else None), recv_w


def moe_combine(desc: LayoutDesc, layout: Layout, expert_out: torch.Tensor, w=None, shared_out=None,
                out=None, stream=None) -> torch.Tensor:
    dev = expert_out.device
    H = expert_out.shape[-1]
    _check(expert_out, "expert_out", torch.bfloat16)
    if expert_out.shape[0] < moe_max_recv_rows(desc):
        raise ValueError("expert_out must hold moe_max_recv_rows rows")
    _check(w, "w", torch.float32, (desc.S, desc.K))
    _check(shared_out, "shared_out", torch.bfloat16, (desc.S, H))
    if out is None:
        out = torch.empty((desc.S, H), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (desc.S, H))
    d, b = desc.c(), layout.c()
    rc = _lib.moe_combine(ctypes.byref(d), ctypes.byref(b), _ptr(expert_out), H, _ptr(w), _ptr(shared_out),
                          _ptr(out), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_combine")
    return out


def moe_zero_padding(desc: LayoutDesc, layout: Layout, recv: torch.Tensor, recv_scales=None, stream=None):
    """Zero every receive row that no entry maps to (and its FP8 scales).
    FP8 when recv holds E4M3 codes (uint8 or float8_e4m3fn), bf16 otherwise."""
    fp8 = recv.dtype in (torch.uint8, torch.float8_e4m3fn)
    H = recv.shape[-1]
    _check(recv, "recv", (torch.uint8, torch.float8_e4m3fn) if fp8 else torch.bfloat16)
    if recv.shape[0] < moe_max_recv_rows(desc):
        raise ValueError("recv must hold moe_max_recv_rows rows")
    if fp8:
        _check(recv_scales, "recv_scales", torch.float32, (recv.shape[0], H // 128))
    d, b = desc.c(), layout.c()
    rc = _lib.moe_zero_padding(ctypes.byref(d), ctypes.byref(b), H, 1 if fp8 else 0, _ptr(recv),
                               _ptr(recv_scales) if fp8 else None, _stream(stream, recv.device))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_zero_padding")


# ---------------------------------------------------------------------------
# Router and balance loss
# ---------------------------------------------------------------------------

_nothing = contextlib.nullcontext()
_raw_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _alloc_on(stream):
    """Where a call's own outputs come from: memory of the stream that will
    write them, so that the allocator hands it out again in that stream's order."""
    return _nothing if stream is None else torch.cuda.stream(stream)


def _on_device(device):
    """The C calls launch on the current device: make it the tensors' own."""
    return _nothing if device.index == _raw_current_device() else torch.cuda.device(device)


@dataclasses.dataclass(frozen=True)
class RouterDesc(_Descriptor):
    """A router's shape and rule (fields as moe_router_desc; n_groups = 1 and
    seq_len = 0: no groups, one sequence)."""
    S: int
    E: int
    K: int
    n_groups: int = 1
    topk_groups: Optional[int] = None   # None: every group
    renorm: bool = True
    seq_len: int = 0
    alpha: float = 1.0

    @property
    def sequences(self) -> int:
        return self.S // self.seq_len if self.seq_len else 1

    def c(self) -> moe_router_desc:
        return moe_router_desc(self.S, self.E, self.K, self.n_groups,
                               self.n_groups if self.topk_groups is None else self.topk_groups, 1 if self.renorm else 0,
                               self.seq_len, self.alpha)


@dataclasses.dataclass
class Router:
    """Device tensors of one batch's routing.  The last four are None without the loss,
    the first two without a routing of moe_router's own."""
    topk_idx: Optional[torch.Tensor]       # [S,K] int32
    topk_w: Optional[torch.Tensor]         # [S,K] fp32
    expert_count: Optional[torch.Tensor]   # [G,E] int32
    balance_coef: Optional[torch.Tensor]   # [G,E] fp32
    balance_loss: Optional[torch.Tensor]   # [1] fp32
    workspace: Optional[torch.Tensor] = None

    def c(self) -> moe_router_bufs:
        return moe_router_bufs(_ptr(self.topk_idx), _ptr(self.topk_w), _ptr(self.expert_count), _ptr(self.balance_coef),
                               _ptr(self.balance_loss))


def moe_router_workspace_bytes(desc: RouterDesc) -> int:
    return int(_lib.moe_router_workspace_bytes(_made_once(desc)))


def alloc_router(desc: RouterDesc, device, picks: bool = True, loss: bool = True) -> Router:
    """Device buffers for moe_router's outputs (``picks``: the routing, ``loss``:
    counts, coefficients, the loss and its workspace)."""
    empty, i32, f32 = torch.empty, torch.int32, torch.float32
    idx = w = count = coef = value = ws = None
    if picks:
        idx = empty(desc.S, desc.K, dtype=i32, device=device)   # sizes one by one: a tuple takes longer to parse
        w = empty(desc.S, desc.K, dtype=f32, device=device)
    if loss:
        need = moe_router_workspace_bytes(desc)
        if need == 0:
            raise MoeError(MOE_ERR_SHAPE, "alloc_router")
        G, E = desc.sequences, desc.E
        count, coef = empty(G, E, dtype=i32, device=device), empty(G, E, dtype=f32, device=device)
        value, ws = empty(1, dtype=f32, device=device), empty(need, dtype=torch.uint8, device=device)
    return Router(idx, w, count, coef, value, ws)


def _logits(desc: RouterDesc, logits: torch.Tensor, token_mask) -> int:
    """Checks a router call's inputs; the C type of the logits."""
    _check(logits, "logits", (torch.float32, torch.bfloat16), (desc.S, desc.E))
    if token_mask is not None:
        _check(token_mask, "token_mask", (torch.bool, torch.uint8), (desc.S,), logits.device)
    return MOE_BF16 if logits.dtype is torch.bfloat16 else MOE_F32


def _check_picks(desc: RouterDesc, r: Router, device):
    if r.topk_idx is None or r.topk_w is None:
        raise ValueError("router has no buffers for the routing")
    _check(r.topk_idx, "topk_idx", torch.int32, (desc.S, desc.K), device)
    _check(r.topk_w, "topk_w", torch.float32, (desc.S, desc.K), device)


def _check_loss(desc: RouterDesc, r: Router, device):
    if r.balance_loss is None or r.expert_count is None or r.balance_coef is None:
        raise ValueError("router has no buffers for the loss")
    cells = (desc.sequences, desc.E)
    _check(r.expert_count, "expert_count", torch.int32, cells, device)
    _check(r.balance_coef, "balance_coef", torch.float32, cells, device)
    _check(r.balance_loss, "balance_loss", torch.float32, (1,), device)
    _check(r.workspace, "workspace", torch.uint8, None, device)


def moe_router(desc: RouterDesc, logits: torch.Tensor, token_mask=None, loss: bool = True,
               router: Optional[Router] = None, stream=None) -> Router:
    """Top-k routing of logits [S,E] (fp32 or bf16), with the balance loss and
    the counts unless ``loss`` is false (serving: one launch, no workspace).
    token_mask [S] (bool or uint8): false where a token does not count.
    Entries without a pick are -1 with weight 0."""
    dev = logits.device
    kind = _logits(desc, logits, token_mask)
    if router is None:
        with _alloc_on(stream):
            router = alloc_router(desc, dev, loss=loss)
    else:
        _check_picks(desc, router, dev)
        if loss:
            _check_loss(desc, router, dev)
    ws = router.workspace if loss else None
    if loss:
        b = router.c()
    else:
        b = moe_router_bufs(router.topk_idx.data_ptr(), router.topk_w.data_ptr())
    with _on_device(dev):
        rc = _lib.moe_router(_made_once(desc), logits.data_ptr(), kind, _ptr(token_mask), ctypes.byref(b), _ptr(ws),
                             0 if ws is None else ws.numel(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_router")
    return router


def moe_balance_loss(desc: RouterDesc, logits: torch.Tensor, topk_idx: torch.Tensor, token_mask=None,
                     router: Optional[Router] = None, stream=None) -> Router:
    """Balance loss and per-expert counts of the routing topk_idx [S,K] int32
    that the caller made.  The result holds expert_count, balance_coef and
    balance_loss; moe_router_backward takes it without d_topk_w."""
    dev = logits.device
    kind = _logits(desc, logits, token_mask)
    _check(topk_idx, "topk_idx", torch.int32, (desc.S, desc.K), dev)
    if router is None:
        with _alloc_on(stream):
            router = alloc_router(desc, dev, picks=False)
    else:
        _check_loss(desc, router, dev)
    ws = router.workspace
    with _on_device(dev):
        rc = _lib.moe_balance_loss(_made_once(desc), logits.data_ptr(), kind, topk_idx.data_ptr(), _ptr(token_mask),
                                   ctypes.byref(router.c()), _ptr(ws), 0 if ws is None else ws.numel(),
                                   _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_balance_loss")
    return router


def moe_router_backward(desc: RouterDesc, logits: torch.Tensor, router: Router, d_topk_w=None, d_loss=None,
                        token_mask=None, d_logits=None, stream=None) -> torch.Tensor:
    """d logits, from the gradients of the route weights (d_topk_w [S,K] fp32)
    and of the balance loss (d_loss, one fp32 value), at least one of them.
    desc, logits, router and token_mask as moe_router had and returned them."""
    dev = logits.device
    kind = _logits(desc, logits, token_mask)
    idx = w = coef = None
    if d_topk_w is not None:
        _check_picks(desc, router, dev)
        _check(d_topk_w, "d_topk_w", torch.float32, (desc.S, desc.K), dev)
        idx, w = router.topk_idx, router.topk_w
    if d_loss is not None:
        coef = router.balance_coef
        if coef is None:
            raise ValueError("router has no buffers for the loss")
        _check(coef, "balance_coef", torch.float32, (desc.sequences, desc.E), dev)
        _check(d_loss, "d_loss", torch.float32, None, dev)
        if d_loss.numel() != 1:
            raise ValueError(f"d_loss: {d_loss.numel()} values, expected 1")
    if d_logits is None:
        with _alloc_on(stream):
            d_logits = torch.empty_like(logits)
    else:
        _check(d_logits, "d_logits", logits.dtype, (desc.S, desc.E), dev)
    with _on_device(dev):
        rc = _lib.moe_router_backward(_made_once(desc), logits.data_ptr(), kind, _ptr(token_mask), _ptr(idx), _ptr(w),
                                      _ptr(coef), _ptr(d_topk_w), _ptr(d_loss), d_logits.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_router_backward")
    return d_logits


# What an autograd function calls forward and backward: a graph can hold these.
_CAPTURABLE = {
    "router": (("moe_router",), ("moe_router_backward",)),
    "balance_loss": (("moe_balance_loss",), ("moe_router_backward",)),
    "dispatch": (("moe_dispatch", "moe_zero_padding"), ("moe_combine",)),
    "expert_ffn": (("moe_expert_gemm", "moe_zero_padding"),
                   ("moe_expert_gemm_backward_x", "moe_expert_gemm_backward_w", "moe_zero_padding")),
    "combine": (("moe_combine",), ("moe_combine_backward", "moe_zero_padding")),
}


def _no_capture(name: str, backward: bool = False):
    # autograd joins the streams of the leaves that live outside the capture
    if torch.cuda.is_current_stream_capturing():
        calls = _CAPTURABLE[name]
        calls = calls[1] if backward else tuple(dict.fromkeys(calls[0] + calls[1]))
        what = f"the backward pass of {name}" if backward else name
        raise RuntimeError(f"{what} cannot be captured into a graph: capture {', '.join(calls)} instead")


class _RouterFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, desc, token_mask, topk_idx):
        ctx.set_materialize_grads(False)
        given = topk_idx is not None
        r = moe_balance_loss(desc, logits, topk_idx, token_mask) if given else moe_router(desc, logits, token_mask)
        loss = r.balance_loss.view(())
        ctx.desc, ctx.given = desc, given
        ctx.save_for_backward(logits, token_mask, r.topk_idx, r.topk_w, r.balance_coef)
        ctx.mark_non_differentiable(*(t for t in (r.topk_idx, r.expert_count) if t is not None))
        return loss, r.expert_count, r.topk_idx, r.topk_w

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_loss, _count, _idx, d_w):
        if d_loss is None and d_w is None:
            return None, None, None, None
        logits, token_mask, idx, w, coef = ctx.saved_tensors
        _no_capture("balance_loss" if ctx.given else "router", backward=True)
        d = moe_router_backward(ctx.desc, logits, Router(idx, w, None, coef, None), None if d_w is None else d_w.contiguous(),
                                None if d_loss is None else d_loss.contiguous(), token_mask)
        return d, None, None, None


def router(desc: RouterDesc, logits: torch.Tensor, token_mask=None):
    """moe_router as an autograd function of the logits: (topk_idx, topk_w,
    balance_loss, expert_count), of which topk_w and balance_loss (a scalar)
    carry gradients.  Not capturable; moe_router and moe_router_backward are."""
    _no_capture("router")
    loss, count, idx, w = _RouterFunction.apply(logits, desc, token_mask, None)
    return idx, w, loss, count


def balance_loss(desc: RouterDesc, logits: torch.Tensor, topk_idx: torch.Tensor, token_mask=None):
    """moe_balance_loss as an autograd function of the logits: (balance_loss,
    expert_count).  Not capturable, as router."""
    _no_capture("balance_loss")
    return _RouterFunction.apply(logits, desc, token_mask, topk_idx)[:2]


# ---------------------------------------------------------------------------
# MXFP4 rows and the experts' products
# ---------------------------------------------------------------------------

def _check_mx4(codes, scales, names, rows, H, device):
    """Packed rows [.., H/2] and their scales [.., H/32], at least `rows` of them."""
    for t, name, width in ((codes, names[0], H // 2), (scales, names[1], H // 32)):
        if t is None:
            raise ValueError(f"{name} is missing")
        _check(t, name, torch.uint8, None, device)
        shape = t.shape
        if len(shape) != 2 or shape[1] != width or shape[0] < rows:
            raise ValueError(f"{name}: shape {tuple(shape)}, expected [at least {rows}, {width}]")


def _mx4_width(H: int, what: str):
    if H < 128 or H % 128:
        raise MoeError(MOE_ERR_SHAPE, what)


def _check_src(layout: Optional[Layout], rows: int, device):
    if layout is None:
        return None
    _check(layout.src, "layout.src", torch.int32, None, device)
    if layout.src.numel() < rows:
        raise ValueError(f"layout.src: {layout.src.numel()} rows, expected at least {rows}")
    return layout.src


def moe_quantize_mx4(x: torch.Tensor, codes=None, scales=None, layout: Optional[Layout] = None, stream=None):
    """bf16 rows [rows,H] -> MXFP4: (codes [rows,H/2] uint8, scales [rows,H/32]
    uint8).  x may have leading dimensions (expert weights [E,N,H]); so have the
    results then.  With ``layout`` only the rows that hold an entry are converted."""
    dev, H = x.device, x.shape[-1]
    _check(x, "x", torch.bfloat16)
    _mx4_width(H, "moe_quantize_mx4")
    rows = x.numel() // H
    src = _check_src(layout, rows, dev)
    lead = x.shape[:-1]
    with _alloc_on(stream):
        if codes is None:
            codes = torch.empty(*lead, H // 2, dtype=torch.uint8, device=dev)
        else:
            _check(codes, "codes", torch.uint8, (*lead, H // 2), dev)
        if scales is None:
            scales = torch.empty(*lead, H // 32, dtype=torch.uint8, device=dev)
        else:
            _check(scales, "scales", torch.uint8, (*lead, H // 32), dev)
    with _on_device(dev):
        rc = _lib.moe_quantize_mx4(x.data_ptr(), rows, H, _ptr(src), codes.data_ptr(), scales.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_quantize_mx4")
    return codes, scales


def moe_dequantize_mx4(codes: torch.Tensor, scales: torch.Tensor, out=None, layout: Optional[Layout] = None, stream=None):
    """MXFP4 rows -> bf16 [.., H].  With ``layout`` only the rows that hold an
    entry are converted; the others keep what they held."""
    dev, H = codes.device, codes.shape[-1] * 2
    _check(codes, "codes", torch.uint8)
    _mx4_width(H, "moe_dequantize_mx4")
    _check(scales, "scales", torch.uint8, (*codes.shape[:-1], H // 32), dev)
    rows = codes.numel() // (H // 2)
    src = _check_src(layout, rows, dev)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(*codes.shape[:-1], H, dtype=torch.bfloat16, device=dev)
    else:
        _check(out, "out", torch.bfloat16, (*codes.shape[:-1], H), dev)
    with _on_device(dev):
        rc = _lib.moe_dequantize_mx4(codes.data_ptr(), scales.data_ptr(), rows, H, _ptr(src), out.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_dequantize_mx4")
    return out


def moe_dispatch_mx4(desc: LayoutDesc, layout: Layout, hidden: torch.Tensor, topk_w=None, recv=None, recv_scales=None,
                     recv_w=None, stream=None):
    """moe_dispatch in MXFP4.  Returns (recv [max_recv,H/2] uint8, recv_scales
    [max_recv,H/32] uint8, recv_w or None)."""
    dev, H, rows = hidden.device, hidden.shape[-1], int(_lib.moe_max_recv_rows(_made_once(desc)))
    _check(hidden, "hidden", torch.bfloat16, (desc.S, H))
    _check(topk_w, "topk_w", torch.float32, (desc.S, desc.K), dev)
    _mx4_width(H, "moe_dispatch_mx4")
    if rows < 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_dispatch_mx4")
    _check(layout.pos, "layout.pos", torch.int32, (desc.S, desc.K), dev)
    with _alloc_on(stream):
        if recv is None:
            recv = torch.empty(rows, H // 2, dtype=torch.uint8, device=dev)
        if recv_scales is None:
            recv_scales = torch.empty(rows, H // 32, dtype=torch.uint8, device=dev)
        if recv_w is None and topk_w is not None:
            recv_w = torch.empty(rows, dtype=torch.float32, device=dev)
    _check_mx4(recv, recv_scales, ("recv", "recv_scales"), rows, H, dev)
    _check(recv_w, "recv_w", torch.float32, None, dev)
    if recv_w is not None and recv_w.numel() < rows:
        raise ValueError(f"recv_w: {recv_w.numel()} rows, expected at least {rows}")
    b = moe_layout_bufs(pos=layout.pos.data_ptr())
    with _on_device(dev):
        rc = _lib.moe_dispatch_mx4(_made_once(desc), ctypes.byref(b), _ptr(hidden), H, _ptr(topk_w), _ptr(recv),
                                   _ptr(recv_scales), _ptr(recv_w), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_dispatch_mx4")
    return recv, recv_scales, recv_w


def moe_expert_gemm_mx4(desc: LayoutDesc, layout: Layout, x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor,
                        w_scales: torch.Tensor, act: int = MOE_ACT_NONE, out=None, balance: Optional[Balance] = None,
                        slots_per_rank: int = 0, stream=None) -> torch.Tensor:
    """Every expert's rows times its weights: out [max_recv,N] bf16.

    x [max_recv,H/2] and x_scales [max_recv,H/32]: the receive buffer in MXFP4;
    w [E,M,H/2] and w_scales [E,M,H/32]: the experts' weights, M = N, or 2N with
    MOE_ACT_SWIGLU (N gate rows, then N up rows).  ``balance`` and
    ``slots_per_rank`` for a layout of moe_layout_balanced.  Rows that hold no
    entry are neither read nor written."""
    dev, H, rows = x.device, x.shape[-1] * 2, int(_lib.moe_max_recv_rows(_made_once(desc)))
    _mx4_width(H, "moe_expert_gemm_mx4")
    if rows < 0 or act not in (MOE_ACT_NONE, MOE_ACT_SWIGLU):
        raise MoeError(MOE_ERR_SHAPE, "moe_expert_gemm_mx4")
    _check_mx4(x, x_scales, ("x", "x_scales"), rows, H, dev)
    if w.dim() != 3 or (act == MOE_ACT_SWIGLU and w.shape[1] % 2):
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [E, N or 2N, H/2]")
    M = w.shape[1]
    N = M // 2 if act == MOE_ACT_SWIGLU else M
    _check(w, "w", torch.uint8, (desc.E, M, H // 2), dev)
    _check(w_scales, "w_scales", torch.uint8, (desc.E, M, H // 32), dev)
    _check(layout.tokens_per_expert, "layout.tokens_per_expert", torch.int32, (desc.E,), dev)
    _check(layout.expert_offset, "layout.expert_offset", torch.int32, (desc.E + 1,), dev)
    if balance is not None:
        _check(balance.seg_offset, "balance.seg_offset", torch.int32, (desc.E + desc.R * slots_per_rank + 1,), dev)
        _check(balance.slot_expert, "balance.slot_expert", torch.int32, (max(desc.R * slots_per_rank, 1),), dev)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(rows, N, dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, None, dev)
    shape = out.shape
    if len(shape) != 2 or shape[1] != N or shape[0] < rows:
        raise ValueError(f"out: shape {tuple(shape)}, expected [at least {rows}, {N}]")
    b = moe_layout_bufs(layout.tokens_per_expert.data_ptr(), None, layout.expert_offset.data_ptr())
    bal = None if balance is None else ctypes.byref(balance.c())
    with _on_device(dev):
        rc = _lib.moe_expert_gemm_mx4(_made_once(desc), ctypes.byref(b), bal, slots_per_rank, x.data_ptr(), x_scales.data_ptr(),
                                      H, w.data_ptr(), w_scales.data_ptr(), N, act, out.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_expert_gemm_mx4")
    return out


# ---------------------------------------------------------------------------
# The experts in bf16, with their gradients, and in 8-bit integers
# ---------------------------------------------------------------------------

def _check_segments(desc: LayoutDesc, layout: Layout, balance: Optional[Balance], slots_per_rank: int, device):
    """The layout's arrays that a product reads, as C structs (layout, balance or None)."""
    count, offset, E = layout.tokens_per_expert, layout.expert_offset, desc.E
    _check(count, "layout.tokens_per_expert", torch.int32, (E,), device)
    _check(offset, "layout.expert_offset", torch.int32, (E + 1,), device)
    b = moe_layout_bufs(count.data_ptr(), None, offset.data_ptr())
    if balance is None:
        return ctypes.byref(b), None
    _check(balance.seg_offset, "balance.seg_offset", torch.int32, (desc.E + desc.R * slots_per_rank + 1,), device)
    _check(balance.slot_expert, "balance.slot_expert", torch.int32, (max(desc.R * slots_per_rank, 1),), device)
    return ctypes.byref(b), ctypes.byref(balance.c())


def _product_rows(desc: LayoutDesc, what: str) -> int:
    """moe_max_recv_rows, worked out once per descriptor."""
    rows = desc.__dict__.get("_rows")
    if rows is None:
        rows = int(_lib.moe_max_recv_rows(_made_once(desc)))
        if rows < 0:
            raise MoeError(MOE_ERR_SHAPE, what)
        desc.__dict__["_rows"] = rows
    return rows


def _check_rows(t: torch.Tensor, name: str, dtype, rows: int, width: int, device):
    """A row buffer [at least `rows`, width] of `dtype` (or of one of them)."""
    shape = t.shape
    # the usual case in one line
    if t.is_cuda and t.dtype is dtype and t.is_contiguous() and len(shape) == 2 and shape[1] == width and shape[0] >= rows and \
            t.device == device:
        return
    _check(t, name, dtype, None, device)
    if len(shape) != 2 or shape[1] != width or shape[0] < rows:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [at least {rows}, {width}]")


def _gemm_shape(desc: LayoutDesc, x: torch.Tensor, w: torch.Tensor, act: int, dtype, what: str):
    """(H, N, M) of a product of rows x [.., H] with weights w [E,M,H]."""
    if act not in (MOE_ACT_NONE, MOE_ACT_SWIGLU):
        raise MoeError(MOE_ERR_SHAPE, what)
    H = x.shape[-1]
    if w.dim() != 3 or (act == MOE_ACT_SWIGLU and w.shape[1] % 2):
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [E, N or 2N, H]")
    M = w.shape[1]
    _check(w, "w", dtype, (desc.E, M, H), x.device)
    return H, (M // 2 if act == MOE_ACT_SWIGLU else M), M


_PRE_TYPES = (torch.float32, torch.bfloat16)


def _check_pre(pre: torch.Tensor, rows: int, width: int, device):
    _check_rows(pre, "pre", pre.dtype if pre.dtype in _PRE_TYPES else _PRE_TYPES, rows, width, device)


def _pre_type(pre) -> int:
    return MOE_BF16 if pre is not None and pre.dtype is torch.bfloat16 else MOE_F32


def moe_expert_gemm(desc: LayoutDesc, layout: Layout, x: torch.Tensor, w: torch.Tensor, act: int = MOE_ACT_NONE, out=None,
                    pre=None, balance: Optional[Balance] = None, slots_per_rank: int = 0, stream=None) -> torch.Tensor:
    """Every expert's bf16 rows times its weights: out [max_recv,N] bf16.

    x [max_recv,H]; w [E,M,H], M = N, or 2N with MOE_ACT_SWIGLU (N gate rows,
    then N up rows).  ``pre`` [max_recv,2N] (SWIGLU only; fp32, or bf16 for half the
    bytes and gradients off by its rounding) receives the gate's and up's values
    before the activation, for moe_expert_gemm_backward_x.  Rows that hold no entry are neither read nor written."""
    dev, rows = x.device, _product_rows(desc, "moe_expert_gemm")
    H, N, M = _gemm_shape(desc, x, w, act, torch.bfloat16, "moe_expert_gemm")
    _check_rows(x, "x", torch.bfloat16, rows, H, dev)
    if pre is not None:
        if act != MOE_ACT_SWIGLU:
            raise MoeError(MOE_ERR_SHAPE, "moe_expert_gemm")
        _check_pre(pre, rows, M, dev)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(rows, N, dtype=torch.bfloat16, device=dev)
    else:
        _check_rows(out, "out", torch.bfloat16, rows, N, dev)
    b, bal = _check_segments(desc, layout, balance, slots_per_rank, dev)
    with _on_device(dev):
        rc = _lib.moe_expert_gemm(_made_once(desc), b, bal, slots_per_rank, x.data_ptr(), H, w.data_ptr(), N, act, _ptr(pre),
                                  _pre_type(pre), out.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_expert_gemm")
    return out


def moe_expert_gemm_backward_x(desc: LayoutDesc, layout: Layout, d_out: torch.Tensor, w: torch.Tensor, pre=None, out=None,
                               balance: Optional[Balance] = None, slots_per_rank: int = 0, stream=None) -> torch.Tensor:
    """Gradient of a product's rows: d_out [max_recv,N] times w [E,N,H] -> [max_recv,H] bf16.

    With ``pre`` [max_recv,2H], of the SWIGLU product that made those rows, the
    gradient goes on through the activation to pre: [max_recv,2H] (which may be a
    bf16 pre itself).  Rows that hold no entry are neither read nor written."""
    dev, rows = d_out.device, _product_rows(desc, "moe_expert_gemm_backward_x")
    N = d_out.shape[-1]
    _check_rows(d_out, "d_out", torch.bfloat16, rows, N, dev)
    if w.dim() != 3:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [E, N, H]")
    H = w.shape[2]
    _check(w, "w", torch.bfloat16, (desc.E, N, H), dev)
    width = H
    if pre is not None:
        width = 2 * H
        _check_pre(pre, rows, width, dev)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(rows, width, dtype=torch.bfloat16, device=dev)
    else:
        _check_rows(out, "out", torch.bfloat16, rows, width, dev)
    b, bal = _check_segments(desc, layout, balance, slots_per_rank, dev)
    with _on_device(dev):
        rc = _lib.moe_expert_gemm_backward_x(_made_once(desc), b, bal, slots_per_rank, d_out.data_ptr(), N, w.data_ptr(), H,
                                             _ptr(pre), _pre_type(pre), out.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_expert_gemm_backward_x")
    return out


def moe_expert_gemm_backward_w(desc: LayoutDesc, layout: Layout, d_out: torch.Tensor, x: torch.Tensor, out=None,
                               dtype=torch.bfloat16, balance: Optional[Balance] = None, slots_per_rank: int = 0,
                               stream=None) -> torch.Tensor:
    """Gradient of a product's weights: [E,N,H] in ``dtype`` (bf16 or fp32; of
    ``out`` if it is given) from d_out [max_recv,N] and the rows x [max_recv,H].
    Every element is written, 0 for an expert without a row."""
    dev, rows = x.device, _product_rows(desc, "moe_expert_gemm_backward_w")
    N, H = d_out.shape[-1], x.shape[-1]
    _check_rows(d_out, "d_out", torch.bfloat16, rows, N, dev)
    _check_rows(x, "x", torch.bfloat16, rows, H, dev)
    if out is None:
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"dtype {dtype}, expected bfloat16 or float32")
        with _alloc_on(stream):
            out = torch.empty(desc.E, N, H, dtype=dtype, device=dev)
    else:
        _check(out, "out", (torch.bfloat16, torch.float32), (desc.E, N, H), dev)
    b, bal = _check_segments(desc, layout, balance, slots_per_rank, dev)
    with _on_device(dev):
        rc = _lib.moe_expert_gemm_backward_w(_made_once(desc), b, bal, slots_per_rank, d_out.data_ptr(), N, x.data_ptr(), H,
                                             MOE_F32 if out.dtype is torch.float32 else MOE_BF16, out.data_ptr(),
                                             _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_expert_gemm_backward_w")
    return out


def moe_combine_backward(desc: LayoutDesc, layout: Layout, d_out: torch.Tensor, expert_out=None, w=None, d_expert_out=None,
                         d_w=None, rows: bool = True, weights: bool = True, stream=None):
    """Gradient of moe_combine: (d_expert_out [max_recv,H] bf16 or None, d_w
    [S,K] fp32 or None) from d_out [S,H] bf16; ``rows`` and ``weights`` say
    which of the two are wanted.  d_w needs expert_out; w None: weight 1.
    d_expert_out may be expert_out itself; rows that hold no entry are neither
    read nor written."""
    dev, n, H = d_out.device, _product_rows(desc, "moe_combine_backward"), d_out.shape[-1]
    _check(d_out, "d_out", torch.bfloat16, (desc.S, H))
    _check(w, "w", torch.float32, (desc.S, desc.K), dev)
    _check(layout.pos, "layout.pos", torch.int32, (desc.S, desc.K), dev)
    if weights:
        if expert_out is None:
            raise ValueError("d_w needs expert_out")
        _check_rows(expert_out, "expert_out", torch.bfloat16, n, H, dev)
    with _alloc_on(stream):
        if not rows:
            d_expert_out = None
        elif d_expert_out is None:
            d_expert_out = torch.empty(n, H, dtype=torch.bfloat16, device=dev)
        else:
            _check_rows(d_expert_out, "d_expert_out", torch.bfloat16, n, H, dev)
        if not weights:
            d_w = None
        elif d_w is None:
            d_w = torch.empty(desc.S, desc.K, dtype=torch.float32, device=dev)
        else:
            _check(d_w, "d_w", torch.float32, (desc.S, desc.K), dev)
    b = moe_layout_bufs(pos=layout.pos.data_ptr())
    with _on_device(dev):
        rc = _lib.moe_combine_backward(_made_once(desc), ctypes.byref(b), d_out.data_ptr(), H,
                                       _ptr(expert_out) if weights else None, _ptr(w), _ptr(d_expert_out), _ptr(d_w),
                                       _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_combine_backward")
    return d_expert_out, d_w


def moe_quantize_i8(x: torch.Tensor, codes=None, scales=None, layout: Optional[Layout] = None, stream=None):
    """bf16 rows [..,H] -> 8-bit integers: (codes [..,H] int8, scales [..] fp32),
    a scale per row: per token of activations, per output channel of weights
    [E,N,H].  With ``layout`` only the rows that hold an entry are converted."""
    dev, H = x.device, x.shape[-1]
    _check(x, "x", torch.bfloat16)
    if H < 16 or H % 16:
        raise MoeError(MOE_ERR_SHAPE, "moe_quantize_i8")
    rows = x.numel() // H
    src = _check_src(layout, rows, dev)
    lead = x.shape[:-1]
    with _alloc_on(stream):
        if codes is None:
            codes = torch.empty(*lead, H, dtype=torch.int8, device=dev)
        else:
            _check(codes, "codes", torch.int8, x.shape, dev)
        if scales is None:
            scales = torch.empty(lead, dtype=torch.float32, device=dev)
        else:
            _check(scales, "scales", torch.float32, lead, dev)
    with _on_device(dev):
        rc = _lib.moe_quantize_i8(x.data_ptr(), rows, H, _ptr(src), codes.data_ptr(), scales.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_quantize_i8")
    return codes, scales


def moe_dequantize_i8(codes: torch.Tensor, scales: torch.Tensor, out=None, layout: Optional[Layout] = None, stream=None):
    """8-bit rows -> bf16 [..,H].  With ``layout`` only the rows that hold an
    entry are converted; the others keep what they held."""
    dev, H = codes.device, codes.shape[-1]
    _check(codes, "codes", torch.int8)
    if H < 16 or H % 16:
        raise MoeError(MOE_ERR_SHAPE, "moe_dequantize_i8")
    _check(scales, "scales", torch.float32, codes.shape[:-1], dev)
    rows = codes.numel() // H
    src = _check_src(layout, rows, dev)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(codes.shape, dtype=torch.bfloat16, device=dev)
    else:
        _check(out, "out", torch.bfloat16, codes.shape, dev)
    with _on_device(dev):
        rc = _lib.moe_dequantize_i8(codes.data_ptr(), scales.data_ptr(), rows, H, _ptr(src), out.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_dequantize_i8")
    return out


def moe_dispatch_i8(desc: LayoutDesc, layout: Layout, hidden: torch.Tensor, topk_w=None, recv=None, recv_scales=None,
                    recv_w=None, stream=None):
    """moe_dispatch in 8-bit integers.  Returns (recv [max_recv,H] int8,
    recv_scales [max_recv] fp32, recv_w or None)."""
    dev, H, rows = hidden.device, hidden.shape[-1], _product_rows(desc, "moe_dispatch_i8")
    _check(hidden, "hidden", torch.bfloat16, (desc.S, H))
    _check(topk_w, "topk_w", torch.float32, (desc.S, desc.K), dev)
    _check(layout.pos, "layout.pos", torch.int32, (desc.S, desc.K), dev)
    with _alloc_on(stream):
        if recv is None:
            recv = torch.empty(rows, H, dtype=torch.int8, device=dev)
        else:
            _check_rows(recv, "recv", torch.int8, rows, H, dev)
        if recv_scales is None:
            recv_scales = torch.empty(rows, dtype=torch.float32, device=dev)
        if recv_w is None and topk_w is not None:
            recv_w = torch.empty(rows, dtype=torch.float32, device=dev)
    for t, name in ((recv_scales, "recv_scales"), (recv_w, "recv_w")):
        _check(t, name, torch.float32, None, dev)
        if t is not None and t.numel() < rows:
            raise ValueError(f"{name}: {t.numel()} rows, expected at least {rows}")
    b = moe_layout_bufs(pos=layout.pos.data_ptr())
    with _on_device(dev):
        rc = _lib.moe_dispatch_i8(_made_once(desc), ctypes.byref(b), hidden.data_ptr(), H, _ptr(topk_w), recv.data_ptr(),
                                  recv_scales.data_ptr(), _ptr(recv_w), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_dispatch_i8")
    return recv, recv_scales, recv_w


def moe_expert_gemm_i8(desc: LayoutDesc, layout: Layout, x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor,
                       w_scales: torch.Tensor, act: int = MOE_ACT_NONE, out=None, balance: Optional[Balance] = None,
                       slots_per_rank: int = 0, stream=None) -> torch.Tensor:
    """Every expert's 8-bit rows times its 8-bit weights: out [max_recv,N] bf16.

    x [max_recv,H] int8 and x_scales [max_recv] fp32; w [E,M,H] int8 and
    w_scales [E,M] fp32, M = N, or 2N with MOE_ACT_SWIGLU (N gate rows, then N up
    rows).  Rows that hold no entry are neither read nor written."""
    dev, rows = x.device, _product_rows(desc, "moe_expert_gemm_i8")
    H, N, M = _gemm_shape(desc, x, w, act, torch.int8, "moe_expert_gemm_i8")
    _check_rows(x, "x", torch.int8, rows, H, dev)
    _check(x_scales, "x_scales", torch.float32, None, dev)
    if x_scales.dim() != 1 or x_scales.numel() < rows:
        raise ValueError(f"x_scales: shape {tuple(x_scales.shape)}, expected [at least {rows}]")
    _check(w_scales, "w_scales", torch.float32, (desc.E, M), dev)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(rows, N, dtype=torch.bfloat16, device=dev)
    else:
        _check_rows(out, "out", torch.bfloat16, rows, N, dev)
    b, bal = _check_segments(desc, layout, balance, slots_per_rank, dev)
    with _on_device(dev):
        rc = _lib.moe_expert_gemm_i8(_made_once(desc), b, bal, slots_per_rank, x.data_ptr(), x_scales.data_ptr(), H, w.data_ptr(),
                                     w_scales.data_ptr(), N, act, out.data_ptr(), _stream(stream, dev))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_expert_gemm_i8")
    return out


class _DispatchFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, desc, layout):
        ctx.desc = desc
        ctx.save_for_backward(layout.pos)
        recv = moe_dispatch(desc, layout, hidden)[0]
        moe_zero_padding(desc, layout, recv)
        return recv

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d):
        _no_capture("dispatch", backward=True)
        pos, = ctx.saved_tensors
        return moe_combine(ctx.desc, _only(pos=pos), d.contiguous()), None, None


class _ExpertFfnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_in, w_out, desc, layout, balance, slots, pre_dtype):
        rows, M = _product_rows(desc, "expert_ffn"), w_in.shape[1]
        pre = None if pre_dtype is None else torch.empty(rows, M, dtype=pre_dtype, device=x.device)
        h = moe_expert_gemm(desc, layout, x, w_in, MOE_ACT_SWIGLU, pre=pre, balance=balance, slots_per_rank=slots)
        y = moe_expert_gemm(desc, layout, h, w_out, balance=balance, slots_per_rank=slots)
        moe_zero_padding(desc, layout, y)
        ctx.desc, ctx.slots, ctx.balanced = desc, slots, balance is not None
        seg = (balance.seg_offset, balance.slot_expert) if balance is not None else (None, None)
        ctx.save_for_backward(x, w_in, w_out, h, pre, layout.tokens_per_expert, layout.expert_offset, layout.src, *seg)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        _no_capture("expert_ffn", backward=True)
        x, w_in, w_out, h, pre, count, offset, src, seg, slot_expert = ctx.saved_tensors
        layout = _only(tokens_per_expert=count, expert_offset=offset, src=src)
        balance = Balance(seg, slot_expert, None) if ctx.balanced else None
        at = dict(balance=balance, slots_per_rank=ctx.slots)
        want_x, want_in, want_out = ctx.needs_input_grad[:3]
        dy = dy.contiguous()
        dx = dw_in = dw_out = None
        if want_out:
            dw_out = moe_expert_gemm_backward_w(ctx.desc, layout, dy, h, **at)
        if want_x or want_in:
            d_pre = moe_expert_gemm_backward_x(ctx.desc, layout, dy, w_out, pre=pre, **at)
        if want_in:
            dw_in = moe_expert_gemm_backward_w(ctx.desc, layout, d_pre, x, **at)
        if want_x:
            dx = moe_expert_gemm_backward_x(ctx.desc, layout, d_pre, w_in, **at)
            moe_zero_padding(ctx.desc, layout, dx)
        return dx, dw_in, dw_out, None, None, None, None, None


class _CombineFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, expert_out, w, shared_out, desc, layout):
        ctx.desc = desc
        ctx.save_for_backward(expert_out, w, layout.pos, layout.src)
        return moe_combine(desc, layout, expert_out, w, shared_out)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d):
        _no_capture("combine", backward=True)
        expert_out, w, pos, src = ctx.saved_tensors
        want_y, want_w, want_shared = ctx.needs_input_grad[:3]
        d = d.contiguous()
        dy = dw = None
        if want_y or want_w:
            layout = _only(pos=pos, src=src)
            dy, dw = moe_combine_backward(ctx.desc, layout, d, expert_out, w, rows=want_y, weights=want_w)
            if want_y:
                moe_zero_padding(ctx.desc, layout, dy)
        return dy, dw, d if want_shared else None, None, None


def _only(**arrays) -> Layout:
    """A layout of which a call reads these arrays alone."""
    return Layout(**{f.name: arrays.get(f.name) for f in dataclasses.fields(Layout)})


def dispatch(desc: LayoutDesc, layout: Layout, hidden: torch.Tensor) -> torch.Tensor:
    """moe_dispatch in bf16 as an autograd function of hidden: the receive rows
    [max_recv,H], those that hold no entry zero.  As for router, not capturable
    (nor are expert_ffn and combine); the layout must stay as it is until the
    backward pass has run."""
    _no_capture("dispatch")
    with _on_device(hidden.device):
        return _DispatchFunction.apply(hidden, desc, layout)


def expert_ffn(desc: LayoutDesc, layout: Layout, x: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor,
               balance: Optional[Balance] = None, slots_per_rank: int = 0, pre_dtype=torch.float32) -> torch.Tensor:
    """The experts' gated feed-forward block as an autograd function of its rows
    x [max_recv,H] and of the weights w_in [E,2N,H] (N gate rows, then N up rows) and
    w_out [E,H',N], all bf16: moe_expert_gemm twice.  Rows that hold no entry are
    zero, in the result and in x's gradient.  The activation's arguments are kept
    for the gradients of x and w_in in ``pre_dtype``: fp32, or bf16 for half the
    memory and gradients off by its rounding."""
    _no_capture("expert_ffn")
    if pre_dtype not in _PRE_TYPES:
        raise TypeError(f"pre_dtype {pre_dtype}, expected float32 or bfloat16")
    _check(x, "x", torch.bfloat16, (_product_rows(desc, "expert_ffn"), x.shape[-1]))
    _check(layout.src, "layout.src", torch.int32, (x.shape[0],), x.device)
    kept = pre_dtype if torch.is_grad_enabled() and (x.requires_grad or w_in.requires_grad) else None
    with _on_device(x.device):
        return _ExpertFfnFunction.apply(x, w_in, w_out, desc, layout, balance, slots_per_rank, kept)


def combine(desc: LayoutDesc, layout: Layout, expert_out: torch.Tensor, w=None, shared_out=None) -> torch.Tensor:
    """moe_combine as an autograd function of the experts' rows, the route
    weights and the shared output."""
    _no_capture("combine")
    _check(expert_out, "expert_out", torch.bfloat16, (_product_rows(desc, "combine"), expert_out.shape[-1]))
    _check(layout.src, "layout.src", torch.int32, (expert_out.shape[0],), expert_out.device)
    with _on_device(expert_out.device):
        return _CombineFunction.apply(expert_out, w, shared_out, desc, layout)


# ---------------------------------------------------------------------------
# Static-shape buffer: validate once, then bare C calls
# ---------------------------------------------------------------------------

class Buffer:
    """All device buffers of one batch shape, allocated once (static shapes, no
    host sync between layers), with prepared C calls.

    Mirrors the call shape of MoonEP's Buffer (MoonEP article, basic usage):
    ``dispatch(hidden, topk_w, topk_idx)`` returns the expert-grouped rows,
    their per-row weights and the per-expert offsets; ``combine(expert_out)``
    returns the token-order result.  Every call is asynchronous on the current
    stream (or the one given); outputs are views of the buffer's own tensors
    and are overwritten by the next call.

    With ``balance_slots=B`` the layout is the balanced one (moe_layout_balanced:
    every rank receives the same number of rows, the surplus of hot experts
    going to B replica slots per rank; MoonEP article, section 1); dispatch and
    combine are unchanged.  ``balance.slot_expert`` then tells which expert each
    slot must hold.

    With ``mx4`` the rows travel in MXFP4 (recv [rows,H/2] and recv_scales
    [rows,H/32], both uint8; moe_dispatch_mx4), and expert_gemm multiplies them
    with the experts' weights, with either layout.  With ``i8`` they travel in
    8-bit integers (recv [rows,H] int8, recv_scales [rows] fp32; moe_dispatch_i8).
    """

    def __init__(self, S: int, H: int, K: int, E: int, R: int, fp8: bool = False,
                 pad_mode: int = MOE_PAD_NONE, pad_rows: int = 0, device="cuda",
                 balance_slots: Optional[int] = None, mx4: bool = False, i8: bool = False):
        if balance_slots is not None and pad_mode != MOE_PAD_NONE:
            raise MoeError(MOE_ERR_SHAPE, "Buffer: the balanced layout has no padding")
        self.desc = LayoutDesc(S, K, E, R, pad_mode, pad_rows)
        self.rows = moe_max_recv_rows(self.desc)
        if self.rows < 0 or H < 8 or H % 8 or ((fp8 or mx4) and H % 128) or (i8 and H % 16) or \
                fp8 + mx4 + i8 > 1:
            raise MoeError(MOE_ERR_SHAPE, "Buffer")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.H, self.fp8, self.mx4, self.i8, self.device, self._index = H, fp8, mx4, i8, dev, dev.index
        self.layout = alloc_layout(self.desc, dev)
        if mx4:
            self.recv = torch.empty((self.rows, H // 2), dtype=torch.uint8, device=dev)
            self.recv_scales = torch.empty((self.rows, H // 32), dtype=torch.uint8, device=dev)
        elif i8:
            self.recv = torch.empty((self.rows, H), dtype=torch.int8, device=dev)
            self.recv_scales = torch.empty(self.rows, dtype=torch.float32, device=dev)
        else:
            self.recv = torch.empty((self.rows, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
            self.recv_scales = torch.empty((self.rows, H // 128), dtype=torch.float32, device=dev) if fp8 else None
        self.recv_w = torch.empty(self.rows, dtype=torch.float32, device=dev)
        self.out = torch.empty((S, H), dtype=torch.bfloat16, device=dev)
        self._d = self.desc.c()
        self._b = self.layout.c()
        self._dp = ctypes.byref(self._d)
        self._bp = ctypes.byref(self._b)
        ws = self.layout.workspace
        self._ws = (_ptr(ws), 0 if ws is None else ws.numel())
        self._recv = _ptr(self.recv)
        self._scales = _ptr(self.recv_scales)
        self._recv_w = _ptr(self.recv_w)
        self._out = _ptr(self.out)
        self.balance, self.slots = None, balance_slots
        if balance_slots is not None:
            self.balance = alloc_balance(self.desc, balance_slots, dev)
            self._bal = self.balance.c()
            self._balp = ctypes.byref(self._bal)
            bws = self.balance.workspace
            self._bws = (_ptr(bws), 0 if bws is None else bws.numel())

    def _inputs(self, hidden, topk_idx, topk_w):
        S, K = self.desc.S, self.desc.K
        _check(topk_idx, "topk_idx", torch.int32, (S, K), self.device)
        _check(hidden, "hidden", torch.bfloat16, (S, self.H), self.device)
        _check(topk_w, "topk_w", torch.float32, (S, K), self.device)

    # The C calls launch on the current device.  A call that finds another one
    # than the buffer's makes itself again with the buffer's: one comparison in
    # the usual case (a context manager around every call takes 0.3 us).

    def layout_call(self, topk_idx, stream=None, check=True):
        if self._index != _raw_current_device():
            with torch.cuda.device(self.device):
                return self.layout_call(topk_idx, stream, check)
        if check:
            _check(topk_idx, "topk_idx", torch.int32, (self.desc.S, self.desc.K), self.device)
        if self.balance is not None:
            rc = _lib.moe_layout_balanced(self._dp, self.slots, _ptr(topk_idx), self._bp, self._balp,
                                          self._bws[0], self._bws[1], _stream(stream, self.device))
            if rc != MOE_OK:
                raise MoeError(rc, "moe_layout_balanced")
            return
        rc = _lib.moe_layout(self._dp, _ptr(topk_idx), self._bp, self._ws[0], self._ws[1],
                             _stream(stream, self.device))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_layout")

    def dispatch_call(self, hidden, topk_idx=None, topk_w=None, stream=None, check=True):
        if self._index != _raw_current_device():
            with torch.cuda.device(self.device):
                return self.dispatch_call(hidden, topk_idx, topk_w, stream, check)
        if check:
            self._inputs(hidden, topk_idx, topk_w)
        if self.mx4 or self.i8:
            call = _lib.moe_dispatch_mx4 if self.mx4 else _lib.moe_dispatch_i8
            rc = call(self._dp, self._bp, _ptr(hidden), self.H, _ptr(topk_w), self._recv, self._scales,
                      self._recv_w if topk_w is not None else None, _stream(stream, self.device))
            if rc != MOE_OK:
                raise MoeError(rc, "moe_dispatch_mx4" if self.mx4 else "moe_dispatch_i8")
            return
        rc = _lib.moe_dispatch(self._dp, self._bp, _ptr(hidden), self.H, _ptr(topk_idx), _ptr(topk_w),
                               1 if self.fp8 else 0, self._recv, self._scales,
                               self._recv_w if topk_w is not None else None, _stream(stream, self.device))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_dispatch")

    def layout_dispatch_call(self, hidden, topk_idx, topk_w=None, stream=None, check=True):
        """moe_layout_dispatch: one launch for decode-sized batches (with a
        balanced layout, MXFP4 or 8-bit rows: the layout, then the dispatch)."""
        if self._index != _raw_current_device():
            with torch.cuda.device(self.device):
                return self.layout_dispatch_call(hidden, topk_idx, topk_w, stream, check)
        if check:
            self._inputs(hidden, topk_idx, topk_w)
        if self.balance is not None or self.mx4 or self.i8:
            self.layout_call(topk_idx, stream, check=False)
            self.dispatch_call(hidden, topk_idx, topk_w, stream, check=False)
            return
        rc = _lib.moe_layout_dispatch(self._dp, _ptr(topk_idx), self._bp, self._ws[0], self._ws[1], _ptr(hidden),
                                      self.H, _ptr(topk_w), 1 if self.fp8 else 0, self._recv, self._scales,
                                      self._recv_w if topk_w is not None else None, _stream(stream, self.device))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_layout_dispatch")

    def combine_call(self, expert_out, w=None, shared_out=None, stream=None, check=True):
        if self._index != _raw_current_device():
            with torch.cuda.device(self.device):
                return self.combine_call(expert_out, w, shared_out, stream, check)
        if check:
            _check(expert_out, "expert_out", torch.bfloat16, (self.rows, self.H), self.device)
            _check(w, "w", torch.float32, (self.desc.S, self.desc.K), self.device)
            _check(shared_out, "shared_out", torch.bfloat16, (self.desc.S, self.H), self.device)
        rc = _lib.moe_combine(self._dp, self._bp, _ptr(expert_out), self.H, _ptr(w), _ptr(shared_out),
                              self._out, _stream(stream, self.device))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_combine")

    def zero_padding_call(self, stream=None):
        """moe_zero_padding on this buffer's receive rows (after a dispatch; not
        for MXFP4 and 8-bit rows, whose consumers skip padding)."""
        if self.mx4 or self.i8:
            raise MoeError(MOE_ERR_SHAPE, "moe_zero_padding")
        if self._index != _raw_current_device():
            with torch.cuda.device(self.device):
                return self.zero_padding_call(stream)
        rc = _lib.moe_zero_padding(self._dp, self._bp, self.H, 1 if self.fp8 else 0, self._recv, self._scales,
                                   _stream(stream, self.device))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_zero_padding")

    def dispatch(self, hidden, topk_w, topk_idx, stream=None):
        """Layout + dispatch.  Returns (recv, recv_w, expert_offset, recv_scales)."""
        self.layout_dispatch_call(hidden, topk_idx, topk_w, stream)
        return self.recv, self.recv_w, self.layout.expert_offset, self.recv_scales

    def combine(self, expert_out, w=None, shared_out=None, stream=None):
        """Route-weighted gather back to token order.  Returns out [S,H] bf16."""
        self.combine_call(expert_out, w, shared_out, stream)
        return self.out

    def expert_gemm(self, w, w_scales=None, act: int = MOE_ACT_NONE, x=None, x_scales=None, out=None, stream=None):
        """The experts' product in the weights' format, MXFP4 (uint8), 8-bit integers
        (int8) or bf16 (no scales): moe_expert_gemm_mx4, moe_expert_gemm_i8 or
        moe_expert_gemm on the rows of the last dispatch, or on x and x_scales (rows of
        that format in the same order, such as the previous product's result,
        quantised).  Returns [rows,N] bf16."""
        mx4, i8 = w.dtype is torch.uint8, w.dtype is torch.int8
        if x is None:
            if self.fp8 or (self.mx4, self.i8) != (mx4, i8):
                raise MoeError(MOE_ERR_SHAPE, "Buffer.expert_gemm: the receive rows have another format than the weights")
            x, x_scales = self.recv, self.recv_scales
        if mx4 or i8:
            call = moe_expert_gemm_mx4 if mx4 else moe_expert_gemm_i8
            return call(self.desc, self.layout, x, x_scales, w, w_scales, act, out, self.balance, self.slots or 0, stream)
        if w_scales is not None or x_scales is not None:
            raise ValueError("bf16 rows and weights have no scales")
        return moe_expert_gemm(self.desc, self.layout, x, w, act, out, None, self.balance, self.slots or 0, stream)
