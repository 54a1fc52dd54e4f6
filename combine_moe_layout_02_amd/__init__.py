"""MI355X-native MoE expert-parallel layout, dispatch and combine.

Thin ctypes binding over libmoe_ep.so (declared in include/moe_ep.h).  The
Python functions carry the C names and only marshal arguments: torch tensors
supply device memory and the current HIP stream, every step of the path runs
in the library's HIP kernels.  ``router`` and ``balance_loss`` are the same
calls as autograd functions.  Importing this package fails loudly when the
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
            "moe_router_backward", "moe_quantize_mx4", "moe_dequantize_mx4", "moe_dispatch_mx4", "moe_expert_gemm_mx4")


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
    for f in (L.moe_router, L.moe_balance_loss, L.moe_router_backward, L.moe_quantize_mx4, L.moe_dequantize_mx4,
              L.moe_dispatch_mx4, L.moe_expert_gemm_mx4):
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
        return {k: v for k, v in self.__dict__.items() if k != "_ref"}


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
        return moe_layout_bufs(*(t.data_ptr() for t in (
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


def _no_capture(what: str):
    # autograd joins the streams of the leaves that live outside the capture
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what} cannot be captured into a graph: capture moe_router / moe_balance_loss and "
                           "moe_router_backward instead")


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
        _no_capture("the backward pass of router / balance_loss")
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
    with the experts' weights, with either layout.
    """

    def __init__(self, S: int, H: int, K: int, E: int, R: int, fp8: bool = False,
                 pad_mode: int = MOE_PAD_NONE, pad_rows: int = 0, device="cuda",
                 balance_slots: Optional[int] = None, mx4: bool = False):
        if balance_slots is not None and pad_mode != MOE_PAD_NONE:
            raise MoeError(MOE_ERR_SHAPE, "Buffer: the balanced layout has no padding")
        self.desc = LayoutDesc(S, K, E, R, pad_mode, pad_rows)
        self.rows = moe_max_recv_rows(self.desc)
        if self.rows < 0 or H < 8 or H % 8 or ((fp8 or mx4) and H % 128) or (fp8 and mx4):
            raise MoeError(MOE_ERR_SHAPE, "Buffer")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.H, self.fp8, self.mx4, self.device, self._index = H, fp8, mx4, dev, dev.index
        self.layout = alloc_layout(self.desc, dev)
        if mx4:
            self.recv = torch.empty((self.rows, H // 2), dtype=torch.uint8, device=dev)
            self.recv_scales = torch.empty((self.rows, H // 32), dtype=torch.uint8, device=dev)
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
        if self.mx4:
            rc = _lib.moe_dispatch_mx4(self._dp, self._bp, _ptr(hidden), self.H, _ptr(topk_w), self._recv, self._scales,
                                       self._recv_w if topk_w is not None else None, _stream(stream, self.device))
            if rc != MOE_OK:
                raise MoeError(rc, "moe_dispatch_mx4")
            return
        rc = _lib.moe_dispatch(self._dp, self._bp, _ptr(hidden), self.H, _ptr(topk_idx), _ptr(topk_w),
                               1 if self.fp8 else 0, self._recv, self._scales,
                               self._recv_w if topk_w is not None else None, _stream(stream, self.device))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_dispatch")

    def layout_dispatch_call(self, hidden, topk_idx, topk_w=None, stream=None, check=True):
        """moe_layout_dispatch: one launch for decode-sized batches (with a
        balanced layout or MXFP4 rows: the layout, then the dispatch)."""
        if self._index != _raw_current_device():
            with torch.cuda.device(self.device):
                return self.layout_dispatch_call(hidden, topk_idx, topk_w, stream, check)
        if check:
            self._inputs(hidden, topk_idx, topk_w)
        if self.balance is not None or self.mx4:
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
        for MXFP4 rows, whose consumers skip padding)."""
        if self.mx4:
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

    def expert_gemm(self, w, w_scales, act: int = MOE_ACT_NONE, x=None, x_scales=None, out=None, stream=None):
        """moe_expert_gemm_mx4 on the rows of the last dispatch, or on x and
        x_scales (MXFP4 rows in the same order, such as the previous product's
        result through moe_quantize_mx4).  Returns [rows,N] bf16."""
        if x is None:
            if not self.mx4:
                raise MoeError(MOE_ERR_SHAPE, "Buffer.expert_gemm: the receive rows are not MXFP4")
            x, x_scales = self.recv, self.recv_scales
        return moe_expert_gemm_mx4(self.desc, self.layout, x, x_scales, w, w_scales, act, out, self.balance,
                                   self.slots or 0, stream)
