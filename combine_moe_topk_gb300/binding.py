"""ctypes binding of ``libmoe_gb300.so`` (C ABI in ``include/moe_gb300.h``).

Argument marshalling only: every step of the token path runs in the CUDA
library.  PyTorch supplies device memory (outputs are allocated with
``torch.empty`` when the caller does not pass them) and the current CUDA
stream.  The functions keep the C names; tensors replace (pointer, size)
pairs.  Every non-OK status raises ``MoEError``; if the shared library is
missing the first call raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")

MOE_OK = 0
STATUS = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_DTYPE",
    4: "MOE_ERR_HANDLE_MISMATCH", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_OOM", 7: "MOE_ERR_TIMEOUT",
    8: "MOE_ERR_NONFINITE", 9: "MOE_ERR_BAD_ROUTE",
}
MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
MOE_DEV_NONFINITE, MOE_DEV_BAD_ROUTE, MOE_DEV_TIMEOUT, MOE_DEV_ROWS_EXCEEDED = 0x1, 0x2, 0x4, 0x8
KERNELS = ["topk_gate", "layout", "dispatch", "combine", "combine_bwd", "dispatch_bwd", "topk_gate_bwd",
           "grouped_gemm", "dispatch_gemm", "rank_slots", "combine_gate_bwd", "gate_layout", "ep_pack", "ep_unpack",
           "ep_dispatch", "ep_combine", "layernorm", "layernorm_bwd", "balance", "balance_bwd", "linear",
           "linear_bwd", "gated", "gated_bwd", "grouped_gated", "grouped_gated_bwd", "grouped_gemm_bwd", "grad_norm",
           "grad_clip"]
KERNEL_ID = {n: i for i, n in enumerate(KERNELS)}

# every entry point the header declares (checked by the CPU test-suite)
EXPORTS = [
    "moe_topk_gate", "moe_dispatch_layout", "moe_dispatch", "moe_combine", "moe_combine_bwd",
    "moe_dispatch_bwd", "moe_handle_info", "moe_handle_status", "moe_handle_destroy", "moe_capacity",
    "moe_status_string", "moe_last_error", "moe_launch_count", "moe_debug_hold_layout_tile",
    "moe_dispatch_layout_noalloc", "moe_topk_gate_bwd", "moe_dispatch_layout_ex", "moe_grouped_gemm",
    "moe_dispatch_grouped_gemm", "moe_combine_gate_bwd", "moe_layout_create", "moe_layout_rebuild",
    "moe_topk_gate_layout", "moe_ep_pack", "moe_ep_dispatch", "moe_ep_combine", "moe_ep_unpack_dgate",
    "moe_layernorm", "moe_layernorm_bwd", "moe_layernorm_bwd_workspace", "moe_balance_loss", "moe_balance_loss_bwd",
    "moe_balance_loss_workspace", "moe_linear", "moe_linear_bwd", "moe_linear_bwd_workspace",
    "moe_linear_bwd_workspace_for", "moe_gated_linear", "moe_gated_linear_bwd", "moe_gated_linear_bwd_workspace",
    "moe_grouped_gated", "moe_dispatch_grouped_gated", "moe_grouped_gated_bwd", "moe_grouped_gated_bwd_workspace",
    "moe_grouped_gemm_bwd", "moe_tensor_list_create", "moe_tensor_list_destroy", "moe_grad_norm_workspace",
    "moe_grad_norm", "moe_grad_clip", "moe_clip_grad_norm",
]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{where}: {self.name}" + (f" ({detail})" if detail else ""))


class LayoutOptions(ctypes.Structure):
    _fields_ = [("capacity", ctypes.c_int32), ("num_virtual_ranks", ctypes.c_int32), ("priority", ctypes.c_int32),
                ("pad_multiple", ctypes.c_int32), ("send_slots", ctypes.c_int32), ("absent_routes", ctypes.c_int32),
                ("rows_bound", ctypes.c_int32)]


PRIORITY = {"token": 0, "kmajor": 1}


class LayoutInfo(ctypes.Structure):
    _fields_ = [("s", ctypes.c_int32), ("e", ctypes.c_int32), ("k", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("R", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("device", ctypes.c_int32), ("priority", ctypes.c_int32), ("pad_multiple", ctypes.c_int32)] + [
        (n, ctypes.c_void_p) for n in ("idx", "loc", "row", "drop", "raw_counts", "counts", "offsets",
                                       "token_in_rank", "rank_counts", "status", "inv_row", "rank_slot")]


class LinearDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("s", "K", "N", "act", "out_dtype", "bias_dtype", "residual_dtype")] + [
        (n, ctypes.c_int64) for n in ("ldx", "ldw", "ldres")]


class LinearBwdDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("s", "K", "N", "act", "dy_dtype", "dx_dtype", "dw_dtype")] + [
        (n, ctypes.c_int64) for n in ("lddy", "ldx", "ldw", "ldz")]


class GatedDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("s", "K", "N", "act", "bias_dtype")] + [
        (n, ctypes.c_int64) for n in ("ldx", "ldw")]


class GatedBwdDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("s", "K", "N", "act", "dh_dtype", "dx_dtype", "dw_dtype")] + [
        (n, ctypes.c_int64) for n in ("lddh", "ldx", "ldw", "ldz")]


class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32)]


ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_lib = None


def lib() -> ctypes.CDLL:
    """Load the CUDA library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
                               "g.build()\"` (nvcc, sm_103a); there is no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        P, I, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64
        I64, F, Z = ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        sig = {
            "moe_topk_gate": [P, I, I, I, I, P, P, P, P],
            "moe_topk_gate_bwd": [P, P, P, P, I, I, I, I, P, P],
            "moe_dispatch_layout": [P, I, I, I, I, I, P, ctypes.POINTER(P)],
            "moe_dispatch_layout_ex": [P, I, I, I, ctypes.POINTER(LayoutOptions), P, ctypes.POINTER(P)],
            "moe_layout_create": [I, I, I, ctypes.POINTER(LayoutOptions), P, ctypes.POINTER(P)],
            "moe_layout_rebuild": [P, P, P],
            "moe_topk_gate_layout": [P, P, I, P, P, P],
            "moe_ep_pack": [P, P, I, P, P, P, P],
            "moe_ep_dispatch": [P, P, I, I, I, P, P, P],
            "moe_ep_combine": [P, P, I, I, I, P, P, P],
            "moe_ep_unpack_dgate": [P, P, I, P, P, P],
            "moe_dispatch": [P, I, I, I, I, P, P, P],
            "moe_combine": [P, I, I, I, I, P, P, P, P],
            "moe_combine_bwd": [P, I, I, I, I, P, P, P, P, P, P],
            "moe_combine_gate_bwd": [P, I, I, I, I, P, P, P, P, I, P, P, P, P],
            "moe_dispatch_bwd": [P, I, I, I, I, P, P, P],
            "moe_grouped_gemm": [P, I, I, I, P, P, P, P],
            "moe_dispatch_grouped_gemm": [P, I, I, I, I, P, P, P, P],
            "moe_handle_info": [P, ctypes.POINTER(LayoutInfo)],
            "moe_handle_status": [P, P, ctypes.POINTER(ctypes.c_int32)],
            "moe_handle_destroy": [P],
            "moe_debug_hold_layout_tile": [I, I],
            "moe_dispatch_layout_noalloc": [P, I, I, I, I, I] + [P] * 11,
            "moe_layernorm": [I, I, I, P, I64, I, P, P, F, P, P, P, P],
            "moe_layernorm_bwd": [I, I, I, P, I64, P, I64, I, P, P, P, P, I64, P, P, P, P, Z, P],
            "moe_balance_loss": [P, P, P, P, I, I, I, I, P, P, P, P, P, P, P, Z, P, P],
            "moe_balance_loss_bwd": [P] * 8 + [I, I, I, P, P],
            "moe_linear": [ctypes.POINTER(LinearDesc)] + [P] * 8,
            "moe_linear_bwd": [ctypes.POINTER(LinearBwdDesc)] + [P] * 8 + [Z, P, P],
            "moe_gated_linear": [ctypes.POINTER(GatedDesc)] + [P] * 7,
            "moe_gated_linear_bwd": [ctypes.POINTER(GatedBwdDesc)] + [P] * 8 + [Z, P, P],
            "moe_grouped_gated": [P, I, I, I, I] + [P] * 5,
            "moe_dispatch_grouped_gated": [P, I, I, I, I, I] + [P] * 5,
            "moe_grouped_gated_bwd": [P, I, I, I, I] + [P] * 7 + [Z, P],
            "moe_grouped_gemm_bwd": [P, I, I, I] + [P] * 6,
            "moe_tensor_list_create": [ctypes.POINTER(Tensor), I, ctypes.POINTER(P)],
            "moe_tensor_list_destroy": [P],
            "moe_grad_norm": [P, P, P, Z, P, P],
            "moe_grad_clip": [P, P, P, F, P],
            "moe_clip_grad_norm": [P, P, F, P, P, Z, P, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = I
        for name in ("moe_layernorm_bwd_workspace", "moe_balance_loss_workspace", "moe_linear_bwd_workspace",
                     "moe_grouped_gated_bwd_workspace"):
            f = getattr(L, name)
            f.argtypes = [I, I]
            f.restype = Z
        L.moe_linear_bwd_workspace_for.argtypes = [ctypes.POINTER(LinearBwdDesc), I, I, I]
        L.moe_linear_bwd_workspace_for.restype = Z
        L.moe_gated_linear_bwd_workspace.argtypes = [ctypes.POINTER(GatedBwdDesc), I, I, I]
        L.moe_gated_linear_bwd_workspace.restype = Z
        L.moe_grad_norm_workspace.argtypes = [I]
        L.moe_grad_norm_workspace.restype = Z
        L.moe_capacity.argtypes = [ctypes.c_double, I, I, I]
        L.moe_capacity.restype = I
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_launch_count.argtypes = [I]
        L.moe_launch_count.restype = U
        _lib = L
    return _lib


def _check(rc: int, where: str):
    if rc != MOE_OK:
        detail = lib().moe_last_error().decode(errors="replace")
        raise MoEError(rc, where, detail)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else None


def _rows_ptr(t: torch.Tensor | None):
    """Pointer and row stride (elements) of a 2-D tensor whose rows are contiguous; the rows may be apart."""
    if t is None:
        return None, 0
    if t.is_contiguous():
        return t.data_ptr(), t.shape[1]
    s, m = t.shape
    if m > 1 and t.stride(1) != 1:
        raise ValueError("the rows of tensors passed to the MoE library must be contiguous")
    # with at most one row the stride is never used
    ld = t.stride(0) if s > 1 else m
    if ld < m:
        raise ValueError("rows that overlap (a broadcast or a negative stride) are not supported")
    return t.data_ptr(), ld


def _addr(t: torch.Tensor | None):
    """Address of a contiguous tensor, as an int (a cheaper _ptr)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


def _status_addr(t: torch.Tensor | None, where: str):
    """Address of a status word: the kernels set bits of an int32."""
    if t is not None and 0 < t.numel() * t.element_size() < 4:
        raise MoEError(1, where, "device_status must hold an int32")
    return _addr(t)


def _raw_stream(t: torch.Tensor):
    """The current stream of a CUDA tensor's device; a host tensor goes to the library, which rejects it."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if t.is_cuda else None


# torch's own short way to an uninitialised CUDA tensor on the current device;
# beside a launch torch.empty takes 3.9 us of host time, this 1.4.  It goes past
# the dispatcher, so while a dispatch mode (a memory tracker, say) is active,
# or where either name is missing, torch.empty it is.
_strided = getattr(getattr(torch._C, "_dynamo", None) and torch._C._dynamo.guards, "_empty_strided_cuda", None)
_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
if _modes is None:
    _strided = None


def _new_here(dtype: torch.dtype, n: int, m: int | None = None) -> torch.Tensor:
    return _strided((n,), (1,), dtype) if m is None else _strided((n, m), (m, 1), dtype)


def _new(t: torch.Tensor):
    """How outputs beside t are allocated: new(dtype, n) or new(dtype, n, m), contiguous."""
    if _strided is not None and t.is_cuda and not _modes() and t.get_device() == torch._C._cuda_getDevice():
        return _new_here
    dev = t.device
    return lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=dev)


def _stream(device: torch.device):
    # a host tensor still goes to the library, which rejects it; use the current device's stream
    dev = device if device.type == "cuda" else None
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float16:
        return MOE_F16
    return -1


# ------------------------------------------------------------------ handle --

class _DeviceArray:
    """A CUDA array view of handle memory (``__cuda_array_interface__``); treat it as read-only."""

    def __init__(self, owner, ptr: int, shape: tuple, typestr: str):
        self._owner = owner  # keeps the handle (and its memory) alive
        self.__cuda_array_interface__ = {
            "shape": shape, "typestr": typestr, "data": (ptr or 0, False), "version": 3, "strides": None,
            "stream": None,
        }


class Handle:
    """Owns a ``moe_handle``; destroys it when garbage-collected.  ``gaps``: there may be rows that no route owns."""

    def __init__(self, raw: ctypes.c_void_p, device: torch.device, gaps: bool = False):
        self._raw = raw
        self.device = device
        info = LayoutInfo()
        _check(lib().moe_handle_info(raw, ctypes.byref(info)), "moe_handle_info")
        self.info = info
        self.s, self.e, self.k = info.s, info.e, info.k
        self.capacity, self.R, self.rows = info.capacity, info.R, info.rows
        self.priority, self.pad_multiple = info.priority, info.pad_multiple
        self.gaps = gaps or self.capacity > 0 or self.pad_multiple > 1

    @property
    def raw(self):
        if self._raw is None:
            raise MoEError(4, "handle", "destroyed")
        return self._raw

    def _view(self, name: str, shape: tuple, typestr: str) -> torch.Tensor:
        ptr = getattr(self.info, name)
        if not ptr or 0 in shape:
            dt = {"<i4": torch.int32, "|u1": torch.uint8}[typestr]
            return torch.empty(shape, dtype=dt, device=self.device)
        return torch.as_tensor(_DeviceArray(self, ptr, shape, typestr), device=self.device)

    # device arrays of the layout (views of handle memory, valid while the handle lives)
    def idx(self): return self._view("idx", (self.s, self.k), "<i4")
    def loc(self): return self._view("loc", (self.s, self.k), "<i4")
    def row(self): return self._view("row", (self.s, self.k), "<i4")
    def drop(self): return self._view("drop", (self.s, self.k), "|u1")
    def raw_counts(self): return self._view("raw_counts", (self.e,), "<i4")
    def counts(self): return self._view("counts", (self.e,), "<i4")
    def offsets(self): return self._view("offsets", (self.e + 1,), "<i4")
    def token_in_rank(self): return self._view("token_in_rank", (self.s, self.R), "|u1")
    def rank_counts(self): return self._view("rank_counts", (self.R,), "<i4")
    def inv_row(self): return self._view("inv_row", (self.rows,), "<i4")
    def rank_slot(self):
        if not self.info.rank_slot:
            raise MoEError(1, "rank_slot", "the handle was built without send_slots")
        return self._view("rank_slot", (self.s, self.R), "<i4")

    def status(self) -> int:
        """Synchronise and read the device status word (MOE_DEV_* bits)."""
        v = ctypes.c_int32(0)
        _check(lib().moe_handle_status(self.raw, _stream(self.device), ctypes.byref(v)), "moe_handle_status")
        return v.value

    def destroy(self):
        if self._raw is not None:
            raw, self._raw = self._raw, None
            with torch.cuda.device(self.device):
                _check(lib().moe_handle_destroy(raw), "moe_handle_destroy")

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


# ------------------------------------------------------------- entry points --

def moe_capacity(capacity_factor: float, s: int, k: int, e: int) -> int:
    return lib().moe_capacity(float(capacity_factor), int(s), int(k), int(e))


def moe_launch_count(kernel: str | int) -> int:
    return lib().moe_launch_count(KERNEL_ID.get(kernel, kernel) if isinstance(kernel, str) else kernel)


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def moe_debug_hold_layout_tile(tile: int, timeout_ms: int = 200):
    _check(lib().moe_debug_hold_layout_tile(int(tile), int(timeout_ms)), "moe_debug_hold_layout_tile")


def moe_topk_gate(logits: torch.Tensor, k: int, renorm: int = 1, topk_idx: torch.Tensor | None = None,
                  topk_gate: torch.Tensor | None = None, device_status: torch.Tensor | None = None):
    """logits f32 [s,e] -> (idx i32 [s,k], gate f32 [s,k])."""
    if logits.dim() != 2:
        raise ValueError("logits must be [s, e]")
    s, e = logits.shape
    if logits.dtype != torch.float32:
        raise MoEError(3, "moe_topk_gate", "logits must be float32")
    dev = logits.device
    if topk_idx is None:
        topk_idx = torch.empty(s, k, dtype=torch.int32, device=dev)
    if topk_gate is None:
        topk_gate = torch.empty(s, k, dtype=torch.float32, device=dev)
    rc = lib().moe_topk_gate(_ptr(logits), s, e, int(k), int(renorm), _ptr(topk_idx), _ptr(topk_gate),
                             _status_addr(device_status, "moe_topk_gate"), _stream(dev))
    _check(rc, "moe_topk_gate")
    return topk_idx, topk_gate


def moe_topk_gate_bwd(logits: torch.Tensor | None, topk_idx: torch.Tensor, topk_gate: torch.Tensor,
                      dgate: torch.Tensor, e: int, renorm: int = 1, dlogits: torch.Tensor | None = None):
    """(logits f32 [s,e] or None when renorm=1, idx [s,k], gate [s,k], dgate [s,k]) -> dlogits f32 [s,e]."""
    s, k = topk_idx.shape
    for t, name in ((topk_gate, "topk_gate"), (dgate, "dgate")):
        if t.dtype != torch.float32 or tuple(t.shape) != (s, k):
            raise MoEError(1, "moe_topk_gate_bwd", f"{name} must be float32 [s, k]")
    if logits is not None and (logits.dtype != torch.float32 or tuple(logits.shape) != (s, e)):
        raise MoEError(1, "moe_topk_gate_bwd", "logits must be float32 [s, e]")
    dev = topk_idx.device
    if dlogits is None:
        dlogits = torch.empty(s, e, dtype=torch.float32, device=dev)
    rc = lib().moe_topk_gate_bwd(_ptr(logits), _ptr(topk_idx), _ptr(topk_gate), _ptr(dgate), s, int(e), k,
                                 int(renorm), _ptr(dlogits), _stream(dev))
    _check(rc, "moe_topk_gate_bwd")
    return dlogits


def moe_dispatch_layout(topk_idx: torch.Tensor, e: int, capacity: int = 0, num_virtual_ranks: int = 0) -> Handle:
    """topk_idx i32 [s,k] -> Handle (counts, locations, rows, drops, dedup counts)."""
    if topk_idx.dim() != 2 or topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be int32 [s, k]")
    s, k = topk_idx.shape
    raw = ctypes.c_void_p()
    dev = topk_idx.device
    rc = lib().moe_dispatch_layout(_ptr(topk_idx), s, int(e), k, int(capacity), int(num_virtual_ranks),
                                   _stream(dev), ctypes.byref(raw))
    _check(rc, "moe_dispatch_layout")
    return Handle(raw, dev)


def moe_dispatch_layout_ex(topk_idx: torch.Tensor, e: int, capacity: int = 0, num_virtual_ranks: int = 0,
                           priority: str = "token", pad_multiple: int = 1, send_slots: bool = False,
                           absent_routes: bool = False, rows_bound: int = 0) -> Handle:
    """Layout with a capacity priority ("token" or "kmajor"), per-expert
    padding of the dropless rows (handle.rows is then an upper bound),
    with send_slots each token's token-order slot per virtual rank
    (handle.rank_slot()), with absent_routes expert id -1 taken as a
    route that does not exist, and with rows_bound (dropless) the caller's
    bound on the kept routes as the handle's rows."""
    if topk_idx.dim() != 2 or topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be int32 [s, k]")
    s, k = topk_idx.shape
    opt = LayoutOptions(int(capacity), int(num_virtual_ranks), PRIORITY[priority], int(pad_multiple),
                        int(bool(send_slots)), int(bool(absent_routes)), int(rows_bound))
    raw = ctypes.c_void_p()
    dev = topk_idx.device
    rc = lib().moe_dispatch_layout_ex(_ptr(topk_idx), s, int(e), k, ctypes.byref(opt), _stream(dev),
                                      ctypes.byref(raw))
    _check(rc, "moe_dispatch_layout_ex")
    return Handle(raw, dev, bool(absent_routes) or rows_bound != 0)


def moe_layout_create(s: int, e: int, k: int, capacity: int = 0, num_virtual_ranks: int = 0,
                      priority: str = "token", pad_multiple: int = 1, send_slots: bool = False,
                      device: torch.device | None = None, absent_routes: bool = False,
                      rows_bound: int = 0) -> Handle:
    """An empty handle for [s, k] routes over e experts with these layout
    options, to be built (and rebuilt) in place by moe_layout_rebuild or
    moe_topk_gate_layout without allocating."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    opt = LayoutOptions(int(capacity), int(num_virtual_ranks), PRIORITY[priority], int(pad_multiple),
                        int(bool(send_slots)), int(bool(absent_routes)), int(rows_bound))
    raw = ctypes.c_void_p()
    with torch.cuda.device(dev):
        rc = lib().moe_layout_create(int(s), int(e), int(k), ctypes.byref(opt), _stream(dev), ctypes.byref(raw))
    _check(rc, "moe_layout_create")
    return Handle(raw, dev, bool(absent_routes) or rows_bound != 0)


def moe_layout_rebuild(h: Handle, topk_idx: torch.Tensor) -> Handle:
    """Rebuild h's layout in place from new expert ids i32 [s, k]."""
    if topk_idx.dtype != torch.int32 or tuple(topk_idx.shape) != (h.s, h.k):
        raise MoEError(1, "moe_layout_rebuild", "topk_idx must be int32 [s, k] of the handle's shape")
    _check(lib().moe_layout_rebuild(h.raw, _ptr(topk_idx), _stream(topk_idx.device)), "moe_layout_rebuild")
    return h


def moe_topk_gate_layout(h: Handle, logits: torch.Tensor, renorm: int = 1, topk_idx: torch.Tensor | None = None,
                         topk_gate: torch.Tensor | None = None):
    """The top-k gate and the layout build in one kernel: logits f32 [s, e]
    -> (topk_idx i32 [s, k], topk_gate f32 [s, k]), h rebuilt on those ids."""
    if logits.dtype != torch.float32 or tuple(logits.shape) != (h.s, h.e):
        raise MoEError(1, "moe_topk_gate_layout", "logits must be float32 [s, e] of the handle's shape")
    dev = logits.device
    if topk_idx is None:
        topk_idx = torch.empty(h.s, h.k, dtype=torch.int32, device=dev)
    if topk_gate is None:
        topk_gate = torch.empty(h.s, h.k, dtype=torch.float32, device=dev)
    if tuple(topk_idx.shape) != (h.s, h.k) or tuple(topk_gate.shape) != (h.s, h.k) or \
            topk_idx.dtype != torch.int32 or topk_gate.dtype != torch.float32:
        raise MoEError(1, "moe_topk_gate_layout", "output shapes")
    rc = lib().moe_topk_gate_layout(h.raw, _ptr(logits), int(renorm), _ptr(topk_idx), _ptr(topk_gate), _stream(dev))
    _check(rc, "moe_topk_gate_layout")
    return topk_idx, topk_gate


def _rows2(t: torch.Tensor, name: str) -> tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape[0], t.shape[1]


def moe_dispatch(h: Handle, x: torch.Tensor, X: torch.Tensor | None = None) -> torch.Tensor:
    """x [s,m] -> X [rows,m]."""
    s, m = _rows2(x, "x")
    if X is None:
        X = torch.empty(h.rows, m, dtype=x.dtype, device=x.device)
    rows, mX = _rows2(X, "X")
    if mX != m or X.dtype != x.dtype:
        raise MoEError(1, "moe_dispatch", "x and X disagree in width or dtype")
    _check(lib().moe_dispatch(h.raw, s, rows, m, _dtype(x), _ptr(x), _ptr(X), _stream(x.device)), "moe_dispatch")
    return X


def moe_combine(h: Handle, y: torch.Tensor, gate: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """y [rows,m], gate f32 [s,k] -> out [s,m]."""
    rows, m = _rows2(y, "y")
    if gate.dtype != torch.float32 or gate.shape != (h.s, h.k):
        raise MoEError(1, "moe_combine", "gate must be float32 [s, k]")
    if out is None:
        out = torch.empty(h.s, m, dtype=y.dtype, device=y.device)
    s, mo = _rows2(out, "out")
    if mo != m or out.dtype != y.dtype:
        raise MoEError(1, "moe_combine", "y and out disagree in width or dtype")
    _check(lib().moe_combine(h.raw, s, rows, m, _dtype(y), _ptr(y), _ptr(gate), _ptr(out), _stream(y.device)),
           "moe_combine")
    return out


def moe_combine_bwd(h: Handle, dout: torch.Tensor, gate: torch.Tensor, y: torch.Tensor,
                    dY: torch.Tensor | None = None, dgate: torch.Tensor | None = None):
    """dout [s,m], gate f32 [s,k], y [rows,m] -> (dY [rows,m], dgate f32 [s,k])."""
    s, m = _rows2(dout, "dout")
    rows, my = _rows2(y, "y")
    if my != m or y.dtype != dout.dtype:
        raise MoEError(1, "moe_combine_bwd", "dout and y disagree in width or dtype")
    if gate.dtype != torch.float32 or gate.shape != (h.s, h.k):
        raise MoEError(1, "moe_combine_bwd", "gate must be float32 [s, k]")
    if dY is None:
        dY = torch.empty(rows, m, dtype=dout.dtype, device=dout.device)
    if dgate is None:
        dgate = torch.empty(h.s, h.k, dtype=torch.float32, device=dout.device)
    if dY.shape != (rows, m) or dY.dtype != dout.dtype or dgate.shape != (h.s, h.k):
        raise MoEError(1, "moe_combine_bwd", "output shapes")
    rc = lib().moe_combine_bwd(h.raw, s, rows, m, _dtype(dout), _ptr(dout), _ptr(gate), _ptr(y), _ptr(dY),
                               _ptr(dgate), _stream(dout.device))
    _check(rc, "moe_combine_bwd")
    return dY, dgate


def moe_combine_gate_bwd(h: Handle, dout: torch.Tensor, gate: torch.Tensor, y: torch.Tensor,
                         logits: torch.Tensor | None, renorm: int = 1, dY: torch.Tensor | None = None,
                         dgate: torch.Tensor | None = None, dlogits: torch.Tensor | None = None):
    """The combine backward and the top-k gate backward in one kernel:
    (dY [rows,m], dgate f32 [s,k], dlogits f32 [s,e]); logits f32 [s,e] only
    needed when renorm = 0."""
    s, m = _rows2(dout, "dout")
    rows, my = _rows2(y, "y")
    if my != m or y.dtype != dout.dtype:
        raise MoEError(1, "moe_combine_gate_bwd", "dout and y disagree in width or dtype")
    if gate.dtype != torch.float32 or gate.shape != (h.s, h.k):
        raise MoEError(1, "moe_combine_gate_bwd", "gate must be float32 [s, k]")
    if not renorm and (logits is None or logits.dtype != torch.float32 or logits.shape != (h.s, h.e)):
        raise MoEError(1, "moe_combine_gate_bwd", "logits must be float32 [s, e] when renorm = 0")
    if dY is None:
        dY = torch.empty(rows, m, dtype=dout.dtype, device=dout.device)
    if dgate is None:
        dgate = torch.empty(h.s, h.k, dtype=torch.float32, device=dout.device)
    if dlogits is None:
        dlogits = torch.empty(h.s, h.e, dtype=torch.float32, device=dout.device)
    if dY.shape != (rows, m) or dY.dtype != dout.dtype or dgate.shape != (h.s, h.k) or \
            dlogits.shape != (h.s, h.e) or dlogits.dtype != torch.float32:
        raise MoEError(1, "moe_combine_gate_bwd", "output shapes")
    rc = lib().moe_combine_gate_bwd(h.raw, s, rows, m, _dtype(dout), _ptr(dout), _ptr(gate), _ptr(y),
                                    _ptr(None if renorm else logits), int(renorm), _ptr(dY), _ptr(dgate),
                                    _ptr(dlogits), _stream(dout.device))
    _check(rc, "moe_combine_gate_bwd")
    return dY, dgate, dlogits


def moe_dispatch_bwd(h: Handle, dX: torch.Tensor, dx: torch.Tensor | None = None) -> torch.Tensor:
    """dX [rows,m] -> dx [s,m]."""
    rows, m = _rows2(dX, "dX")
    if dx is None:
        dx = torch.empty(h.s, m, dtype=dX.dtype, device=dX.device)
    s, mx = _rows2(dx, "dx")
    if mx != m or dx.dtype != dX.dtype:
        raise MoEError(1, "moe_dispatch_bwd", "dX and dx disagree in width or dtype")
    _check(lib().moe_dispatch_bwd(h.raw, s, rows, m, _dtype(dX), _ptr(dX), _ptr(dx), _stream(dX.device)),
           "moe_dispatch_bwd")
    return dx


# ---------------------------------------------------- expert parallelism --

def moe_ep_pack(h: Handle, gate: torch.Tensor, rows_sent: int, send_row: torch.Tensor | None = None,
                meta_idx: torch.Tensor | None = None, meta_gate: torch.Tensor | None = None):
    """The send map of a source handle (built with send slots over R ranks):
    (send_row i32 [s,R], meta_idx i32 [rows_sent,k], meta_gate f32 [rows_sent,k])."""
    dev = gate.device
    if gate.dtype != torch.float32 or tuple(gate.shape) != (h.s, h.k):
        raise MoEError(1, "moe_ep_pack", "gate must be float32 [s, k]")
    if send_row is None:
        send_row = torch.empty(h.s, h.R, dtype=torch.int32, device=dev)
    if meta_idx is None:
        meta_idx = torch.empty(rows_sent, h.k, dtype=torch.int32, device=dev)
    if meta_gate is None:
        meta_gate = torch.empty(rows_sent, h.k, dtype=torch.float32, device=dev)
    if tuple(send_row.shape) != (h.s, h.R) or tuple(meta_idx.shape) != (rows_sent, h.k) or \
            tuple(meta_gate.shape) != (rows_sent, h.k):
        raise MoEError(1, "moe_ep_pack", "output shapes")
    _check(lib().moe_ep_pack(h.raw, _ptr(gate), int(rows_sent), _ptr(send_row), _ptr(meta_idx), _ptr(meta_gate),
                             _stream(dev)), "moe_ep_pack")
    return send_row, meta_idx, meta_gate


def moe_ep_dispatch(h: Handle, send_row: torch.Tensor, rows_sent: int, x: torch.Tensor,
                    X_send: torch.Tensor | None = None) -> torch.Tensor:
    """The send buffer [rows_sent, m]: each token row once per destination rank."""
    s, m = _rows2(x, "x")
    if X_send is None:
        X_send = torch.empty(rows_sent, m, dtype=x.dtype, device=x.device)
    if tuple(X_send.shape) != (rows_sent, m) or X_send.dtype != x.dtype or s != h.s:
        raise MoEError(1, "moe_ep_dispatch", "shapes")
    _check(lib().moe_ep_dispatch(h.raw, _ptr(send_row), int(rows_sent), m, _dtype(x), _ptr(x), _ptr(X_send),
                                 _stream(x.device)), "moe_ep_dispatch")
    return X_send


def moe_ep_combine(h: Handle, send_row: torch.Tensor, rows_sent: int, P: torch.Tensor,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """out [s, m] = the returned partials P [rows_sent, m] summed over ranks in rank order."""
    rows, m = _rows2(P, "P")
    if rows != rows_sent:
        raise MoEError(1, "moe_ep_combine", "P must have rows_sent rows")
    if out is None:
        out = torch.empty(h.s, m, dtype=P.dtype, device=P.device)
    if tuple(out.shape) != (h.s, m) or out.dtype != P.dtype:
        raise MoEError(1, "moe_ep_combine", "output shape")
    _check(lib().moe_ep_combine(h.raw, _ptr(send_row), int(rows_sent), m, _dtype(P), _ptr(P), _ptr(out),
                                _stream(P.device)), "moe_ep_combine")
    return out


def moe_ep_unpack_dgate(h: Handle, send_row: torch.Tensor, rows_sent: int, dgate_back: torch.Tensor,
                        dgate: torch.Tensor | None = None) -> torch.Tensor:
    """dgate f32 [s, k] from the gate gradients returned per sent row [rows_sent, k]."""
    if tuple(dgate_back.shape) != (rows_sent, h.k) or dgate_back.dtype != torch.float32:
        raise MoEError(1, "moe_ep_unpack_dgate", "dgate_back must be float32 [rows_sent, k]")
    if dgate is None:
        dgate = torch.empty(h.s, h.k, dtype=torch.float32, device=dgate_back.device)
    _check(lib().moe_ep_unpack_dgate(h.raw, _ptr(send_row), int(rows_sent), _ptr(dgate_back), _ptr(dgate),
                                     _stream(dgate_back.device)), "moe_ep_unpack_dgate")
    return dgate


def moe_grouped_gemm(h: Handle, X: torch.Tensor, W: torch.Tensor, Y: torch.Tensor | None = None) -> torch.Tensor:
    """X bf16 [rows,K], W bf16 [e,N,K] -> Y bf16 [rows,N] per expert segment (tensor cores)."""
    rows, K = _rows2(X, "X")
    if W.dim() != 3 or W.shape[0] != h.e or W.shape[2] != K:
        raise MoEError(1, "moe_grouped_gemm", "W must be [e, N, K]")
    if X.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise MoEError(3, "moe_grouped_gemm", "X and W must be bf16")
    N = W.shape[1]
    if Y is None:
        Y = torch.empty(rows, N, dtype=torch.bfloat16, device=X.device)
    _check(lib().moe_grouped_gemm(h.raw, rows, K, N, _ptr(X), _ptr(W), _ptr(Y), _stream(X.device)),
           "moe_grouped_gemm")
    return Y


def moe_dispatch_grouped_gemm(h: Handle, x: torch.Tensor, W: torch.Tensor,
                              Y: torch.Tensor | None = None) -> torch.Tensor:
    """x bf16 [s,K], W bf16 [e,N,K] -> Y bf16 [rows,N]: the grouped GEMM on the
    token rows gathered through the handle, without a dispatched buffer."""
    s, K = _rows2(x, "x")
    if W.dim() != 3 or W.shape[0] != h.e or W.shape[2] != K:
        raise MoEError(1, "moe_dispatch_grouped_gemm", "W must be [e, N, K]")
    if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise MoEError(3, "moe_dispatch_grouped_gemm", "x and W must be bf16")
    N = W.shape[1]
    if Y is None:
        Y = torch.empty(h.rows, N, dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_dispatch_grouped_gemm(h.raw, s, h.rows, K, N, _ptr(x), _ptr(W), _ptr(Y),
                                           _stream(x.device)), "moe_dispatch_grouped_gemm")
    return Y


# ------------------------------------- layer norm, balance loss, products --
# Small calls are bound by the host, so these marshal with as few Python
# operations as they can; which device a pointer lives on is checked by the
# library alone.

_DTYPE = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}


def moe_layernorm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                  eps: float = 1e-5, y: torch.Tensor | None = None, stats: bool = True):
    """x [s,m] f32 or bf16 (rows may be strided), weight and bias [m] f32 or
    bf16 -> (y [s,m], mean f32 [s], rstd f32 [s]); stats=False returns y alone."""
    s, m = _rows2(x, "x")
    new, dt = _new(x), x.dtype
    wt = weight if weight is not None else bias
    for t in (weight, bias):
        if t is not None and (t.shape != (m,) or t.dtype != wt.dtype):
            raise MoEError(1, "moe_layernorm", "weight and bias must be [m], of one dtype")
    if y is None:
        y = new(dt, s, m)
    elif y.shape != (s, m) or y.dtype != dt:
        raise MoEError(1, "moe_layernorm", "output shape")
    mean = rstd = None
    if stats:
        mean = new(torch.float32, s)
        rstd = new(torch.float32, s)
    px, ldx = _rows_ptr(x)
    rc = lib().moe_layernorm(s, m, _DTYPE.get(dt, -1), px, ldx, 0 if wt is None else _DTYPE.get(wt.dtype, -1),
                             _addr(weight), _addr(bias), eps, _addr(y), _addr(mean), _addr(rstd), _raw_stream(x))
    if rc:
        _check(rc, "moe_layernorm")
    return (y, mean, rstd) if stats else y


def moe_layernorm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor,
                      rstd: torch.Tensor, dres: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                      need_dweight: bool = True, need_dbias: bool = True):
    """(dy, x [s,m], weight [m] or None, mean, rstd f32 [s]) -> (dx [s,m],
    dweight f32 [m] or None, dbias f32 [m] or None).  dres [s,m]: a gradient
    that reaches x past the norm (the residual branch), added to dx."""
    s, m = _rows2(x, "x")
    new, dt = _new(x), x.dtype
    for t in (dy, dres, dx):
        if t is not None and (t.shape != (s, m) or t.dtype != dt):
            raise MoEError(1, "moe_layernorm_bwd", "dy, dres and dx must have x's shape and dtype")
    if mean.shape != (s,) or rstd.shape != (s,) or mean.dtype != torch.float32 or rstd.dtype != torch.float32:
        raise MoEError(1, "moe_layernorm_bwd", "mean and rstd must be float32 [s]")
    if weight is not None and weight.shape != (m,):
        raise MoEError(1, "moe_layernorm_bwd", "weight must be [m]")
    if dx is None:
        dx = new(dt, s, m)
    dw = new(torch.float32, m) if need_dweight else None
    db = new(torch.float32, m) if need_dbias else None
    L, nbytes, ws = lib(), 0, None
    if need_dweight or need_dbias:
        nbytes = L.moe_layernorm_bwd_workspace(s, m)
        ws = new(torch.uint8, nbytes)
    pdy, lddy = _rows_ptr(dy)
    px, ldx = _rows_ptr(x)
    pres, ldres = _rows_ptr(dres)
    rc = L.moe_layernorm_bwd(s, m, _DTYPE.get(dt, -1), pdy, lddy, px, ldx,
                             0 if weight is None else _DTYPE.get(weight.dtype, -1), _addr(weight), _addr(mean),
                             _addr(rstd), pres, ldres, _addr(dx), _addr(dw), _addr(db), _addr(ws), nbytes,
                             _raw_stream(x))
    if rc:
        _check(rc, "moe_layernorm_bwd")
    return dx, dw, db


class BalanceLoss(NamedTuple):
    """What moe_balance_loss returns; lse, coef and norm feed its backward pass."""
    loss: torch.Tensor       # f32 [2]: the balance loss, the z loss
    counts: torch.Tensor     # i32 [num_seqs, e]: valid routes per expert
    mean_prob: torch.Tensor  # f32 [num_seqs, e]: mean router probability
    lse: torch.Tensor        # f32 [s]
    coef: torch.Tensor       # f32 [num_seqs, e]
    norm: torch.Tensor       # f32 [2]


def _check_balance(where: str, s: int, logits, valid, seq_offsets) -> int:
    if logits.dtype != torch.float32:
        raise MoEError(3, where, "logits must be float32")
    if valid is not None and (valid.shape != (s,) or valid.dtype not in (torch.uint8, torch.bool)):
        raise MoEError(1, where, "valid must be uint8 or bool [s]")
    if seq_offsets is None:
        return 1
    if seq_offsets.dim() != 1 or seq_offsets.dtype != torch.int32 or seq_offsets.numel() < 2:
        raise MoEError(1, where, "seq_offsets must be int32 [num_seqs + 1]")
    return seq_offsets.numel() - 1


def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, valid: torch.Tensor | None = None,
                     seq_offsets: torch.Tensor | None = None, device_status: torch.Tensor | None = None) -> BalanceLoss:
    """logits f32 [s,e], topk_idx i32 [s,k] (-1: absent), valid u8/bool [s]
    (padding is 0), seq_offsets i32 [num_seqs+1] -> BalanceLoss."""
    s, e = _rows2(logits, "logits")
    if topk_idx.dim() != 2 or topk_idx.dtype != torch.int32 or topk_idx.shape[0] != s:
        raise MoEError(1, "moe_balance_loss", "topk_idx must be int32 [s, k]")
    n = _check_balance("moe_balance_loss", s, logits, valid, seq_offsets)
    new, f32, L = _new(logits), torch.float32, lib()
    loss = new(f32, 2)
    counts = new(torch.int32, n, e)
    mean_prob = new(f32, n, e)
    lse = new(f32, s)
    coef = new(f32, n, e)
    norm = new(f32, 2)
    nbytes = L.moe_balance_loss_workspace(e, n)
    ws = new(torch.uint8, nbytes)
    rc = L.moe_balance_loss(_addr(logits), _addr(topk_idx), _addr(valid), _addr(seq_offsets), s, e, topk_idx.shape[1],
                            n, loss.data_ptr(), counts.data_ptr(), mean_prob.data_ptr(), lse.data_ptr(),
                            coef.data_ptr(), norm.data_ptr(), ws.data_ptr(), nbytes,
                            _status_addr(device_status, "moe_balance_loss"), _raw_stream(logits))
    if rc:
        _check(rc, "moe_balance_loss")
    return BalanceLoss(loss, counts, mean_prob, lse, coef, norm)


def moe_balance_loss_bwd(logits: torch.Tensor, lse: torch.Tensor, coef: torch.Tensor, norm: torch.Tensor,
                         dloss: torch.Tensor, valid: torch.Tensor | None = None,
                         seq_offsets: torch.Tensor | None = None, add: torch.Tensor | None = None,
                         dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """dloss f32 [2] (the gradients reaching the two losses) -> dlogits f32
    [s,e], plus add [s,e] (may be dlogits itself) where given."""
    s, e = _rows2(logits, "logits")
    n = _check_balance("moe_balance_loss_bwd", s, logits, valid, seq_offsets)
    f32 = torch.float32
    for t, name, shape in ((lse, "lse", (s,)), (coef, "coef", (n, e)), (norm, "norm", (2,)), (dloss, "dloss", (2,)),
                           (add, "add", (s, e)), (dlogits, "dlogits", (s, e))):
        if t is not None and (t.shape != shape or t.dtype != f32):
            raise MoEError(1, "moe_balance_loss_bwd", f"{name} must be float32 {list(shape)}")
    if dlogits is None:
        dlogits = _new(logits)(f32, s, e)
    rc = lib().moe_balance_loss_bwd(_addr(logits), _addr(lse), _addr(coef), _addr(norm), _addr(dloss), _addr(valid),
                                    _addr(seq_offsets), _addr(add), s, e, n, _addr(dlogits), _raw_stream(logits))
    if rc:
        _check(rc, "moe_balance_loss_bwd")
    return dlogits


def _check_linear(where: str, x: torch.Tensor, W: torch.Tensor, act: str):
    s, K = _rows2(x, "x")
    N, KW = _rows2(W, "W")
    if KW != K:
        raise MoEError(1, where, "W must be [N, K]")
    if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise MoEError(3, where, "x and W must be bf16")
    if act not in ACT:
        raise MoEError(1, where, f"act must be one of {', '.join(ACT)}")
    return s, K, N


def moe_linear(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
               residual: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, save_z: bool = False,
               y: torch.Tensor | None = None, device_status: torch.Tensor | None = None):
    """y [s,N] = act(x W^T + bias) + residual on the tensor cores: x bf16
    [s,K], W bf16 [N,K] (rows may be strided; K a multiple of 8), bias [N] and
    residual [s,N] f32 or bf16, y f32 or bf16 (default bf16); act: none, relu,
    gelu, gelu_tanh, silu.  save_z: return (y, z), z bf16 [s,N] the value
    before the activation, for moe_linear_bwd."""
    s, K, N = _check_linear("moe_linear", x, W, act)
    new = _new(x)
    if bias is not None and bias.shape != (N,):
        raise MoEError(1, "moe_linear", "bias must be [N]")
    if residual is not None and residual.shape != (s, N):
        raise MoEError(1, "moe_linear", "residual must be [s, N]")
    if y is None:
        y = new(torch.bfloat16 if out_dtype is None else out_dtype, s, N)
    elif y.shape != (s, N) or (out_dtype is not None and y.dtype != out_dtype):
        raise MoEError(1, "moe_linear", "output shape or dtype")
    z = new(torch.bfloat16, s, N) if save_z else None
    px, ldx = _rows_ptr(x)
    pw, ldw = _rows_ptr(W)
    pres, ldres = _rows_ptr(residual)
    d = LinearDesc(s, K, N, ACT[act], _DTYPE.get(y.dtype, -1), 0 if bias is None else _DTYPE.get(bias.dtype, -1),
                   0 if residual is None else _DTYPE.get(residual.dtype, -1), ldx, ldw, ldres)
    rc = lib().moe_linear(d, px, pw, _addr(bias), pres, _addr(y), _addr(z),
                          _status_addr(device_status, "moe_linear"), _raw_stream(x))
    if rc:
        _check(rc, "moe_linear")
    return (y, z) if save_z else y


def moe_linear_bwd(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor, z: torch.Tensor | None = None,
                   act: str = "none", need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
                   dx_dtype: torch.dtype = torch.bfloat16, dw_dtype: torch.dtype = torch.bfloat16,
                   device_status: torch.Tensor | None = None):
    """(dy [s,N] f32 or bf16, x bf16 [s,K], W bf16 [N,K], z bf16 [s,N] with an
    activation) -> (dx [s,K], dW [N,K], db f32 [N]), None for those not
    needed.  The residual's gradient is dy itself."""
    s, K, N = _check_linear("moe_linear_bwd", x, W, act)
    new = _new(x)
    if dy.shape != (s, N):
        raise MoEError(1, "moe_linear_bwd", "dy must be [s, N]")
    if act == "none":
        z = None
    elif z is None or z.shape != (s, N) or z.dtype != torch.bfloat16:
        raise MoEError(1, "moe_linear_bwd", "z must be bf16 [s, N] with an activation")
    dx = new(dx_dtype, s, K) if need_dx else None
    dW = new(dw_dtype, N, K) if need_dw else None
    db = new(torch.float32, N) if need_db else None
    L = lib()
    pdy, lddy = _rows_ptr(dy)
    px, ldx = _rows_ptr(x)
    pw, ldw = _rows_ptr(W)
    pz, ldz = _rows_ptr(z)
    d = LinearBwdDesc(s, K, N, ACT[act], _DTYPE.get(dy.dtype, -1), _DTYPE.get(dx_dtype, -1), _DTYPE.get(dw_dtype, -1),
                      lddy, ldx, ldw, ldz)
    nbytes = L.moe_linear_bwd_workspace_for(d, need_dx, need_dw, need_db)
    ws = new(torch.uint8, nbytes) if nbytes else None
    rc = L.moe_linear_bwd(d, pdy, px, pw, pz, _addr(dx), _addr(dW), _addr(db), _addr(ws), nbytes,
                          _status_addr(device_status, "moe_linear_bwd"), _raw_stream(x))
    if rc:
        _check(rc, "moe_linear_bwd")
    return dx, dW, db


# ------------------------- gated experts: products, gradients, clipping --

def _check_gated(where: str, x: torch.Tensor, W: torch.Tensor, act: str):
    s, K = _rows2(x, "x")
    N2, KW = _rows2(W, "W")
    if KW != K or N2 % 2:
        raise MoEError(1, where, "W must be [2N, K], the gate's rows first")
    if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise MoEError(3, where, "x and W must be bf16")
    if act not in ACT:
        raise MoEError(1, where, f"act must be one of {', '.join(ACT)}")
    return s, K, N2 // 2


def moe_gated_linear(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: str = "silu",
                     save_z: bool = False, h: torch.Tensor | None = None, device_status: torch.Tensor | None = None):
    """h bf16 [s,N] = act(x Wg^T + bg) * (x Wu^T + bu): x bf16 [s,K], W bf16
    [2N,K] = [Wg; Wu] (rows may be strided; K and N multiples of 8), bias [2N]
    f32 or bf16.  save_z: return (h, z), z bf16 [s,2N] both projections, for
    moe_gated_linear_bwd."""
    s, K, N = _check_gated("moe_gated_linear", x, W, act)
    new = _new(x)
    if bias is not None and bias.shape != (2 * N,):
        raise MoEError(1, "moe_gated_linear", "bias must be [2N]")
    if h is None:
        h = new(torch.bfloat16, s, N)
    elif h.shape != (s, N) or h.dtype != torch.bfloat16:
        raise MoEError(1, "moe_gated_linear", "h must be bf16 [s, N]")
    z = new(torch.bfloat16, s, 2 * N) if save_z else None
    px, ldx = _rows_ptr(x)
    pw, ldw = _rows_ptr(W)
    d = GatedDesc(s, K, N, ACT[act], 0 if bias is None else _DTYPE.get(bias.dtype, -1), ldx, ldw)
    rc = lib().moe_gated_linear(d, px, pw, _addr(bias), _addr(h), _addr(z),
                                _status_addr(device_status, "moe_gated_linear"), _raw_stream(x))
    if rc:
        _check(rc, "moe_gated_linear")
    return (h, z) if save_z else h


def moe_gated_linear_bwd(dh: torch.Tensor, x: torch.Tensor, W: torch.Tensor, z: torch.Tensor, act: str = "silu",
                         need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
                         dx_dtype: torch.dtype = torch.bfloat16, dw_dtype: torch.dtype = torch.bfloat16,
                         device_status: torch.Tensor | None = None):
    """(dh [s,N] f32 or bf16, x bf16 [s,K], W bf16 [2N,K], z bf16 [s,2N]) ->
    (dx [s,K], dW [2N,K], db f32 [2N]), None for those not needed."""
    s, K, N = _check_gated("moe_gated_linear_bwd", x, W, act)
    new = _new(x)
    if dh.shape != (s, N):
        raise MoEError(1, "moe_gated_linear_bwd", "dh must be [s, N]")
    if z.shape != (s, 2 * N) or z.dtype != torch.bfloat16:
        raise MoEError(1, "moe_gated_linear_bwd", "z must be bf16 [s, 2N]")
    dx = new(dx_dtype, s, K) if need_dx else None
    dW = new(dw_dtype, 2 * N, K) if need_dw else None
    db = new(torch.float32, 2 * N) if need_db else None
    L = lib()
    pdh, lddh = _rows_ptr(dh)
    px, ldx = _rows_ptr(x)
    pw, ldw = _rows_ptr(W)
    pz, ldz = _rows_ptr(z)
    d = GatedBwdDesc(s, K, N, ACT[act], _DTYPE.get(dh.dtype, -1), _DTYPE.get(dx_dtype, -1), _DTYPE.get(dw_dtype, -1),
                     lddh, ldx, ldw, ldz)
    nbytes = L.moe_gated_linear_bwd_workspace(d, need_dx, need_dw, need_db)
    ws = new(torch.uint8, nbytes) if nbytes else None
    rc = L.moe_gated_linear_bwd(d, pdh, px, pw, pz, _addr(dx), _addr(dW), _addr(db), _addr(ws), nbytes,
                                _status_addr(device_status, "moe_gated_linear_bwd"), _raw_stream(x))
    if rc:
        _check(rc, "moe_gated_linear_bwd")
    return dx, dW, db


def _check_experts(where: str, h: Handle, x: torch.Tensor | None, W: torch.Tensor, gated: bool, act: str = "none"):
    """(rows of x, K, N) of an expert product's operands; without x the handle's rows."""
    s, K = _rows2(x, "x") if x is not None else (h.rows, W.shape[-1])
    if W.dim() != 3 or W.shape[0] != h.e or W.shape[2] != K or (gated and W.shape[1] % 2):
        raise MoEError(1, where, "W must be [e, 2N, K], the gate's rows first" if gated else "W must be [e, N, K]")
    if (x is not None and x.dtype != torch.bfloat16) or W.dtype != torch.bfloat16:
        raise MoEError(3, where, "x and W must be bf16")
    if act not in ACT:
        raise MoEError(1, where, f"act must be one of {', '.join(ACT)}")
    return s, K, W.shape[1] // 2 if gated else W.shape[1]


def _bf16(where: str, t: torch.Tensor | None, name: str, *shape):
    if t is not None and (t.shape != shape or t.dtype != torch.bfloat16):
        raise MoEError(1, where, f"{name} must be bf16 {list(shape)}")


def _gated_rows(where: str, call, h: Handle, x, W, act, H, Z, save_z, gather: bool):
    s, K, N = _check_experts(where, h, x, W, True, act)
    new, rows = _new(x), h.rows
    if s != (h.s if gather else rows):
        raise MoEError(4, where, "x has another number of rows than the handle's")
    _bf16(where, H, "H", rows, N)
    _bf16(where, Z, "Z", rows, 2 * N)
    if H is None:
        H = new(torch.bfloat16, rows, N)
    if not save_z:
        Z = None
    elif Z is None:
        Z = new(torch.bfloat16, rows, 2 * N)
    sizes = (s, rows, K, N) if gather else (rows, K, N)
    rc = call(h.raw, *sizes, ACT[act], _addr(x), _addr(W), _addr(H), _addr(Z), _raw_stream(x))
    if rc:
        _check(rc, where)
    return (H, Z) if save_z else H


def moe_grouped_gated(h: Handle, X: torch.Tensor, W: torch.Tensor, act: str = "silu", save_z: bool = False,
                      H: torch.Tensor | None = None, Z: torch.Tensor | None = None):
    """X bf16 [rows,K], W bf16 [e,2N,K] (each expert's gate rows first) -> H
    bf16 [rows,N] = act(X Wg[x]^T) * (X Wu[x]^T) per expert segment; save_z:
    (H, Z), Z bf16 [rows,2N] for moe_grouped_gated_bwd.  Rows no route owns
    are not written."""
    return _gated_rows("moe_grouped_gated", lib().moe_grouped_gated, h, X, W, act, H, Z, save_z, False)


def moe_dispatch_grouped_gated(h: Handle, x: torch.Tensor, W: torch.Tensor, act: str = "silu", save_z: bool = False,
                               H: torch.Tensor | None = None, Z: torch.Tensor | None = None):
    """The same on the token rows x bf16 [s,K] gathered through the handle, without a dispatched buffer."""
    return _gated_rows("moe_dispatch_grouped_gated", lib().moe_dispatch_grouped_gated, h, x, W, act, H, Z, save_z, True)


def _grouped_bwd_args(where: str, h: Handle, D, X, W, need_dx, need_dw, dX, dW, gated: bool, act: str = "none"):
    if X is None and need_dw:
        raise MoEError(1, where, "dW needs X")
    rows, K, N = _check_experts(where, h, X, W, gated, act)
    _bf16(where, D, "the result's gradient", rows, N)
    _bf16(where, dX, "dX", rows, K)
    _bf16(where, dW, "dW", *W.shape)
    new = _new(W)
    if dX is None and need_dx:
        dX = new(torch.bfloat16, rows, K)
    if dW is None and need_dw:
        dW = new(torch.bfloat16, W.shape[0] * W.shape[1], K).view(W.shape)
    return rows, K, N, dX if need_dx else None, dW if need_dw else None


def moe_grouped_gemm_bwd(h: Handle, dY: torch.Tensor, X: torch.Tensor | None, W: torch.Tensor, need_dx: bool = True,
                         need_dw: bool = True, dX: torch.Tensor | None = None, dW: torch.Tensor | None = None):
    """Backward of moe_grouped_gemm: (dY bf16 [rows,N], X bf16 [rows,K], W bf16
    [e,N,K]) -> (dX [rows,K], dW [e,N,K]), None for those not needed.  Rows of
    dX that no route owns are not written.  X may be None without dW."""
    rows, K, N, dX, dW = _grouped_bwd_args("moe_grouped_gemm_bwd", h, dY, X, W, need_dx, need_dw, dX, dW, False)
    rc = lib().moe_grouped_gemm_bwd(h.raw, rows, K, N, _addr(dY), _addr(X), _addr(W), _addr(dX), _addr(dW), _raw_stream(W))
    if rc:
        _check(rc, "moe_grouped_gemm_bwd")
    return dX, dW


def moe_grouped_gated_bwd(h: Handle, dH: torch.Tensor, X: torch.Tensor | None, W: torch.Tensor, Z: torch.Tensor,
                          act: str = "silu", need_dx: bool = True, need_dw: bool = True,
                          dX: torch.Tensor | None = None, dW: torch.Tensor | None = None):
    """Backward of moe_grouped_gated (X = moe_dispatch's output also for the
    gathering form): (dH bf16 [rows,N], X bf16 [rows,K], W bf16 [e,2N,K], Z bf16
    [rows,2N]) -> (dX [rows,K], dW [e,2N,K]), None for those not needed.  X may
    be None without dW."""
    where = "moe_grouped_gated_bwd"
    rows, K, N, dX, dW = _grouped_bwd_args(where, h, dH, X, W, need_dx, need_dw, dX, dW, True, act)
    _bf16(where, Z, "Z", rows, 2 * N)
    L = lib()
    nbytes = L.moe_grouped_gated_bwd_workspace(rows, N) if need_dx or need_dw else 0
    ws = _new(W)(torch.uint8, nbytes) if nbytes else None
    rc = L.moe_grouped_gated_bwd(h.raw, rows, K, N, ACT[act], _addr(dH), _addr(X), _addr(W), _addr(Z), _addr(dX), _addr(dW),
                                 _addr(ws), nbytes, _raw_stream(W))
    if rc:
        _check(rc, where)
    return dX, dW


class GradList:
    """Tensors whose norm is taken and which are clipped together, checked once:
    f32 or bf16 on one device, each without gaps or overlaps in memory (any
    order of its axes).  It keeps the tensors alive; a program whose gradients
    stay in place makes it once."""

    def __init__(self, tensors):
        self.tensors = tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
        self.device = tensors[0].device if tensors else None
        self.ordered = True  # every tensor's elements are in the order of its axes
        flat = []
        for i, t in enumerate(tensors):
            if t.layout != torch.strided or not t.is_contiguous():
                if t.layout != torch.strided or not _dense(t):
                    raise ValueError(f"tensor {i}: gradients must be dense tensors without gaps or overlaps in memory")
                self.ordered = False
            if t.device != self.device:
                raise MoEError(1, "GradList", "the tensors are on different devices")
            flat += (t.data_ptr(), t.numel(), _DTYPE.get(t.dtype, -1))
        spec = (Tensor * max(1, len(tensors))).from_buffer_copy(struct.pack("=" + "Qqi4x" * len(tensors), *flat) if flat else
                                                                bytes(ctypes.sizeof(Tensor)))
        self.workspace = lib().moe_grad_norm_workspace(len(tensors))
        self._raw = raw = ctypes.c_void_p()
        if self.device is not None and self.device.type == "cuda":
            with torch.cuda.device(self.device):
                rc = lib().moe_tensor_list_create(spec, len(tensors), ctypes.byref(raw))
        else:  # no tensors, or host tensors, which the library rejects
            rc = lib().moe_tensor_list_create(spec, len(tensors), ctypes.byref(raw))
        if rc:
            _check(rc, "moe_tensor_list_create")
        if self.device is None:
            self.device = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else None

    def __len__(self):
        return len(self.tensors)

    @property
    def raw(self):
        return self._raw

    def __del__(self):
        raw = getattr(self, "_raw", None)
        if raw and _lib is not None:
            _lib.moe_tensor_list_destroy(raw)


def _dense(t: torch.Tensor) -> bool:
    """The elements fill a stretch of memory, in some order of the axes."""
    if t.numel() == 0:
        return True
    expect = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
        if stride != expect:
            return False
        expect *= size
    return True


def _grads(grads) -> GradList:
    return grads if isinstance(grads, GradList) else GradList(grads)


def _clip_lists(where: str, grads, out):
    g = _grads(grads)
    o = None if out is None else _grads(out)
    if o is not None and not (g.ordered and o.ordered):  # the library compares sizes
        for a, b in zip(g.tensors, o.tensors):
            if a.shape != b.shape or a.stride() != b.stride():
                raise MoEError(1, where, "out must have the gradients' shapes and strides")
    return g, o


def _check_norm(where: str, norm: torch.Tensor):
    if norm.shape != (1,) or norm.dtype != torch.float32:
        raise MoEError(1, where, "norm must be float32 [1]")


def _norm_call(where: str, g: GradList, norm, device_status, call):
    """call(norm, workspace, its bytes, status, stream) on the list's device."""
    if g.device is None:
        raise RuntimeError("no CUDA device")
    if g.device.type == "cuda" and g.device.index != torch.cuda.current_device():
        with torch.cuda.device(g.device):
            return _norm_call(where, g, norm, device_status, call)
    new = _new_here if _strided is not None and not _modes() else \
        lambda dtype, n: torch.empty(n, dtype=dtype, device=g.device)
    if norm is None:
        norm = new(torch.float32, 1)
    else:
        _check_norm(where, norm)
    ws = new(torch.uint8, g.workspace)
    rc = call(_addr(norm), ws.data_ptr(), g.workspace, _status_addr(device_status, where), _raw_stream(norm))
    if rc:
        _check(rc, where)
    return norm


def moe_grad_norm(grads, norm: torch.Tensor | None = None, device_status: torch.Tensor | None = None) -> torch.Tensor:
    """f32 [1]: the 2-norm of all elements of all tensors (a sequence or a
    GradList).  A NaN or an infinity reaches it (and device_status)."""
    g = _grads(grads)
    return _norm_call("moe_grad_norm", g, norm, device_status, lambda *a: lib().moe_grad_norm(g.raw, *a))


def moe_grad_clip(grads, norm: torch.Tensor, max_norm: float, out=None):
    """Scale the gradients by min(1, max_norm / (norm + 1e-6)) in place, or into the tensors of `out`; norm f32 [1] on
    the device (joined over ranks, say).  A norm that is not finite leaves them unscaled."""
    g, o = _clip_lists("moe_grad_clip", grads, out)
    _check_norm("moe_grad_clip", norm)
    with torch.cuda.device(g.device):
        rc = lib().moe_grad_clip(g.raw, None if o is None else o.raw, _addr(norm), max_norm, _raw_stream(norm))
    if rc:
        _check(rc, "moe_grad_clip")


def moe_clip_grad_norm(grads, max_norm: float, out=None, norm: torch.Tensor | None = None,
                       device_status: torch.Tensor | None = None) -> torch.Tensor:
    """moe_grad_norm and moe_grad_clip in two kernels at most; returns the norm before clipping, f32 [1]."""
    g, o = _clip_lists("moe_clip_grad_norm", grads, out)
    ro = None if o is None else o.raw
    return _norm_call("moe_clip_grad_norm", g, norm, device_status,
                      lambda *a: lib().moe_clip_grad_norm(g.raw, ro, max_norm, *a))
