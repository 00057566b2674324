"""Gated DeltaNet layer for AMD MI355X (gfx950): Python binding of libgdn.so.

This module only marshals arguments: it checks tensor shapes, dtypes and
devices on the host (so that no kernel is launched on buffers smaller than
its grid assumes), then passes raw device pointers and the current HIP stream
to the C ABI declared in include/gdn.h.  Every step of the layer runs in the
library's HIP kernels; there is no fallback.  If libgdn.so has not been built
the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32 = 0
GDN_BF16 = 1
GDN_FLAG_L2NORM_QK = 1
POS_ONE = 65536
POS_STRIDE = 32  # int32 words per slot in conv_pos: slot s's position is conv_pos[s, 0]
CHUNK = 64

ABI_VERSION = 9  # GDN_ABI_VERSION of include/gdn.h that these signatures follow
DEV_OK = 0
DEV_BAD_SLOT = 1
DEV_BAD_ACCEPTED = 2
DEV_BAD_SEQLENS = 3
DEV_WAIT_TIMEOUT = 4
DEV_BAD_K = 5
DEV_INCOMPLETE = 6
DEV_DUP_SLOT = 7  # libgdn_debug.so only
DEV_BAD_PAGE = 8
DEV_NO_PAGES = 9
DEV_BAD_LENGTH = 10
DEV_BAD_PARENT = 11


class GdnGeometry(ctypes.Structure):
    _fields_ = [
        ("n_k_heads", ctypes.c_int32),
        ("n_v_heads", ctypes.c_int32),
        ("d_k", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("conv_width", ctypes.c_int32),
        ("conv_channels", ctypes.c_int32),
        ("conv_ring", ctypes.c_int32),
        ("max_draft", ctypes.c_int32),
        ("n_slots", ctypes.c_int32),
        ("dtype_in", ctypes.c_int32),
        ("dtype_out", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("q_scale", ctypes.c_float),
        ("l2_eps", ctypes.c_float),
    ]


class GdnAttnGeometry(ctypes.Structure):
    _fields_ = [
        ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("d_head", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("max_tree", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class GdnError(RuntimeError):
    def __init__(self, status: int, name: str, message: str):
        super().__init__(f"{name}: {message}")
        self.status = status
        self.name = name
        self.message = message


_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_Z = ctypes.c_size_t
_SIGS = {
    "gdn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "gdn_last_error": (ctypes.c_char_p, []),
    "gdn_version": (ctypes.c_char_p, []),
    "gdn_abi_version": (ctypes.c_int32, []),
    "gdn_check_geometry": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), ctypes.c_char_p, ctypes.c_size_t]),
    "gdn_prefill_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(GdnGeometry), _I, _I]),
    "gdn_conv_state_step": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _I, _P, _P, _P]),
    "gdn_decode_step": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _P, _P, _P, _I,
                                       _P, _P, _P]),
    "gdn_prefill_chunked": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                           _P, _I, _I, _I, _P, ctypes.c_size_t, _P, _P, _P]),
    "gdn_prefill_chunked_ckpt": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _P, _P, _P,
                                                _P, _P, _I, _I, _I, _P, ctypes.c_size_t, _P, _I, _P,
                                                ctypes.c_size_t, _P, _P]),
    "gdn_prefill_chunked_static": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _P, _P, _P,
                                                  _P, _P, _I, _I, _I, _P, _P, _P]),
    "gdn_verify_k": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _P, _P, _P, _I, _I,
                                    _P, _P, _P, _P]),
    "gdn_rollback": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _I, _I, _P, _P]),
    "gdn_verify_k_slots": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _P, _P, _P, _P, _I, _I,
                                          _P, _P, _P, _P, _P]),
    "gdn_commit_slots": (ctypes.c_int, [ctypes.POINTER(GdnGeometry), _P, _P, _P, _P, _I, _I, _P, _P, _P]),
    "gdn_prefill_timing_events": (ctypes.c_int, [_P, _P]),
    "gdn_verify_tree_slots": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P]),
    "gdn_check_attn_geometry": (ctypes.c_int, [_P, ctypes.c_char_p, _Z]),
    "gdn_kv_plan": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "gdn_kv_write": (ctypes.c_int, [_P, _P, _P, _P, _L, _P, _L, _P, _I, _P, _P]),
    "gdn_attn_prefill": (ctypes.c_int, [_P, _P, _L, _P, _L, _P, _L, _P, _I, _I, _P, _P, _P, _P, _P, _Z, _P, _P, _P]),
    "gdn_attn_prefill_workspace_bytes": (_Z, [_P, _I, _I]),
    "gdn_attn_prefill_workspace_max_bytes": (_Z, [_P, _I, _I]),
    "gdn_attn_tree": (ctypes.c_int, [_P, _P, _L, _P, _L, _P, _L, _P, _P, _I, _I, _P, _P, _P, _P, _P, _Z, _P, _P, _P]),
    "gdn_attn_tree_workspace_bytes": (_Z, [_P, _I, _I]),
    "gdn_attn_tree_workspace_max_bytes": (_Z, [_P, _I, _I]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                               "or python -m gated_deltanet_delta_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        if L.gdn_abi_version() != ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI version {L.gdn_abi_version()}, this binding needs "
                               f"{ABI_VERSION}; rebuild it with __graft_entry__.build()")
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        L = lib()
        raise GdnError(status, L.gdn_status_string(status).decode(), L.gdn_last_error().decode())


# --------------------------------------------------------------------------
# geometry
# --------------------------------------------------------------------------

@dataclass(frozen=True)
class Geometry:
    """Python mirror of gdn_geometry (see include/gdn.h for every field)."""

    n_k_heads: int = 16
    n_v_heads: int = 48
    d_k: int = 128
    d_v: int = 128
    conv_width: int = 4
    conv_ring: int = 8
    max_draft: int = 4
    n_slots: int = 8
    dtype: torch.dtype = torch.bfloat16
    l2norm_qk: bool = True
    q_scale: float = 1.0
    l2_eps: float = 1e-6

    @property
    def conv_channels(self) -> int:
        return 2 * self.n_k_heads * self.d_k + self.n_v_heads * self.d_v

    def c_struct(self) -> GdnGeometry:
        code = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}[self.dtype]
        return GdnGeometry(self.n_k_heads, self.n_v_heads, self.d_k, self.d_v, self.conv_width,
                           self.conv_channels, self.conv_ring, self.max_draft, self.n_slots, code, code,
                           GDN_FLAG_L2NORM_QK if self.l2norm_qk else 0, self.q_scale, self.l2_eps)

    def check(self):
        g = self.c_struct()
        _check(lib().gdn_check_geometry(ctypes.byref(g), None, 0))


# --------------------------------------------------------------------------
# host-side marshalling helpers
# --------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        return ctypes.c_void_p(_current_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


# the current stream's handle without a Stream object around it (0.1 us instead of 1.3), where torch has it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda device: torch.cuda.current_stream(device).cuda_stream)


def _index(t: torch.Tensor) -> Optional[int]:
    """The GPU that a call's tensors are to be on, that of its first one (None: it is not on a GPU, which _need refuses)."""
    return t.get_device() if t.is_cuda else None


def _here(device: int, stream) -> ctypes.c_void_p:
    """The stream of a call whose tensors are on `device`, which has to be the current one (the call launches there)."""
    cur = torch.cuda.current_device()
    if device != cur:
        raise ValueError(f"tensors on cuda:{device}, required: the current device cuda:{cur}")
    if stream is None:
        return ctypes.c_void_p(_current_stream(cur))
    if getattr(stream, "device_index", cur) != cur:
        raise ValueError(f"stream: of cuda:{stream.device_index}, required: of the current device cuda:{cur}")
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: Optional[torch.Tensor], name: str, shape, dtype, optional=False, device: Optional[int] = None):
    if (t is not None and (t.is_cuda if device is None else t.get_device() == device) and t.dtype == dtype
            and t.shape == shape and t.is_contiguous()):
        return
    if t is None:
        if optional:
            return
        raise ValueError(f"{name}: missing")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, required {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, required {tuple(shape)}")
    _need_device(t, name, device)


def _need_device(t: torch.Tensor, name: str, device: Optional[int]):
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, required: cuda:{device}, as the call's other tensors")


@dataclass
class SlotPool:
    """Caller-owned device buffers of one layer's slot pool."""

    state: torch.Tensor       # fp32 [n_slots][H_v][d_v][d_k]
    conv_state: torch.Tensor  # fp32 [n_slots][R][C]
    conv_pos: torch.Tensor    # int32 [n_slots][POS_STRIDE], position in column 0, units of 1/65536 token

    @staticmethod
    def zeros(geom: Geometry, device="cuda") -> "SlotPool":
        C, R = geom.conv_channels, max(geom.conv_ring, 1)
        return SlotPool(
            torch.zeros(geom.n_slots, geom.n_v_heads, geom.d_v, geom.d_k, dtype=torch.float32, device=device),
            torch.zeros(geom.n_slots, R, C, dtype=torch.float32, device=device),
            torch.zeros(geom.n_slots, POS_STRIDE, dtype=torch.int32, device=device))


def _check_pool(geom: Geometry, pool: SlotPool, device: Optional[int] = None):
    _need(pool.state, "state", (geom.n_slots, geom.n_v_heads, geom.d_v, geom.d_k), torch.float32, device=device)
    if geom.conv_width > 0:
        _need(pool.conv_state, "conv_state", (geom.n_slots, geom.conv_ring, geom.conv_channels), torch.float32, device=device)
        _need(pool.conv_pos, "conv_pos", (geom.n_slots, POS_STRIDE), torch.int32, device=device)


# --------------------------------------------------------------------------
# the five entry points
# --------------------------------------------------------------------------

def conv_state_step(geom: Geometry, pool: SlotPool, x, conv_w, slot, y, dev_err=None, stream=None):
    """gdn_conv_state_step: y = SiLU(causal conv) for all channels; append x to the ring."""
    B = slot.shape[0]
    C = geom.conv_channels
    _check_pool(geom, pool)
    _need(x, "x", (B, C), geom.dtype)
    _need(conv_w, "conv_w", (C, geom.conv_width), torch.float32)
    _need(slot, "slot", (B,), torch.int32)
    _need(y, "y", (B, C), geom.dtype)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    g = geom.c_struct()
    _check(lib().gdn_conv_state_step(ctypes.byref(g), _ptr(pool.conv_state), _ptr(pool.conv_pos), _ptr(x),
                                     _ptr(conv_w), _ptr(slot), B, _ptr(y), _ptr(dev_err), _stream(stream)))


def decode_step(geom: Geometry, pool: SlotPool, x, a, b, conv_w, slot, o, dev_err=None, stream=None):
    """gdn_decode_step: one fused token per batch row; state updated in place."""
    B = slot.shape[0]
    C, Hv, dv = geom.conv_channels, geom.n_v_heads, geom.d_v
    _check_pool(geom, pool)
    _need(x, "x", (B, C), geom.dtype)
    _need(a, "a", (B, Hv), geom.dtype)
    _need(b, "b", (B, Hv), geom.dtype)
    _need(conv_w, "conv_w", (C, geom.conv_width), torch.float32, optional=geom.conv_width == 0)
    _need(slot, "slot", (B,), torch.int32)
    _need(o, "o", (B, Hv, dv), geom.dtype)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    g = geom.c_struct()
    _check(lib().gdn_decode_step(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_state), _ptr(pool.conv_pos),
                                 _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w), _ptr(slot), B, _ptr(o),
                                 _ptr(dev_err), _stream(stream)))


def verify_k(geom: Geometry, pool: SlotPool, x, a, b, conv_w, slot, snap, o, dev_err=None, stream=None):
    """gdn_verify_k: k drafts per batch row, snapshot after each; committed state untouched."""
    B, k = x.shape[0], x.shape[1]
    C, Hv, dv, dk = geom.conv_channels, geom.n_v_heads, geom.d_v, geom.d_k
    _check_pool(geom, pool)
    _need(x, "x", (B, k, C), geom.dtype)
    _need(a, "a", (B, k, Hv), geom.dtype)
    _need(b, "b", (B, k, Hv), geom.dtype)
    _need(conv_w, "conv_w", (C, geom.conv_width), torch.float32, optional=geom.conv_width == 0)
    _need(slot, "slot", (B,), torch.int32)
    _need(snap, "snap", (B, k, Hv, dv, dk), torch.float32)
    _need(o, "o", (B, k, Hv, dv), geom.dtype)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    g = geom.c_struct()
    _check(lib().gdn_verify_k(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_state), _ptr(pool.conv_pos),
                              _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w), _ptr(slot), B, k, _ptr(snap), _ptr(o),
                              _ptr(dev_err), _stream(stream)))


def rollback(geom: Geometry, pool: SlotPool, snap, slot, accepted, dev_err=None, stream=None):
    """gdn_rollback: commit accepted[i] drafts of batch row i (0 keeps the slot as it was)."""
    B, k = snap.shape[0], snap.shape[1]
    _check_pool(geom, pool)
    _need(snap, "snap", (B, k, geom.n_v_heads, geom.d_v, geom.d_k), torch.float32)
    _need(slot, "slot", (B,), torch.int32)
    _need(accepted, "accepted", (B,), torch.int32)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    g = geom.c_struct()
    _check(lib().gdn_rollback(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_pos), _ptr(snap), _ptr(slot),
                              _ptr(accepted), B, k, _ptr(dev_err), _stream(stream)))


def verify_k_slots(geom: Geometry, pool: SlotPool, x, a, b, conv_w, slot, snap_slot, o, dev_err=None,
                   stream=None, k_row=None):
    """gdn_verify_k_slots: as verify_k, but snapshot j of row i becomes pool slot snap_slot[i][j];
    k_row (device int32 [batch], optional) gives each row its own number of drafts."""
    B, k = x.shape[0], x.shape[1]
    C, Hv, dv = geom.conv_channels, geom.n_v_heads, geom.d_v
    _check_pool(geom, pool)
    _need(x, "x", (B, k, C), geom.dtype)
    _need(a, "a", (B, k, Hv), geom.dtype)
    _need(b, "b", (B, k, Hv), geom.dtype)
    _need(conv_w, "conv_w", (C, geom.conv_width), torch.float32, optional=geom.conv_width == 0)
    _need(slot, "slot", (B,), torch.int32)
    _need(snap_slot, "snap_slot", (B, k), torch.int32)
    _need(k_row, "k_row", (B,), torch.int32, optional=True)
    _need(o, "o", (B, k, Hv, dv), geom.dtype)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    g = geom.c_struct()
    _check(lib().gdn_verify_k_slots(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_state),
                                    _ptr(pool.conv_pos), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w), _ptr(slot), B,
                                    k, _ptr(k_row), _ptr(snap_slot), _ptr(o), _ptr(dev_err), _stream(stream)))


def commit_slots(geom: Geometry, slot, snap_slot, accepted, next_slot, dev_err=None, stream=None, k_row=None):
    """gdn_commit_slots: next_slot[i] = snap_slot[i][accepted[i]-1], or slot[i] when accepted[i] == 0."""
    B, k = snap_slot.shape[0], snap_slot.shape[1]
    _need(slot, "slot", (B,), torch.int32)
    _need(k_row, "k_row", (B,), torch.int32, optional=True)
    _need(snap_slot, "snap_slot", (B, k), torch.int32)
    _need(accepted, "accepted", (B,), torch.int32)
    _need(next_slot, "next_slot", (B,), torch.int32)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    g = geom.c_struct()
    _check(lib().gdn_commit_slots(ctypes.byref(g), _ptr(slot), _ptr(k_row), _ptr(snap_slot), _ptr(accepted), B,
                                  k, _ptr(next_slot), _ptr(dev_err), _stream(stream)))


_err_words = {}


def _default_err(device) -> torch.Tensor:
    """The binding's own device error word of a device (prefill calls without
    a dev_err of their own report into it; read it with device_error())."""
    idx = torch.device(device).index
    if idx is None:
        idx = torch.cuda.current_device()
    w = _err_words.get(idx)
    if w is None:
        w = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", idx))
        _err_words[idx] = w
    return w


def device_error(device="cuda", clear: bool = True) -> int:
    """First device error code the prefill calls without a dev_err of their
    own reported on this device since the last clear (synchronises)."""
    w = _default_err(device)
    v = int(w.item())
    if clear and v:
        w.zero_()
    return v


def prefill_workspace_bytes(geom: Geometry, n_tokens: int, n_seqs: int) -> int:
    g = geom.c_struct()
    return int(lib().gdn_prefill_workspace_bytes(ctypes.byref(g), n_tokens, n_seqs))


def alloc_prefill_workspace(geom: Geometry, n_tokens: int, n_seqs: int, device="cuda") -> torch.Tensor:
    """A caller-owned workspace of the size gdn_prefill_workspace_bytes reports."""
    n = prefill_workspace_bytes(geom, n_tokens, n_seqs)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def prefill_chunked(geom: Geometry, pool: SlotPool, x, a, b, conv_w, cu_seqlens, slot, has_init, o,
                    workspace, dev_err=None, stream=None, ckpt=None, ckpt_every=0):
    """gdn_prefill_chunked: varlen chunked prefill; final states and histories go to the slots.

    With ckpt_every > 0 it calls gdn_prefill_chunked_ckpt instead, which also
    writes the state after every ckpt_every tokens of each sequence into ckpt,
    an fp32 device tensor [n][H_v][d_v][d_k] with n >= n_tokens // ckpt_every
    (see ``checkpoint_count`` for the number a partition produces).
    Without a dev_err of the caller's, device errors go to the binding's own
    word for the device (``device_error``).
    """
    N = x.shape[0]
    S = slot.shape[0]
    C, Hv, dv = geom.conv_channels, geom.n_v_heads, geom.d_v
    _check_pool(geom, pool)
    _need(x, "x", (N, C), geom.dtype)
    _need(a, "a", (N, Hv), geom.dtype)
    _need(b, "b", (N, Hv), geom.dtype)
    _need(conv_w, "conv_w", (C, geom.conv_width), torch.float32, optional=geom.conv_width == 0)
    _need(cu_seqlens, "cu_seqlens", (S + 1,), torch.int32)
    _need(slot, "slot", (S,), torch.int32)
    _need(has_init, "has_init", (S,), torch.int32)
    _need(o, "o", (N, Hv, dv), geom.dtype)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    if dev_err is None:  # a stalled hand-off or unscheduled work is never silent
        dev_err = _default_err(x.device)
    if workspace is None or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous device tensor")
    g = geom.c_struct()
    nbytes = workspace.numel() * workspace.element_size()
    if ckpt_every:
        cap = N // ckpt_every if ckpt_every > 0 else 0
        if ckpt is None and cap == 0:
            ck_bytes = 0
        else:
            if (ckpt is None or not ckpt.is_cuda or ckpt.dtype != torch.float32 or not ckpt.is_contiguous()
                    or ckpt.dim() != 4 or tuple(ckpt.shape[1:]) != (Hv, dv, geom.d_k)):
                raise ValueError(f"ckpt: need a contiguous float32 device tensor [n][{Hv}][{dv}][{geom.d_k}]")
            ck_bytes = ckpt.numel() * 4
        _check(lib().gdn_prefill_chunked_ckpt(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_state),
                                              _ptr(pool.conv_pos), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w),
                                              _ptr(cu_seqlens), _ptr(slot), _ptr(has_init), S, N, CHUNK,
                                              _ptr(workspace), nbytes, _ptr(o), int(ckpt_every), _ptr(ckpt),
                                              ck_bytes, _ptr(dev_err), _stream(stream)))
        return
    _check(lib().gdn_prefill_chunked(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_state),
                                     _ptr(pool.conv_pos), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w),
                                     _ptr(cu_seqlens), _ptr(slot), _ptr(has_init), S, N, CHUNK,
                                     _ptr(workspace), nbytes, _ptr(o), _ptr(dev_err), _stream(stream)))


def prefill_timing_events(start: Optional[torch.cuda.Event], stop: Optional[torch.cuda.Event]):
    """gdn_prefill_timing_events: this thread's next prefill call records
    ``start`` when its plan kernel completes (its main kernel begins) and
    ``stop`` when its main kernel completes (timing events, recorded once
    before so that they exist), through the kernel launches themselves; both
    None clears it."""
    def handle(ev):
        if ev is None:
            return None
        h = ev.cuda_event
        if not h:
            raise ValueError("prefill_timing_events: the event has no HIP event yet (record it once first)")
        return h
    _check(lib().gdn_prefill_timing_events(handle(start), handle(stop)))


def prefill_chunked_static(geom: Geometry, pool: SlotPool, x, a, b, conv_w, cu_seqlens, slot, has_init, o,
                           dev_err=None, stream=None):
    """gdn_prefill_chunked_static: prefill_chunked with the library's own static
    workspace (no allocation in the call; calls that overlap on one GPU race)."""
    N = x.shape[0]
    S = slot.shape[0]
    C, Hv, dv = geom.conv_channels, geom.n_v_heads, geom.d_v
    _check_pool(geom, pool)
    _need(x, "x", (N, C), geom.dtype)
    _need(a, "a", (N, Hv), geom.dtype)
    _need(b, "b", (N, Hv), geom.dtype)
    _need(conv_w, "conv_w", (C, geom.conv_width), torch.float32, optional=geom.conv_width == 0)
    _need(cu_seqlens, "cu_seqlens", (S + 1,), torch.int32)
    _need(slot, "slot", (S,), torch.int32)
    _need(has_init, "has_init", (S,), torch.int32)
    _need(o, "o", (N, Hv, dv), geom.dtype)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True)
    if dev_err is None:
        dev_err = _default_err(x.device)
    g = geom.c_struct()
    _check(lib().gdn_prefill_chunked_static(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_state),
                                            _ptr(pool.conv_pos), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w),
                                            _ptr(cu_seqlens), _ptr(slot), _ptr(has_init), S, N, CHUNK,
                                            _ptr(o), _ptr(dev_err), _stream(stream)))


def checkpoint_count(seq_lens, ckpt_every: int) -> int:
    """Checkpoints gdn_prefill_chunked_ckpt writes for these sequence lengths."""
    return sum(int(n) // ckpt_every for n in seq_lens)


# --------------------------------------------------------------------------
# verify over a tree of drafts
# --------------------------------------------------------------------------

def verify_tree_slots(geom: Geometry, pool: SlotPool, x, a, b, conv_w, slot, parent, snap_slot, o, dev_err=None,
                      stream=None, k_row=None):
    """gdn_verify_tree_slots: as verify_k_slots, but draft j of row i continues from draft parent[i][j]
    (device int32 [batch][k]; -1: from the row's committed state); commit with commit_slots, accepted =
    1 + the last accepted node.  Without a dev_err, device errors go to ``device_error``'s word."""
    B, k, dev = x.shape[0], x.shape[1], _index(x)
    C, Hv, dv = geom.conv_channels, geom.n_v_heads, geom.d_v
    _check_pool(geom, pool, dev)
    _need(x, "x", (B, k, C), geom.dtype, device=dev)
    _need(a, "a", (B, k, Hv), geom.dtype, device=dev)
    _need(b, "b", (B, k, Hv), geom.dtype, device=dev)
    _need(conv_w, "conv_w", (C, geom.conv_width), torch.float32, optional=geom.conv_width == 0, device=dev)
    _need(slot, "slot", (B,), torch.int32, device=dev)
    _need(parent, "parent", (B, k), torch.int32, device=dev)
    _need(snap_slot, "snap_slot", (B, k), torch.int32, device=dev)
    _need(k_row, "k_row", (B,), torch.int32, optional=True, device=dev)
    _need(o, "o", (B, k, Hv, dv), geom.dtype, device=dev)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True, device=dev)
    st = _here(dev, stream)
    if dev_err is None:
        dev_err = _default_err(x.device)
    g = geom.c_struct()
    _check(lib().gdn_verify_tree_slots(ctypes.byref(g), _ptr(pool.state), _ptr(pool.conv_state),
                                       _ptr(pool.conv_pos), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w), _ptr(slot), B,
                                       k, _ptr(k_row), _ptr(parent), _ptr(snap_slot), _ptr(o), _ptr(dev_err),
                                       st))


# --------------------------------------------------------------------------
# the attention layers of a hybrid stack: paged KV cache and attention over it
# --------------------------------------------------------------------------

@dataclass(frozen=True)
class AttnGeometry:
    """Python mirror of gdn_attn_geometry (see include/gdn.h for every field); scale None: 1/sqrt(d_head)."""

    n_q_heads: int = 24
    n_kv_heads: int = 4
    d_head: int = 256
    page_tokens: int = 16
    n_pages: int = 1024
    max_pages: int = 1024
    max_tree: int = 16
    dtype: torch.dtype = torch.bfloat16
    scale: Optional[float] = None

    def c_struct(self) -> GdnAttnGeometry:
        code = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}[self.dtype]
        return GdnAttnGeometry(self.n_q_heads, self.n_kv_heads, self.d_head, self.page_tokens, self.n_pages,
                               self.max_pages, self.max_tree, code,
                               self.d_head ** -0.5 if self.scale is None else self.scale)

    def check(self):
        _check(lib().gdn_check_attn_geometry(self._ref(), None, 0))

    def _ref(self):
        """The C struct by reference, made once per geometry (it is frozen)."""
        r = self.__dict__.get("_c_ref")
        if r is None:
            r = ctypes.byref(self.c_struct())
            object.__setattr__(self, "_c_ref", r)
        return r

    def __getstate__(self):
        """What copies and pickles carry: the fields, not this object's C struct."""
        return {k: v for k, v in self.__dict__.items() if k != "_c_ref"}


@dataclass
class KVCache:
    """Caller-owned K and V pages of one attention layer: dtype [n_pages][H_kv][page_tokens][d_head] each."""

    k: torch.Tensor
    v: torch.Tensor

    @staticmethod
    def zeros(geom: AttnGeometry, device="cuda") -> "KVCache":
        shape = (geom.n_pages, geom.n_kv_heads, geom.page_tokens, geom.d_head)
        return KVCache(torch.zeros(shape, dtype=geom.dtype, device=device),
                       torch.zeros(shape, dtype=geom.dtype, device=device))


def _need_rows(t: Optional[torch.Tensor], name: str, shape, dtype, device: Optional[int] = None) -> int:
    """Rows of heads, any row stride, contiguous within a row; returns the row stride in elements."""
    if (t is not None and (t.is_cuda if device is None else t.get_device() == device) and t.dtype == dtype
            and t.shape == shape and t.is_contiguous()):
        return shape[-2] * shape[-1]
    if t is None:
        raise ValueError(f"{name}: missing")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, required {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, required {tuple(shape)}")
    st = t.stride()
    D = shape[-1]
    row = st[-3]
    if shape[-3] == 1:  # one row per leading index: its stride says nothing
        row = st[0] if len(shape) == 4 and shape[0] > 1 else shape[-2] * D
    if (st[-1] != 1 or (st[-2] != D and shape[-2] > 1) or (len(shape) == 4 and shape[0] > 1 and st[0] != shape[1] * row)
            or row < 0):
        raise ValueError(f"{name}: strides {tuple(st)}, required: heads contiguous, rows one stride apart")
    _need_device(t, name, device)
    return row


def _check_cache(geom: AttnGeometry, cache: KVCache, device: Optional[int]):
    shape = (geom.n_pages, geom.n_kv_heads, geom.page_tokens, geom.d_head)
    _need(cache.k, "cache.k", shape, geom.dtype, device=device)
    _need(cache.v, "cache.v", shape, geom.dtype, device=device)


def _workspace(workspace, device: Optional[int]):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous device tensor")
    _need_device(workspace, "workspace", device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def kv_plan(geom: AttnGeometry, kv_len, new_len, free_pages, n_free, block_table, cu_new, slot_map, position,
            kv_len_out, n_free_out, dev_err=None, stream=None):
    """gdn_kv_plan: block tables, slot map and positions of the new tokens from the rows' lengths (new_len -1: the
    row leaves and gives its pages back); slot_map and position may be longer than the new tokens (padding)."""
    B, N, dev = kv_len.shape[0], slot_map.shape[0], _index(kv_len)
    i32 = torch.int32
    _need(kv_len, "kv_len", (B,), i32, device=dev)
    _need(new_len, "new_len", (B,), i32, device=dev)
    _need(free_pages, "free_pages", (geom.n_pages,), i32, device=dev)
    _need(n_free, "n_free", (1,), i32, device=dev)
    _need(block_table, "block_table", (B, geom.max_pages), i32, device=dev)
    _need(cu_new, "cu_new", (B + 1,), i32, device=dev)
    _need(slot_map, "slot_map", (N,), i32, device=dev)
    _need(position, "position", (N,), i32, device=dev)
    _need(kv_len_out, "kv_len_out", (B,), i32, device=dev)
    _need(n_free_out, "n_free_out", (1,), i32, device=dev)
    _need(dev_err, "dev_err", (1,), i32, optional=True, device=dev)
    st = _here(dev, stream)
    if dev_err is None:
        dev_err = _default_err(kv_len.device)
    _check(lib().gdn_kv_plan(geom._ref(), kv_len.data_ptr(), new_len.data_ptr(), free_pages.data_ptr(),
                             n_free.data_ptr(), block_table.data_ptr(), B, N, cu_new.data_ptr(), slot_map.data_ptr(),
                             position.data_ptr(), kv_len_out.data_ptr(), n_free_out.data_ptr(), dev_err.data_ptr(),
                             st))


def kv_write(geom: AttnGeometry, cache: KVCache, k, v, slot_map, dev_err=None, stream=None):
    """gdn_kv_write: k and v rows [n_tokens][H_kv][d_head] (any row stride) into their cache slots; slot -1 skips."""
    N, dev = slot_map.shape[0], _index(cache.k)
    shape = (N, geom.n_kv_heads, geom.d_head)
    _check_cache(geom, cache, dev)
    ks = _need_rows(k, "k", shape, geom.dtype, dev)
    vs = _need_rows(v, "v", shape, geom.dtype, dev)
    _need(slot_map, "slot_map", (N,), torch.int32, device=dev)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True, device=dev)
    st = _here(dev, stream)
    if dev_err is None:
        dev_err = _default_err(k.device)
    _check(lib().gdn_kv_write(geom._ref(), cache.k.data_ptr(), cache.v.data_ptr(), k.data_ptr(), ks, v.data_ptr(), vs,
                              slot_map.data_ptr(), N, dev_err.data_ptr(), st))


def attn_prefill_workspace_bytes(geom: AttnGeometry, n_tokens: int, n_seqs: int, up_to: bool = False) -> int:
    """What a call of these sizes needs; up_to: the most that any call of up to these sizes needs (a shorter one may
    need more than a longer one)."""
    f = lib().gdn_attn_prefill_workspace_max_bytes if up_to else lib().gdn_attn_prefill_workspace_bytes
    return int(f(geom._ref(), n_tokens, n_seqs))


def alloc_attn_prefill_workspace(geom: AttnGeometry, n_tokens: int, n_seqs: int, device="cuda",
                                 up_to: bool = False) -> torch.Tensor:
    """A caller-owned workspace of the size attn_prefill_workspace_bytes reports (may be empty)."""
    return torch.empty(attn_prefill_workspace_bytes(geom, n_tokens, n_seqs, up_to), dtype=torch.uint8, device=device)


def attn_prefill(geom: AttnGeometry, q, k, v, cu_seqlens, o, workspace=None, cache: Optional[KVCache] = None,
                 block_table=None, ctx_len=None, dev_err=None, stream=None):
    """gdn_attn_prefill: causal attention of packed prompts, q [n_tokens][H_q][d_head], k and v
    [n_tokens][H_kv][d_head] (any row strides), sequence s after ctx_len[s] tokens that are in the cache already
    (block table row s); ctx_len None: none.  Without a dev_err, device errors go to ``device_error``'s word."""
    N, S, dev = q.shape[0], cu_seqlens.shape[0] - 1, _index(q)
    if S < 1:
        raise ValueError("cu_seqlens: needs at least two entries")
    qs = _need_rows(q, "q", (N, geom.n_q_heads, geom.d_head), geom.dtype, dev)
    ks = _need_rows(k, "k", (N, geom.n_kv_heads, geom.d_head), geom.dtype, dev)
    vs = _need_rows(v, "v", (N, geom.n_kv_heads, geom.d_head), geom.dtype, dev)
    _need(cu_seqlens, "cu_seqlens", (S + 1,), torch.int32, device=dev)
    _need(o, "o", (N, geom.n_q_heads, geom.d_head), geom.dtype, device=dev)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True, device=dev)
    kc = vc = bt = cl = None
    if ctx_len is not None:
        if cache is None:
            raise ValueError("cache: missing (ctx_len is given)")
        _check_cache(geom, cache, dev)
        _need(block_table, "block_table", (S, geom.max_pages), torch.int32, device=dev)
        _need(ctx_len, "ctx_len", (S,), torch.int32, device=dev)
        kc, vc, bt, cl = cache.k.data_ptr(), cache.v.data_ptr(), block_table.data_ptr(), ctx_len.data_ptr()
    st = _here(dev, stream)
    ws, nbytes = _workspace(workspace, dev)
    if dev_err is None:
        dev_err = _default_err(q.device)
    _check(lib().gdn_attn_prefill(geom._ref(), q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                                  cu_seqlens.data_ptr(), S, N, kc, vc, bt, cl, ws, nbytes, o.data_ptr(),
                                  dev_err.data_ptr(), st))


def attn_tree_workspace_bytes(geom: AttnGeometry, batch: int, n: int, up_to: bool = False) -> int:
    """What a call of these sizes needs; up_to: the most that any call of up to these sizes needs."""
    f = lib().gdn_attn_tree_workspace_max_bytes if up_to else lib().gdn_attn_tree_workspace_bytes
    return int(f(geom._ref(), batch, n))


def alloc_attn_tree_workspace(geom: AttnGeometry, batch: int, n: int, device="cuda", up_to: bool = False) -> torch.Tensor:
    """A caller-owned workspace of the size attn_tree_workspace_bytes reports (may be empty)."""
    return torch.empty(attn_tree_workspace_bytes(geom, batch, n, up_to), dtype=torch.uint8, device=device)


def attn_tree(geom: AttnGeometry, cache: KVCache, block_table, ctx_len, q, k, v, parent, o, workspace=None,
              n_row=None, dev_err=None, stream=None):
    """gdn_attn_tree: each row's n drafted nodes attend its ctx_len cached tokens, their ancestors among the drafts
    (parent [batch][n], -1: the cached tokens) and themselves; q [batch][n][H_q][d_head], k and v
    [batch][n][H_kv][d_head].  n = 1 with parent -1 is the decode step."""
    B, n, dev = q.shape[0], q.shape[1], _index(cache.k)
    _check_cache(geom, cache, dev)
    qs = _need_rows(q, "q", (B, n, geom.n_q_heads, geom.d_head), geom.dtype, dev)
    ks = _need_rows(k, "k", (B, n, geom.n_kv_heads, geom.d_head), geom.dtype, dev)
    vs = _need_rows(v, "v", (B, n, geom.n_kv_heads, geom.d_head), geom.dtype, dev)
    _need(block_table, "block_table", (B, geom.max_pages), torch.int32, device=dev)
    _need(ctx_len, "ctx_len", (B,), torch.int32, device=dev)
    _need(parent, "parent", (B, n), torch.int32, device=dev)
    _need(n_row, "n_row", (B,), torch.int32, optional=True, device=dev)
    _need(o, "o", (B, n, geom.n_q_heads, geom.d_head), geom.dtype, device=dev)
    _need(dev_err, "dev_err", (1,), torch.int32, optional=True, device=dev)
    st = _here(dev, stream)
    ws, nbytes = _workspace(workspace, dev)
    if dev_err is None:
        dev_err = _default_err(q.device)
    _check(lib().gdn_attn_tree(geom._ref(), q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, parent.data_ptr(),
                               None if n_row is None else n_row.data_ptr(), B, n, cache.k.data_ptr(),
                               cache.v.data_ptr(), block_table.data_ptr(), ctx_len.data_ptr(), ws, nbytes,
                               o.data_ptr(), dev_err.data_ptr(), st))


__all__ = [
    "Geometry", "GdnGeometry", "GdnError", "SlotPool", "lib", "conv_state_step", "decode_step", "verify_k",
    "rollback", "verify_k_slots", "commit_slots", "prefill_chunked", "prefill_chunked_static", "prefill_workspace_bytes", "alloc_prefill_workspace",
    "checkpoint_count", "POS_ONE", "CHUNK",
    "DEV_OK", "DEV_BAD_SLOT", "DEV_BAD_ACCEPTED", "DEV_BAD_SEQLENS", "DEV_WAIT_TIMEOUT", "DEV_BAD_K",
    "DEV_INCOMPLETE", "device_error",
    "verify_tree_slots", "AttnGeometry", "GdnAttnGeometry", "KVCache", "kv_plan", "kv_write", "attn_prefill",
    "attn_prefill_workspace_bytes", "alloc_attn_prefill_workspace", "attn_tree", "attn_tree_workspace_bytes",
    "alloc_attn_tree_workspace", "DEV_BAD_PAGE", "DEV_NO_PAGES", "DEV_BAD_LENGTH", "DEV_BAD_PARENT",
]
