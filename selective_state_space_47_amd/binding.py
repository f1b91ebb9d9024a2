"""Thin ctypes binding over the C ABI in include/mamba_scan.h.

Argument marshalling only: checks dtypes, shapes and devices, allocates outputs and workspace with
torch, passes raw device pointers and torch's current HIP stream to the library.  Every step of
the computation runs in the library's kernels.  There is no fallback: if the native library is
missing the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
import threading

import torch

from . import _build

MAMBA_F32 = 0
MAMBA_BF16 = 1
DSTATE = 16

_lock = threading.Lock()
_LIB = None


class mamba_block_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("d_model", ctypes.c_int64), ("d_inner", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("dt_rank", ctypes.c_int64),
                ("conv_width", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class mamba_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("dim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("seqlen", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("chunk_len", ctypes.c_int32)]


class mamba_delta_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("qk_heads", ctypes.c_int64), ("v_heads", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class mamba_gated_norm_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("weight_groups", ctypes.c_int32),
                ("gate_first", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class mamba_add_norm_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32)]


class mamba_window_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("kv_len", ctypes.c_int64),
                ("q_heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("window", ctypes.c_int64), ("sinks", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class mamba_qk_norm_rope_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("q_heads", ctypes.c_int64), ("k_heads", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("rotary_dim", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


EXPORTS = ("mamba_scan_fwd", "mamba_scan_fwd_noalloc", "mamba_scan_fwd_conv", "mamba_state_update",
           "mamba_scan_workspace_bytes",
           "mamba_scan_bwd", "mamba_scan_bwd_workspace_bytes", "mamba_gemm_bf16",
           "mamba_block_fwd", "mamba_block_workspace_bytes", "mamba_delta_fwd",
           "mamba_delta_workspace_bytes", "mamba_delta_update", "mamba_delta_bwd",
           "mamba_delta_bwd_workspace_bytes", "mamba_gated_norm_fwd",
           "mamba_gated_norm_bwd", "mamba_gated_norm_bwd_workspace_bytes", "mamba_add_norm_fwd",
           "mamba_add_norm_bwd", "mamba_add_norm_bwd_workspace_bytes", "mamba_qk_norm_rope_fwd",
           "mamba_qk_norm_rope_bwd", "mamba_qk_norm_rope_bwd_workspace_bytes", "mamba_linear_attn_fwd",
           "mamba_linear_attn_workspace_bytes", "mamba_linear_attn_update", "mamba_linear_attn_bwd",
           "mamba_linear_attn_bwd_workspace_bytes", "mamba_window_attn_fwd", "mamba_window_attn_bwd",
           "mamba_window_attn_bwd_workspace_bytes", "mamba_window_cache_store", "mamba_window_attn_update",
           "mamba_window_attn_update_workspace_bytes", "mamba_status_string",
           "mamba_abi_version")


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """The loaded native library (raises RuntimeError if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    with _lock:
        if _LIB is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"native library {path} is missing: build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'` (hipcc, gfx950)")
            L = ctypes.CDLL(path)
            vp, fp = ctypes.c_void_p, ctypes.c_void_p
            dp = ctypes.POINTER(mamba_dims)
            L.mamba_scan_fwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, ctypes.c_int, vp, fp, dp,
                                         vp, ctypes.c_size_t, vp]
            L.mamba_scan_fwd.restype = ctypes.c_int
            L.mamba_scan_fwd_noalloc.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, ctypes.c_int, vp,
                                                 fp, dp, vp]
            L.mamba_scan_fwd_noalloc.restype = ctypes.c_int
            L.mamba_scan_fwd_conv.argtypes = [vp, fp, fp, ctypes.c_int, vp, fp, vp, vp, fp, vp,
                                              fp, ctypes.c_int, vp, fp, vp, dp, vp,
                                              ctypes.c_size_t, vp]
            L.mamba_scan_fwd_conv.restype = ctypes.c_int
            L.mamba_state_update.argtypes = [fp, vp, vp, fp, vp, vp, fp, vp, fp, ctypes.c_int, vp,
                                             dp, vp]
            L.mamba_state_update.restype = ctypes.c_int
            L.mamba_scan_workspace_bytes.argtypes = [dp]
            L.mamba_scan_workspace_bytes.restype = ctypes.c_size_t
            L.mamba_scan_bwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, ctypes.c_int, vp, fp,
                                         vp, vp, fp, vp, vp, fp, vp, fp, dp, vp,
                                         ctypes.c_size_t, vp]
            L.mamba_scan_bwd.restype = ctypes.c_int
            L.mamba_scan_bwd_workspace_bytes.argtypes = [dp]
            L.mamba_scan_bwd_workspace_bytes.restype = ctypes.c_size_t
            i64 = ctypes.c_int64
            L.mamba_gemm_bf16.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64,
                                          i64, ctypes.c_int, ctypes.c_int, vp]
            L.mamba_gemm_bf16.restype = ctypes.c_int
            bp = ctypes.POINTER(mamba_block_dims)
            L.mamba_block_fwd.argtypes = [vp, vp, fp, fp, vp, vp, fp, fp, fp, vp, vp, bp, vp,
                                          ctypes.c_size_t, vp]
            L.mamba_block_fwd.restype = ctypes.c_int
            L.mamba_block_workspace_bytes.argtypes = [bp]
            L.mamba_block_workspace_bytes.restype = ctypes.c_size_t
            f32, sz = ctypes.c_float, ctypes.c_size_t
            ep = ctypes.POINTER(mamba_delta_dims)
            L.mamba_delta_fwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, f32, vp, fp, ep, vp, sz, vp]
            L.mamba_delta_fwd.restype = ctypes.c_int
            L.mamba_delta_workspace_bytes.argtypes = [ep, ctypes.c_int]
            L.mamba_delta_workspace_bytes.restype = sz
            L.mamba_delta_update.argtypes = [fp, vp, vp, vp, vp, vp, f32, vp, ep, vp]
            L.mamba_delta_update.restype = ctypes.c_int
            L.mamba_delta_bwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, f32, vp, fp, vp, vp, vp, vp,
                                          vp, fp, ep, vp, sz, vp]
            L.mamba_delta_bwd.restype = ctypes.c_int
            L.mamba_delta_bwd_workspace_bytes.argtypes = [ep, ctypes.c_int]
            L.mamba_delta_bwd_workspace_bytes.restype = sz
            np_ = ctypes.POINTER(mamba_gated_norm_dims)
            L.mamba_gated_norm_fwd.argtypes = [vp, vp, fp, f32, vp, np_, vp]
            L.mamba_gated_norm_fwd.restype = ctypes.c_int
            L.mamba_gated_norm_bwd.argtypes = [vp, vp, fp, f32, vp, vp, vp, fp, np_, vp, sz, vp]
            L.mamba_gated_norm_bwd.restype = ctypes.c_int
            L.mamba_gated_norm_bwd_workspace_bytes.argtypes = [np_]
            L.mamba_gated_norm_bwd_workspace_bytes.restype = sz
            ap = ctypes.POINTER(mamba_add_norm_dims)
            L.mamba_add_norm_fwd.argtypes = [vp, vp, fp, fp, fp, f32, vp, vp, ap, vp]
            L.mamba_add_norm_fwd.restype = ctypes.c_int
            L.mamba_add_norm_bwd.argtypes = [vp, vp, fp, fp, fp, f32, vp, vp, vp, vp, fp, fp, fp,
                                             ap, vp, sz, vp]
            L.mamba_add_norm_bwd.restype = ctypes.c_int
            L.mamba_add_norm_bwd_workspace_bytes.argtypes = [ap]
            L.mamba_add_norm_bwd_workspace_bytes.restype = sz
            kp = ctypes.POINTER(mamba_qk_norm_rope_dims)
            L.mamba_qk_norm_rope_fwd.argtypes = [vp, vp, fp, fp, vp, vp, f32, vp, vp, kp, vp]
            L.mamba_qk_norm_rope_fwd.restype = ctypes.c_int
            L.mamba_qk_norm_rope_bwd.argtypes = [vp, vp, fp, fp, vp, vp, f32, vp, vp, vp, vp, fp,
                                                 fp, kp, vp, sz, vp]
            L.mamba_qk_norm_rope_bwd.restype = ctypes.c_int
            L.mamba_qk_norm_rope_bwd_workspace_bytes.argtypes = [kp]
            L.mamba_qk_norm_rope_bwd_workspace_bytes.restype = sz
            L.mamba_linear_attn_fwd.argtypes = [vp, vp, vp, fp, fp, vp, f32, vp, fp, ep, vp, sz, vp]
            L.mamba_linear_attn_fwd.restype = ctypes.c_int
            L.mamba_linear_attn_workspace_bytes.argtypes = [ep, ctypes.c_int]
            L.mamba_linear_attn_workspace_bytes.restype = sz
            L.mamba_linear_attn_update.argtypes = [fp, vp, vp, vp, fp, f32, vp, ep, vp]
            L.mamba_linear_attn_update.restype = ctypes.c_int
            L.mamba_linear_attn_bwd.argtypes = [vp, vp, vp, fp, fp, vp, f32, vp, fp, vp, vp, vp, fp, fp,
                                                ep, vp, sz, vp]
            L.mamba_linear_attn_bwd.restype = ctypes.c_int
            L.mamba_linear_attn_bwd_workspace_bytes.argtypes = [ep, ctypes.c_int]
            L.mamba_linear_attn_bwd_workspace_bytes.restype = sz
            wp = ctypes.POINTER(mamba_window_dims)
            L.mamba_window_attn_fwd.argtypes = [vp, vp, vp, vp, vp, f32, vp, fp, wp, vp]
            L.mamba_window_attn_fwd.restype = ctypes.c_int
            L.mamba_window_attn_bwd.argtypes = [vp, vp, vp, vp, vp, f32, vp, fp, vp, vp, vp, vp, wp, vp,
                                                sz, vp]
            L.mamba_window_attn_bwd.restype = ctypes.c_int
            L.mamba_window_attn_bwd_workspace_bytes.argtypes = [wp, ctypes.c_int]
            L.mamba_window_attn_bwd_workspace_bytes.restype = sz
            L.mamba_window_cache_store.argtypes = [vp, vp, vp, vp, vp, wp, vp]
            L.mamba_window_cache_store.restype = ctypes.c_int
            L.mamba_window_attn_update.argtypes = [vp, vp, vp, vp, vp, vp, f32, vp, wp, vp, sz, vp]
            L.mamba_window_attn_update.restype = ctypes.c_int
            L.mamba_window_attn_update_workspace_bytes.argtypes = [wp]
            L.mamba_window_attn_update_workspace_bytes.restype = sz
            L.mamba_status_string.argtypes = [ctypes.c_int]
            L.mamba_status_string.restype = ctypes.c_char_p
            L.mamba_abi_version.argtypes = []
            L.mamba_abi_version.restype = ctypes.c_int
            _LIB = L
    return _LIB


def mamba_status_string(status: int) -> str:
    return lib().mamba_status_string(int(status)).decode()


def mamba_abi_version() -> int:
    return int(lib().mamba_abi_version())


def _io_code(dtype) -> int:
    if dtype == torch.float32:
        return MAMBA_F32
    if dtype == torch.bfloat16:
        return MAMBA_BF16
    raise ValueError(f"unsupported io dtype {dtype}; use float32 or bfloat16")


def make_dims(batch, dim, seqlen, io_dtype, dstate=DSTATE, chunk_len=0) -> mamba_dims:
    return mamba_dims(int(batch), int(dim), int(dstate), int(seqlen), int(io_dtype),
                      int(chunk_len))


def mamba_scan_workspace_bytes(batch, dim, seqlen, io_dtype=torch.float32, dstate=DSTATE,
                               chunk_len=0) -> int:
    code = io_dtype if isinstance(io_dtype, int) else _io_code(io_dtype)
    dm = make_dims(batch, dim, seqlen, code, dstate, chunk_len)
    return int(lib().mamba_scan_workspace_bytes(ctypes.byref(dm)))


def _ptr(t):
    # a plain int: the c_void_p argtypes convert it, which is cheaper than a c_void_p object
    return None if t is None else t.data_ptr()


# torch's own accessor of the current stream's raw handle (one C call); the public path builds a
# Stream object per call, which costs more host time than a short scan's kernel
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    """Raw handle of the current stream on `dev`, as an int."""
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


# dims structs (read-only for the library) and the forward's workspace size, per shape; short
# sequences are called at a high rate with the same shape
_FWD_CACHE = {}


def _fwd_dims(batch, dim, L, code, chunk_len):
    key = (batch, dim, L, code, chunk_len)
    hit = _FWD_CACHE.get(key)
    if hit is None:
        dm = make_dims(batch, dim, L, code, DSTATE, chunk_len)
        hit = (dm, int(lib().mamba_scan_workspace_bytes(ctypes.byref(dm))))
        if len(_FWD_CACHE) >= 1024:
            _FWD_CACHE.clear()
        _FWD_CACHE[key] = hit
    return hit


def _check(t, name, shape, dtype, device):
    if t is None:
        return
    # fast path: one combined test for a well-formed tensor (the per-call host overhead matters
    # for short sequences); anything else goes through the detailed checks below
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape
            and t.get_device() == device.index and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_group(tensors, shape, dtype, device):
    """_check for several (tensor, name) pairs of one shape and dtype; the common case (all
    well-formed) costs one Python call instead of one per tensor."""
    idx = device.index
    for t, name in tensors:
        if t is not None and not (type(t) is torch.Tensor and t.dtype is dtype
                                  and t.shape == shape and t.get_device() == idx
                                  and t.is_contiguous()):
            _check(t, name, shape, dtype, device)


_NO_SWITCH = contextlib.nullcontext()


def _on(dev):
    """Context making `dev` current for a call; nothing to switch when it already is."""
    return _NO_SWITCH if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _raise(status):
    if status != 0:
        raise ValueError(f"mamba library error {status}: {mamba_status_string(status)}")


def _workspace(workspace, need, dev, min_bytes=0):
    """The caller's workspace, checked, or a new one of `need` bytes (at least min_bytes).
    Returns (tensor or None, its size in bytes)."""
    if workspace is None:
        n = max(need, min_bytes)
        if n == 0:
            return None, 0
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def mamba_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False,
                   return_last_state=False, chunk_len=0, out=None, last_state=None,
                   workspace=None):
    """Selective-scan forward (see mamba_scan_fwd in include/mamba_scan.h).

    u, delta, z: (batch, dim, L); B, C: (batch, 16, L) -- all float32 or all bfloat16;
    A: (dim, 16) float32; D, delta_bias: (dim,) float32.  Returns out, or (out, last_state).
    """
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, seqlen)")
    batch, dim, L = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io = u.dtype
    code = _io_code(io)
    if out is None:
        out = torch.empty((batch, dim, L), dtype=io, device=dev)
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, dim, DSTATE), dtype=torch.float32, device=dev)
    _check_group(((u, "u"), (delta, "delta"), (z, "z"), (out, "out")), (batch, dim, L), io, dev)
    _check_group(((B, "B"), (C, "C")), (batch, DSTATE, L), io, dev)
    _check(A, "A", (dim, DSTATE), torch.float32, dev)
    _check_group(((D, "D"), (delta_bias, "delta_bias")), (dim,), torch.float32, dev)
    _check(last_state, "last_state", (batch, dim, DSTATE), torch.float32, dev)
    dm, ws_bytes = _fwd_dims(batch, dim, L, code, chunk_len)
    L_ = lib()
    workspace, ws_len = _workspace(workspace, ws_bytes, dev)
    with _on(dev):
        stream = _stream(dev)
        st = L_.mamba_scan_fwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                               _ptr(z), _ptr(delta_bias), int(bool(delta_softplus)), _ptr(out),
                               _ptr(last_state), ctypes.byref(dm), _ptr(workspace), ws_len,
                               stream)
    _raise(st)
    return (out, last_state) if return_last_state else out


def mamba_scan_fwd_noalloc(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                           delta_softplus=False, return_last_state=False, chunk_len=0, out=None,
                           last_state=None):
    """mamba_scan_fwd_noalloc of include/mamba_scan.h: the forward with its chunk records in the
    library's fixed per-GPU scratch array (no workspace).  Arguments and results as for
    mamba_scan_fwd; outputs are allocated here only when not passed in."""
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, seqlen)")
    batch, dim, L = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io = u.dtype
    code = _io_code(io)
    for t, name, shape, dt in ((u, "u", (batch, dim, L), io), (delta, "delta", (batch, dim, L), io),
                               (z, "z", (batch, dim, L), io), (B, "B", (batch, DSTATE, L), io),
                               (C, "C", (batch, DSTATE, L), io),
                               (A, "A", (dim, DSTATE), torch.float32),
                               (D, "D", (dim,), torch.float32),
                               (delta_bias, "delta_bias", (dim,), torch.float32)):
        _check(t, name, shape, dt, dev)
    if out is None:
        out = torch.empty((batch, dim, L), dtype=io, device=dev)
    _check(out, "out", (batch, dim, L), io, dev)
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, dim, DSTATE), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", (batch, dim, DSTATE), torch.float32, dev)
    dm = _fwd_dims(batch, dim, L, code, chunk_len)[0]
    with _on(dev):
        stream = _stream(dev)
        st = lib().mamba_scan_fwd_noalloc(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                                          _ptr(D), _ptr(z), _ptr(delta_bias),
                                          int(bool(delta_softplus)), _ptr(out), _ptr(last_state),
                                          ctypes.byref(dm), stream)
    _raise(st)
    return (out, last_state) if return_last_state else out


def mamba_scan_fwd_conv(x, conv_weight, delta, A, B, C, D=None, z=None, delta_bias=None,
                        delta_softplus=False, conv_bias=None, return_last_state=False,
                        return_u=False, chunk_len=0, out=None, last_state=None, u_out=None,
                        workspace=None):
    """Forward with the causal conv1d + SiLU fused into the load stage (mamba_scan_fwd_conv in
    include/mamba_scan.h).  x: (batch, dim, L) like u of mamba_scan_fwd; conv_weight: (dim, W)
    float32, W in 1..4; conv_bias: (dim,) float32 or None.  Returns out, plus last_state and/or
    u when requested, in that order."""
    if x.dim() != 3:
        raise ValueError("x must be (batch, dim, seqlen)")
    batch, dim, L = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io = x.dtype
    code = _io_code(io)
    if conv_weight is None or conv_weight.dim() != 2:
        raise ValueError("conv_weight must be (dim, width)")
    width = conv_weight.shape[1]
    _check(x, "x", (batch, dim, L), io, dev)
    _check(conv_weight, "conv_weight", (dim, width), torch.float32, dev)
    _check(conv_bias, "conv_bias", (dim,), torch.float32, dev)
    _check(delta, "delta", (batch, dim, L), io, dev)
    _check(z, "z", (batch, dim, L), io, dev)
    _check(B, "B", (batch, DSTATE, L), io, dev)
    _check(C, "C", (batch, DSTATE, L), io, dev)
    _check(A, "A", (dim, DSTATE), torch.float32, dev)
    _check(D, "D", (dim,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    if out is None:
        out = torch.empty((batch, dim, L), dtype=io, device=dev)
    _check(out, "out", (batch, dim, L), io, dev)
    if return_last_state and last_state is None:
        last_state = torch.empty((batch, dim, DSTATE), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", (batch, dim, DSTATE), torch.float32, dev)
    if return_u and u_out is None:
        u_out = torch.empty((batch, dim, L), dtype=io, device=dev)
    _check(u_out, "u_out", (batch, dim, L), io, dev)
    dm = make_dims(batch, dim, L, code, DSTATE, chunk_len)
    L_ = lib()
    ws_bytes = int(L_.mamba_scan_workspace_bytes(ctypes.byref(dm)))
    workspace, ws_len = _workspace(workspace, ws_bytes, dev)
    with _on(dev):
        stream = _stream(dev)
        st = L_.mamba_scan_fwd_conv(_ptr(x), _ptr(conv_weight), _ptr(conv_bias), int(width),
                                    _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                    _ptr(delta_bias), int(bool(delta_softplus)), _ptr(out),
                                    _ptr(last_state), _ptr(u_out), ctypes.byref(dm),
                                    _ptr(workspace), ws_len, stream)
    _raise(st)
    res = [out]
    if return_last_state:
        res.append(last_state)
    if return_u:
        res.append(u_out)
    return res[0] if len(res) == 1 else tuple(res)


def mamba_state_update(state, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                       delta_softplus=False, out=None):
    """One generation step (see mamba_state_update in include/mamba_scan.h).

    state: (batch, dim, 16) float32, updated in place; u, delta, z: (batch, dim);
    B, C: (batch, 16); A: (dim, 16) float32; D, delta_bias: (dim,) float32.  Returns out.
    """
    if state.dim() != 3:
        raise ValueError("state must be (batch, dim, 16)")
    batch, dim, _ = state.shape
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io = u.dtype
    code = _io_code(io)
    _check(state, "state", (batch, dim, DSTATE), torch.float32, dev)
    _check(u, "u", (batch, dim), io, dev)
    _check(delta, "delta", (batch, dim), io, dev)
    _check(z, "z", (batch, dim), io, dev)
    _check(B, "B", (batch, DSTATE), io, dev)
    _check(C, "C", (batch, DSTATE), io, dev)
    _check(A, "A", (dim, DSTATE), torch.float32, dev)
    _check(D, "D", (dim,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    if out is None:
        out = torch.empty((batch, dim), dtype=io, device=dev)
    _check(out, "out", (batch, dim), io, dev)
    dm = _fwd_dims(batch, dim, 1, code, 0)[0]
    with _on(dev):
        stream = _stream(dev)
        st = lib().mamba_state_update(_ptr(state), _ptr(u), _ptr(delta), _ptr(A), _ptr(B),
                                      _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
                                      int(bool(delta_softplus)), _ptr(out), ctypes.byref(dm),
                                      stream)
    _raise(st)
    return out


def mamba_scan_bwd_workspace_bytes(batch, dim, seqlen, io_dtype=torch.float32, dstate=DSTATE,
                                   chunk_len=0) -> int:
    code = io_dtype if isinstance(io_dtype, int) else _io_code(io_dtype)
    dm = make_dims(batch, dim, seqlen, code, dstate, chunk_len)
    return int(lib().mamba_scan_bwd_workspace_bytes(ctypes.byref(dm)))


def mamba_scan_bwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False,
                   dout=None, dlast=None, chunk_len=0, workspace=None, grads=None):
    """Gradients of mamba_scan_fwd (see mamba_scan_bwd in include/mamba_scan.h).

    Same inputs as mamba_scan_fwd plus dout (batch, dim, L) in the io dtype and optionally dlast
    (batch, dim, 16) float32.  Returns a dict with du, ddelta, dz (io dtype, dz None without z),
    dB, dC (io dtype), dA, dD, ddelta_bias (float32; dD / ddelta_bias None when D / delta_bias is
    None).  `grads` may hold preallocated output tensors under the same keys.
    """
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, seqlen)")
    batch, dim, L = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io = u.dtype
    code = _io_code(io)
    if dout is None:
        raise ValueError("dout is required")
    for t, name, shape in ((u, "u", (batch, dim, L)), (delta, "delta", (batch, dim, L)),
                           (z, "z", (batch, dim, L)), (dout, "dout", (batch, dim, L)),
                           (B, "B", (batch, DSTATE, L)), (C, "C", (batch, DSTATE, L))):
        _check(t, name, shape, io, dev)
    _check(A, "A", (dim, DSTATE), torch.float32, dev)
    _check(D, "D", (dim,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    _check(dlast, "dlast", (batch, dim, DSTATE), torch.float32, dev)
    g = dict(grads or {})
    spec = {"du": ((batch, dim, L), io), "ddelta": ((batch, dim, L), io),
            "dB": ((batch, DSTATE, L), io), "dC": ((batch, DSTATE, L), io),
            "dA": ((dim, DSTATE), torch.float32)}
    if z is not None:
        spec["dz"] = ((batch, dim, L), io)
    if D is not None:
        spec["dD"] = ((dim,), torch.float32)
    if delta_bias is not None:
        spec["ddelta_bias"] = ((dim,), torch.float32)
    for k, (shape, dt) in spec.items():
        if g.get(k) is None:
            g[k] = torch.empty(shape, dtype=dt, device=dev)
        _check(g[k], k, shape, dt, dev)
    for k in ("dz", "dD", "ddelta_bias"):
        if k not in spec:
            g[k] = None
    dm = make_dims(batch, dim, L, code, DSTATE, chunk_len)
    L_ = lib()
    ws_bytes = int(L_.mamba_scan_bwd_workspace_bytes(ctypes.byref(dm)))
    workspace, ws_len = _workspace(workspace, ws_bytes, dev, min_bytes=1)
    with _on(dev):
        stream = _stream(dev)
        st = L_.mamba_scan_bwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                               _ptr(z), _ptr(delta_bias), int(bool(delta_softplus)), _ptr(dout),
                               _ptr(dlast), _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dA"]),
                               _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dz"]),
                               _ptr(g["ddelta_bias"]), ctypes.byref(dm), _ptr(workspace),
                               ws_len, stream)
    _raise(st)
    return {k: g[k] for k in ("du", "ddelta", "dz", "dA", "dB", "dC", "dD", "ddelta_bias")}


def mamba_gemm_bf16(A, B, b_kcontig=True, c_trans=False, out=None):
    """Batched bf16 GEMM on the matrix cores (mamba_gemm_bf16 in include/mamba_scan.h).

    A: (M, K) bfloat16.  B: (batch, N, K) when b_kcontig (element (k, n) = B[b, n, k]), else
    (batch, K, N).  Returns C: (batch, M, N), or (batch, N, M) when c_trans, bfloat16.
    """
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be (M, K) and B (batch, N, K) or (batch, K, N)")
    M, K = A.shape
    batch = B.shape[0]
    N = B.shape[1] if b_kcontig else B.shape[2]
    dev = A.device
    _check(A, "A", (M, K), torch.bfloat16, dev)
    _check(B, "B", (batch, N, K) if b_kcontig else (batch, K, N), torch.bfloat16, dev)
    shape = (batch, N, M) if c_trans else (batch, M, N)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _check(out, "out", shape, torch.bfloat16, dev)
    ldb = K if b_kcontig else N
    ldc = M if c_trans else N
    with _on(dev):
        stream = _stream(dev)
        st = lib().mamba_gemm_bf16(_ptr(A), _ptr(B), _ptr(out), M, N, K, batch, K, ldb, N * K,
                                   ldc, M * N, int(bool(b_kcontig)), int(bool(c_trans)), stream)
    _raise(st)
    return out


def block_dims(hidden, w_in, w_x, w_dt, conv_weight, dstate=DSTATE) -> mamba_block_dims:
    batch, L, d_model = hidden.shape
    E = w_in.shape[0] // 2
    R = w_dt.shape[1]
    return mamba_block_dims(int(batch), int(L), int(d_model), int(E), int(dstate), int(R),
                            int(conv_weight.shape[1]), 0)


def mamba_block_workspace_bytes(dims: mamba_block_dims) -> int:
    return int(lib().mamba_block_workspace_bytes(ctypes.byref(dims)))


def mamba_block_fwd(hidden, w_in, conv_weight, conv_bias, w_x, w_dt, dt_bias, A, D, w_out,
                    out=None, workspace=None):
    """A Mamba block forward (mamba_block_fwd in include/mamba_scan.h).

    hidden: (batch, L, d_model) bf16; w_in (2E, d_model), w_x (R + 32, E), w_dt (E, R),
    w_out (d_model, E) bf16; conv_weight (E, W), conv_bias (E,), dt_bias (E,), A (E, 16), D (E,)
    float32 (conv_bias, dt_bias, D may be None).  Returns out (batch, L, d_model) bf16.
    """
    if hidden.dim() != 3:
        raise ValueError("hidden must be (batch, seqlen, d_model)")
    batch, L, d_model = hidden.shape
    dev = hidden.device
    E = w_in.shape[0] // 2
    R = w_dt.shape[1] if w_dt.dim() == 2 else -1
    bf, f32 = torch.bfloat16, torch.float32
    _check(hidden, "hidden", (batch, L, d_model), bf, dev)
    _check(w_in, "w_in", (2 * E, d_model), bf, dev)
    _check(w_x, "w_x", (R + 2 * DSTATE, E), bf, dev)
    _check(w_dt, "w_dt", (E, R), bf, dev)
    _check(w_out, "w_out", (d_model, E), bf, dev)
    if conv_weight is None or conv_weight.dim() != 2:
        raise ValueError("conv_weight must be (d_inner, width)")
    _check(conv_weight, "conv_weight", (E, conv_weight.shape[1]), f32, dev)
    _check(conv_bias, "conv_bias", (E,), f32, dev)
    _check(dt_bias, "dt_bias", (E,), f32, dev)
    _check(A, "A", (E, DSTATE), f32, dev)
    _check(D, "D", (E,), f32, dev)
    if out is None:
        out = torch.empty((batch, L, d_model), dtype=bf, device=dev)
    _check(out, "out", (batch, L, d_model), bf, dev)
    dm = block_dims(hidden, w_in, w_x, w_dt, conv_weight)
    L_ = lib()
    ws_bytes = int(L_.mamba_block_workspace_bytes(ctypes.byref(dm)))
    workspace, ws_len = _workspace(workspace, ws_bytes, dev, min_bytes=1)
    with _on(dev):
        stream = _stream(dev)
        st = L_.mamba_block_fwd(_ptr(hidden), _ptr(w_in), _ptr(conv_weight), _ptr(conv_bias),
                                _ptr(w_x), _ptr(w_dt), _ptr(dt_bias), _ptr(A), _ptr(D),
                                _ptr(w_out), _ptr(out), ctypes.byref(dm), _ptr(workspace),
                                ws_len, stream)
    _raise(st)
    return out


# ---------------------------------------------------------------------------- gated delta rule

def _token_stride(t, name, vec):
    """Elements between tokens of a (..., tokens, heads, values) tensor whose tokens lie at one
    stride, heads and values packed inside each; raises where the layout is another."""
    H, d = t.shape[-2:]
    if t.dim() == 4:
        batch, L = t.shape[:2]
        stride = t.stride(1) if L > 1 else t.stride(0) if batch > 1 else H * d
        one = L == 1 or batch == 1 or t.stride(0) == L * stride
    else:
        stride = t.stride(0) if t.shape[0] > 1 else H * d
        one = True
    if (not one or (d > 1 and t.stride(-1) != 1) or (H > 1 and t.stride(-2) != d)
            or stride < H * d or stride % vec):
        raise ValueError(f"{name} must have packed heads and tokens at one stride, a multiple of "
                         f"{vec} elements; its strides are {tuple(t.stride())}")
    return stride


# The per-call part in native code (mamba_marshal.cpp): a call's tensors as one bytes key of their types,
# shapes, strides and devices, and their addresses handed to the entry point.  A key that has passed the
# checks below passes them again; its entry in _CHECKED holds the dims struct (read-only for the library),
# its address, the workspace size and the device.
_CHECKED = {}
_MARSHAL = None
(_DELTA_FWD, _DELTA_UPDATE, _DELTA_BWD, _GATED_FWD, _GATED_BWD, _ADD_FWD, _ADD_BWD, _QK_FWD,
 _QK_BWD, _LINEAR_FWD, _LINEAR_UPDATE, _LINEAR_BWD, _WINDOW_FWD, _WINDOW_BWD, _WINDOW_UPDATE,
 _WINDOW_STORE) = range(16)


def _marshal():
    """The native module (raises RuntimeError if it has not been built)."""
    global _MARSHAL
    if _MARSHAL is None:
        lib()
        with _lock:
            path = _build.MARSHAL_PATH
            if not os.path.exists(path):
                raise RuntimeError(
                    f"native module {path} is missing: build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            spec = importlib.util.spec_from_file_location("mamba_marshal", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            if module.torch_version != torch.__version__:  # it reads torch's own structures
                raise RuntimeError(
                    f"native module {path} was built for torch {module.torch_version}, this is "
                    f"{torch.__version__}: build it again with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            _MARSHAL = module
    return _MARSHAL


class _Entry:
    """What a checked call needs again."""
    __slots__ = ("dims", "address", "workspace_bytes", "device", "index", "factor", "extra")

    def __init__(self, dims, workspace_bytes, device, factor=0.0, extra=None):
        self.dims, self.address = dims, ctypes.addressof(dims)
        self.workspace_bytes, self.device, self.index = workspace_bytes, device, device.index
        self.factor, self.extra = factor, extra


def _remember(key, entry):
    if len(_CHECKED) >= 2048:
        _CHECKED.clear()
    _CHECKED[key] = entry
    return entry


# device that a launch would go to, without torch.cuda's own checks (a host-side cost per call)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(which, e, factor, ws_len, *tensors):
    """The entry point on the entry's device and its current stream; raises what the library refuses."""
    if _current_device() == e.index:
        st = _MARSHAL.call(which, e.address, _stream(e.device), factor, ws_len, *tensors)
    else:
        with torch.cuda.device(e.device):
            st = _MARSHAL.call(which, e.address, _stream(e.device), factor, ws_len, *tensors)
    if st:
        _raise(st)


def _scratch(workspace, like, e):
    """The caller's workspace, checked, or a new one on like's device: (tensor, its size in bytes)."""
    if workspace is not None:
        return _workspace(workspace, e.workspace_bytes, e.device)
    n = e.workspace_bytes or 1
    return _MARSHAL.empty(like, "b", n), n


def _delta_check(q, k, v, g, beta, others, seq_offsets, lead, workspace_bytes):
    """The entry of a delta rule's call on these tensors (_mixer_check with g and beta of the io dtype)."""
    return _mixer_check(q, k, v, ((g, "g", None), (beta, "beta", None)), others, seq_offsets, lead,
                        workspace_bytes)


def _mixer_check(q, k, v, gates, others, seq_offsets, lead, workspace_bytes):
    """The entry of a call on these tensors; raises for tensors that do not belong together.  `gates`:
    (tensor, name, dtype or None for the io dtype) of a number per token and value head; `others`:
    (tensor or None, name, shape function of (states, *token axes), Hk, Hv, dk, dv, dtype or None for
    the io dtype); lead: token axes of q; workspace_bytes: the library's query, or None."""
    n_seq = _offsets_count(seq_offsets, q)
    packed = n_seq is not None
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != lead + 2:
            raise ValueError(f"{name} must have {lead + 2} dimensions, it has shape "
                             f"{tuple(t.shape)}")
        if t.device != q.device or t.dtype != q.dtype or t.layout != torch.strided:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, q {q.dtype} on {q.device}")
    if q.device.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io, dev = q.dtype, q.device
    code = _io_code(io)
    tokens, (Hk, dk), (Hv, dv) = q.shape[:lead], q.shape[lead:], v.shape[lead:]
    if k.shape != q.shape or v.shape[:lead] != tokens:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not "
                         "belong together")
    if Hk == 0 or Hv % Hk:
        raise ValueError(f"{Hv} value heads are no multiple of {Hk} key heads")
    for t, name, dt in gates:
        if t is None:
            raise ValueError(f"{name} is required")
        _check(t, name, (*tokens, Hv), dt or io, dev)
    vec = 8 if code == MAMBA_BF16 else 4
    if packed:
        batch, L = n_seq, tokens[0]
    elif lead == 1:  # one token per sequence
        batch, L = tokens[0], 1
    else:
        batch, L = tokens
    for t, name, shape, dt in others:
        _check(t, name, shape((batch, *tokens), Hk, Hv, dk, dv), dt or io, dev)
    dm = mamba_delta_dims(batch, L, Hk, Hv, dk, dv, _token_stride(q, "q", vec),
                          _token_stride(k, "k", vec), _token_stride(v, "v", vec), code, 0)
    need = 0 if workspace_bytes is None else int(workspace_bytes(ctypes.byref(dm), int(packed)))
    return _Entry(dm, need, dev, dk ** -0.5 if dk else 0.0)


def _state_shape(n, Hk, Hv, dk, dv):
    return (n[0], Hv, dk, dv)


def _out_shape(n, Hk, Hv, dk, dv):
    return (*n[1:], Hv, dv)


def _offsets_count(seq_offsets, q):
    """Number of packed sequences of a (n + 1) int64 offsets tensor; None without one."""
    if seq_offsets is None:
        return None
    if not isinstance(seq_offsets, torch.Tensor) or not isinstance(q, torch.Tensor):
        raise TypeError("q and seq_offsets must be torch.Tensors")
    if (seq_offsets.dim() != 1 or seq_offsets.numel() < 2 or seq_offsets.dtype != torch.int64
            or seq_offsets.device != q.device or not seq_offsets.is_contiguous()):
        raise ValueError("seq_offsets must be a contiguous (sequences + 1,) int64 tensor on "
                         f"{q.device}")
    return seq_offsets.numel() - 1


def mamba_delta_workspace_bytes(dims: mamba_delta_dims, packed=False) -> int:
    return int(lib().mamba_delta_workspace_bytes(ctypes.byref(dims), int(bool(packed))))


def mamba_delta_fwd(q, k, v, g, beta, scale=None, initial_state=None, seq_offsets=None,
                    return_last_state=False, out=None, last_state=None, workspace=None):
    """The gated delta rule over whole sequences (mamba_delta_fwd in include/mamba_scan.h).

    q, k: (batch, L, Hk, dk); v: (batch, L, Hv, dv); g (log decay), beta: (batch, L, Hv) -- all
    float32 or all bfloat16; q, k and v may be slices of one projection's rows.  scale defaults to
    dk ** -0.5.  initial_state: (batch, Hv, dk, dv) float32.  With seq_offsets, an (n + 1,) int64
    tensor on the device, the token tensors have no batch axis: (tokens, H, d), sequence s being
    tokens seq_offsets[s] .. seq_offsets[s + 1] - 1, and there are n states.
    Returns out (batch, L, Hv, dv), or (out, last_state).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_DELTA_FWD, q, k, v, g, beta, initial_state, seq_offsets, out, last_state)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _delta_check(
            q, k, v, g, beta, ((initial_state, "initial_state", _state_shape, torch.float32),
                               (out, "out", _out_shape, None),
                               (last_state, "last_state", _state_shape, torch.float32)),
            seq_offsets, 2 if seq_offsets is None else 1, lib().mamba_delta_workspace_bytes))
    if out is None:
        out = m.empty(v)
    if return_last_state and last_state is None:
        dm = e.dims
        last_state = m.empty(q, "f", dm.batch, dm.v_heads, dm.dk, dm.dv)
    workspace, ws_len = _scratch(workspace, q, e)
    _call(_DELTA_FWD, e, e.factor if scale is None else scale, ws_len, q, k, v, g, beta,
          initial_state, seq_offsets, out, last_state, workspace)
    return (out, last_state) if return_last_state else out


def mamba_delta_update(state, q, k, v, g, beta, scale=None, out=None):
    """One generation step of the gated delta rule (mamba_delta_update in include/mamba_scan.h).

    state: (batch, Hv, dk, dv) float32, updated in place; q, k: (batch, Hk, dk); v: (batch, Hv, dv);
    g, beta: (batch, Hv).  Returns out (batch, Hv, dv).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_DELTA_UPDATE, state, q, k, v, g, beta, out)
    e = _CHECKED.get(key)
    if e is None:
        if state is None:
            raise ValueError("state is required")
        e = _remember(key, _delta_check(q, k, v, g, beta,
                                        ((state, "state", _state_shape, torch.float32),
                                         (out, "out", _out_shape, None)), None, 1, None))
    if out is None:
        out = m.empty(v)
    _call(_DELTA_UPDATE, e, e.factor if scale is None else scale, 0, state, q, k, v, g, beta, out)
    return out


def _qk_shape(n, Hk, Hv, dk, dv):
    return (*n[1:], Hk, dk)


def _head_shape(n, Hk, Hv, dk, dv):
    return (*n[1:], Hv)


def mamba_delta_bwd_workspace_bytes(dims: mamba_delta_dims, packed=False) -> int:
    return int(lib().mamba_delta_bwd_workspace_bytes(ctypes.byref(dims), int(bool(packed))))


_DELTA_GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")


def mamba_delta_bwd(q, k, v, g, beta, dout, scale=None, initial_state=None, seq_offsets=None,
                    dlast=None, workspace=None, grads=None):
    """Gradients of mamba_delta_fwd (mamba_delta_bwd in include/mamba_scan.h).

    Same inputs as mamba_delta_fwd plus dout (like out) and optionally dlast (like last_state).
    Returns a dict with dq, dk, dv, dg, dbeta (io dtype, contiguous) and dinitial_state (float32;
    None when initial_state is None).  `grads` may hold preallocated output tensors under the same
    keys.
    """
    if dout is None:
        raise ValueError("dout is required")
    gr = dict(grads or {})
    given = [gr.get(name) for name in _DELTA_GRADS]
    m = _MARSHAL or _marshal()
    key = m.key(_DELTA_BWD, q, k, v, g, beta, initial_state, seq_offsets, dout, dlast, *given)
    e = _CHECKED.get(key)
    if e is None:
        spec = (_qk_shape, _qk_shape, _out_shape, _head_shape, _head_shape, _state_shape)
        e = _remember(key, _delta_check(
            q, k, v, g, beta,
            ((initial_state, "initial_state", _state_shape, torch.float32),
             (dout, "dout", _out_shape, None), (dlast, "dlast", _state_shape, torch.float32),
             *((t, name, shape, torch.float32 if name == "dinitial_state" else None)
               for t, name, shape in zip(given, _DELTA_GRADS, spec))),
            seq_offsets, 2 if seq_offsets is None else 1, lib().mamba_delta_bwd_workspace_bytes))
    for name, like in zip(_DELTA_GRADS, (q, q, v, g, beta, initial_state)):
        if gr.get(name) is None:
            gr[name] = None if like is None else m.empty(like)
    workspace, ws_len = _scratch(workspace, q, e)
    res = {name: gr[name] for name in _DELTA_GRADS}
    _call(_DELTA_BWD, e, e.factor if scale is None else scale, ws_len, q, k, v, g, beta,
          initial_state, seq_offsets, dout, dlast, *res.values(), workspace)
    return res


# ---------------------------------------------------------------------------- linear attention

def mamba_linear_attn_workspace_bytes(dims: mamba_delta_dims, packed=False) -> int:
    return int(lib().mamba_linear_attn_workspace_bytes(ctypes.byref(dims), int(bool(packed))))


def mamba_linear_attn_fwd(q, k, v, g, scale=None, initial_state=None, seq_offsets=None,
                          return_last_state=False, out=None, last_state=None, workspace=None):
    """Linear attention with a decay per head over whole sequences (mamba_linear_attn_fwd in
    include/mamba_scan.h).

    q, k: (batch, L, Hk, dk); v: (batch, L, Hv, dv) -- all float32 or all bfloat16, also slices of one
    projection's rows; g (log decay): (batch, L, Hv) float32.  scale, initial_state and seq_offsets as
    for mamba_delta_fwd.  Returns out (batch, L, Hv, dv), or (out, last_state).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_LINEAR_FWD, q, k, v, g, initial_state, seq_offsets, out, last_state)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _mixer_check(
            q, k, v, ((g, "g", torch.float32),),
            ((initial_state, "initial_state", _state_shape, torch.float32),
             (out, "out", _out_shape, None), (last_state, "last_state", _state_shape, torch.float32)),
            seq_offsets, 2 if seq_offsets is None else 1, lib().mamba_linear_attn_workspace_bytes))
    if out is None:
        out = m.empty(v)
    if return_last_state and last_state is None:
        dm = e.dims
        last_state = m.empty(q, "f", dm.batch, dm.v_heads, dm.dk, dm.dv)
    ws_len = 0
    if e.workspace_bytes or workspace is not None:
        workspace, ws_len = _scratch(workspace, q, e)
    _call(_LINEAR_FWD, e, e.factor if scale is None else scale, ws_len, q, k, v, g, initial_state,
          seq_offsets, out, last_state, workspace)
    return (out, last_state) if return_last_state else out


def mamba_linear_attn_update(state, q, k, v, g, scale=None, out=None):
    """One generation step of linear attention (mamba_linear_attn_update in include/mamba_scan.h).

    state: (batch, Hv, dk, dv) float32, updated in place; q, k: (batch, Hk, dk); v: (batch, Hv, dv);
    g: (batch, Hv) float32.  Returns out (batch, Hv, dv).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_LINEAR_UPDATE, state, q, k, v, g, out)
    e = _CHECKED.get(key)
    if e is None:
        if state is None:
            raise ValueError("state is required")
        e = _remember(key, _mixer_check(q, k, v, ((g, "g", torch.float32),),
                                        ((state, "state", _state_shape, torch.float32),
                                         (out, "out", _out_shape, None)), None, 1, None))
    if out is None:
        out = m.empty(v)
    _call(_LINEAR_UPDATE, e, e.factor if scale is None else scale, 0, state, q, k, v, g, out)
    return out


def mamba_linear_attn_bwd_workspace_bytes(dims: mamba_delta_dims, packed=False) -> int:
    return int(lib().mamba_linear_attn_bwd_workspace_bytes(ctypes.byref(dims), int(bool(packed))))


_LINEAR_GRADS = ("dq", "dk", "dv", "dg", "dinitial_state")


def mamba_linear_attn_bwd(q, k, v, g, dout, scale=None, initial_state=None, seq_offsets=None, dlast=None,
                          workspace=None, grads=None):
    """Gradients of mamba_linear_attn_fwd (mamba_linear_attn_bwd in include/mamba_scan.h).

    Same inputs as mamba_linear_attn_fwd plus dout (like out) and optionally dlast (like last_state).
    Returns a dict with dq, dk, dv (io dtype), dg (float32), all contiguous, and dinitial_state
    (float32; None when initial_state is None).  `grads` may hold preallocated output tensors under the
    same keys.
    """
    if dout is None:
        raise ValueError("dout is required")
    gr = dict(grads or {})
    given = [gr.get(name) for name in _LINEAR_GRADS]
    m = _MARSHAL or _marshal()
    key = m.key(_LINEAR_BWD, q, k, v, g, initial_state, seq_offsets, dout, dlast, *given)
    e = _CHECKED.get(key)
    if e is None:
        spec = (_qk_shape, _qk_shape, _out_shape, _head_shape, _state_shape)
        e = _remember(key, _mixer_check(
            q, k, v, ((g, "g", torch.float32),),
            ((initial_state, "initial_state", _state_shape, torch.float32),
             (dout, "dout", _out_shape, None), (dlast, "dlast", _state_shape, torch.float32),
             *((t, name, shape, torch.float32 if name in ("dg", "dinitial_state") else None)
               for t, name, shape in zip(given, _LINEAR_GRADS, spec))),
            seq_offsets, 2 if seq_offsets is None else 1, lib().mamba_linear_attn_bwd_workspace_bytes))
    for name, like in zip(_LINEAR_GRADS, (q, q, v, g, initial_state)):
        if gr.get(name) is None:
            gr[name] = None if like is None else m.empty(like)
    workspace, ws_len = _scratch(workspace, q, e)
    res = {name: gr[name] for name in _LINEAR_GRADS}
    _call(_LINEAR_BWD, e, e.factor if scale is None else scale, ws_len, q, k, v, g, initial_state,
          seq_offsets, dout, dlast, *res.values(), workspace)
    return res


# ---------------------------------------------------------------------------- window attention

def _window_check(q, k, v, window, sinks, seq_offsets, kv_offsets, others, lead, workspace_bytes=None):
    """The entry of a call on these tensors.  `others`: (tensor or None, name, "q", "kv" or "head", dtype
    or None for the io dtype); lead: token axes of q (2: batch and tokens; 1: packed tokens, or one token
    per sequence); workspace_bytes(dims): the library's query, or None."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != lead + 2:
            raise ValueError(f"{name} must have {lead + 2} dimensions, it has shape {tuple(t.shape)}")
        if t.device != q.device or t.dtype != q.dtype or t.layout != torch.strided:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, q {q.dtype} on {q.device}")
    if q.device.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    if isinstance(window, bool) or isinstance(sinks, bool) or not isinstance(window, int) or not isinstance(sinks, int):
        raise TypeError("window and sinks must be integers")
    if not 1 <= window <= 1 << 40 or not 0 <= sinks <= 1 << 40:
        raise ValueError(f"window must be in 1 .. 2^40 and sinks in 0 .. 2^40, not {window} and {sinks}")
    n_seq = _offsets_count(seq_offsets, q)
    if kv_offsets is not None and (n_seq is None or _offsets_count(kv_offsets, q) != n_seq):
        raise ValueError("kv_offsets needs seq_offsets of as many sequences")
    io, dev = q.dtype, q.device
    code = _io_code(io)
    (Hq, d), (Hk, dk) = q.shape[lead:], k.shape[lead:]
    if v.shape != k.shape or d != dk or (lead == 2 and k.shape[0] != q.shape[0]):
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not belong "
                         "together")
    if Hk == 0 or Hq % Hk:
        raise ValueError(f"{Hq} query heads are no multiple of {Hk} key heads")
    if n_seq is not None:
        if kv_offsets is None and k.shape[0] != q.shape[0]:
            raise ValueError(f"q has {q.shape[0]} tokens, k {k.shape[0]}: kv_offsets is required")
        batch, L, Lk = n_seq, q.shape[0], k.shape[0]
    elif lead == 1:
        if k.shape[0] != q.shape[0]:
            raise ValueError(f"q has {q.shape[0]} sequences, k {k.shape[0]}")
        batch, L, Lk = q.shape[0], 1, 1
    else:
        (batch, L), Lk = q.shape[:2], k.shape[1]
    shapes = dict(q=q.shape, kv=k.shape, head=q.shape[:-1], cache=(batch, window + sinks, Hk, d))
    for t, name, kind, dt in others:
        _check(t, name, tuple(shapes[kind]), dt or io, dev)
    vec = 8 if code == MAMBA_BF16 else 4
    dm = mamba_window_dims(batch, L, Lk, Hq, Hk, d, _token_stride(q, "q", vec), _token_stride(k, "k", vec),
                           _token_stride(v, "v", vec), window, sinks, code, 0)
    need = 0 if workspace_bytes is None else int(workspace_bytes(dm))
    return _Entry(dm, need, dev, d ** -0.5 if d else 0.0)


def mamba_window_attn_fwd(q, k, v, window, sinks=0, scale=None, seq_offsets=None, kv_offsets=None,
                          return_lse=False, out=None, lse=None):
    """Causal attention with a sliding window and sinks (mamba_window_attn_fwd in include/mamba_scan.h).

    q: (batch, L, Hq, dim); k, v: (batch, Lk, Hk, dim) -- all float32 or all bfloat16, also slices of one
    projection's rows; the queries are the last L of Lk tokens.  A query sees the `window` last keys up to
    its own and the first `sinks`; a window of Lk is plain causal attention.  scale defaults to
    dim ** -0.5.  With seq_offsets, an (n + 1,) int64 tensor on the device, the token tensors have no batch
    axis: (tokens, H, dim), sequence s being tokens seq_offsets[s] .. seq_offsets[s + 1] - 1, of k and v
    those of kv_offsets where it is given.
    Returns out (batch, L, Hq, dim), or (out, lse) with lse (batch, L, Hq) float32.
    """
    m = _MARSHAL or _marshal()
    key = m.key(_WINDOW_FWD, q, k, v, window, sinks, seq_offsets, kv_offsets, out, lse)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _window_check(q, k, v, window, sinks, seq_offsets, kv_offsets,
                                         ((out, "out", "q", None), (lse, "lse", "head", torch.float32)),
                                         2 if seq_offsets is None else 1))
    if out is None:
        out = m.empty(q)
    if return_lse and lse is None:
        lse = m.empty(q, "f", *q.shape[:-1])
    _call(_WINDOW_FWD, e, e.factor if scale is None else scale, 0, q, k, v, seq_offsets,
          seq_offsets if kv_offsets is None else kv_offsets, out, lse)
    return (out, lse) if return_lse else out


def mamba_window_attn_bwd_workspace_bytes(dims: mamba_window_dims, packed=False) -> int:
    return int(lib().mamba_window_attn_bwd_workspace_bytes(ctypes.byref(dims), int(bool(packed))))


_WINDOW_GRADS = ("dq", "dk", "dv")


def mamba_window_attn_bwd(q, k, v, out, lse, dout, window, sinks=0, scale=None, seq_offsets=None,
                          kv_offsets=None, workspace=None, grads=None):
    """Gradients of mamba_window_attn_fwd (mamba_window_attn_bwd in include/mamba_scan.h).

    Same inputs as mamba_window_attn_fwd plus its out and lse, and dout (like out).  Returns a dict with
    dq, dk and dv (io dtype, contiguous).  `grads` may hold preallocated output tensors under the same
    keys.
    """
    for t, name in ((out, "out"), (lse, "lse"), (dout, "dout")):
        if t is None:
            raise ValueError(f"{name} is required")
    gr = dict(grads or {})
    given = [gr.get(name) for name in _WINDOW_GRADS]
    m = _MARSHAL or _marshal()
    key = m.key(_WINDOW_BWD, q, k, v, window, sinks, seq_offsets, kv_offsets, out, lse, dout, *given)
    e = _CHECKED.get(key)
    if e is None:
        packed = seq_offsets is not None
        e = _remember(key, _window_check(
            q, k, v, window, sinks, seq_offsets, kv_offsets,
            ((out, "out", "q", None), (lse, "lse", "head", torch.float32), (dout, "dout", "q", None),
             *zip(given, _WINDOW_GRADS, ("q", "kv", "kv"), (None,) * 3)),
            1 if packed else 2, lambda dm: mamba_window_attn_bwd_workspace_bytes(dm, packed)))
    for name, like in zip(_WINDOW_GRADS, (q, k, v)):
        if gr.get(name) is None:
            gr[name] = m.empty(like)
    workspace, ws_len = _scratch(workspace, q, e)
    res = {name: gr[name] for name in _WINDOW_GRADS}
    _call(_WINDOW_BWD, e, e.factor if scale is None else scale, ws_len, q, k, v, seq_offsets,
          seq_offsets if kv_offsets is None else kv_offsets, out, lse, dout, *res.values(), workspace)
    return res


def _cache_window(k_cache, v_cache, sinks):
    """The window of a pair of ring caches."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be (batch, sinks + window, heads, dim), not {tuple(t.shape)}")
    if isinstance(sinks, bool) or not isinstance(sinks, int):
        raise TypeError("sinks must be an integer")
    return k_cache.shape[1] - sinks


def mamba_window_cache_store(k_cache, v_cache, k, v, sinks=0, seq_offsets=None):
    """Fills ring caches from the keys and values of whole sequences (mamba_window_cache_store in
    include/mamba_scan.h).

    k_cache, v_cache: (batch, sinks + window, Hk, dim), written in place; k, v: (batch, Lk, Hk, dim), or
    with seq_offsets (tokens, Hk, dim) as for mamba_window_attn_fwd.  Position p lies in slot p below
    `sinks`, in slot sinks + (p - sinks) % window from there on; slots without one keep what they hold.
    """
    m = _MARSHAL or _marshal()
    key = m.key(_WINDOW_STORE, k_cache, v_cache, k, v, sinks, seq_offsets)
    e = _CHECKED.get(key)
    if e is None:
        window = _cache_window(k_cache, v_cache, sinks)
        e = _remember(key, _window_check(k, k, v, window, sinks, seq_offsets, None,
                                         ((k_cache, "k_cache", "cache", None),
                                          (v_cache, "v_cache", "cache", None)),
                                         2 if seq_offsets is None else 1))
    _call(_WINDOW_STORE, e, 0.0, 0, k, v, seq_offsets, k_cache, v_cache)


def mamba_window_attn_update_workspace_bytes(dims: mamba_window_dims) -> int:
    return int(lib().mamba_window_attn_update_workspace_bytes(ctypes.byref(dims)))


def mamba_window_attn_update(k_cache, v_cache, q, k, v, positions, sinks=0, scale=None, out=None,
                             workspace=None):
    """One generation step of window attention (mamba_window_attn_update in include/mamba_scan.h).

    k_cache, v_cache: (batch, sinks + window, Hk, dim), updated in place; q: (batch, Hq, dim); k, v:
    (batch, Hk, dim); positions: (batch,) int64, the tokens before the new one (below zero: no token, a
    row of zeros).  Returns out (batch, Hq, dim).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_WINDOW_UPDATE, k_cache, v_cache, q, k, v, positions, sinks, out)
    e = _CHECKED.get(key)
    if e is None:
        window = _cache_window(k_cache, v_cache, sinks)
        e = _window_check(q, k, v, window, sinks, None, None,
                          ((k_cache, "k_cache", "cache", None), (v_cache, "v_cache", "cache", None),
                           (out, "out", "q", None)), 1, mamba_window_attn_update_workspace_bytes)
        if positions is None:
            raise ValueError("positions is required")
        _check(positions, "positions", (q.shape[0],), torch.int64, q.device)
        _remember(key, e)
    if out is None:
        out = m.empty(q)
    ws_len = 0
    if e.workspace_bytes or workspace is not None:
        workspace, ws_len = _scratch(workspace, q, e)
    _call(_WINDOW_UPDATE, e, e.factor if scale is None else scale, ws_len, k_cache, v_cache, q, k, v,
          positions, out, workspace)
    return out


# ---------------------------------------------------------------------------- norms of a block

def _row_stride(t, name):
    """Elements between the rows of a (rows, groups, dim) tensor, packed inside each row."""
    rows, G, d = t.shape
    stride = t.stride(0) if rows > 1 else G * d
    if (d > 1 and t.stride(2) != 1) or (G > 1 and t.stride(1) != d) or stride < G * d:
        raise ValueError(f"{name} must have packed rows; its strides are {tuple(t.stride())}")
    return stride


def _gated_check(y, z, weight, gate_first, others):
    """The entry of a gated norm; `others`: (tensor or None, name, "rows" or "weight")."""
    for t, name in ((y, "y"), (weight, "weight")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if y.dim() != 3 or y.device.type != "cuda" or y.layout != torch.strided:
        raise ValueError("y must be (rows, groups, dim) on a HIP device")
    rows, G, d = y.shape
    io, dev = y.dtype, y.device
    code = _io_code(io)
    if z is not None:
        if not isinstance(z, torch.Tensor):
            raise TypeError("z must be a torch.Tensor")
        if z.shape != y.shape or z.dtype != io or z.device != dev or z.layout != torch.strided:
            raise ValueError(f"z must be like y, {tuple(y.shape)} {io} on {dev}")
    per_group = weight.dim() == 2
    wshape = (G, d) if per_group else (d,)
    _check(weight, "weight", wshape, torch.float32, dev)
    for t, name, kind in others:
        if kind == "weight":
            _check(t, name, wshape, torch.float32, dev)
        else:
            _check(t, name, (rows, G, d), io, dev)
    dm = mamba_gated_norm_dims(rows, G, d, _row_stride(y, "y"),
                               0 if z is None else _row_stride(z, "z"), code,
                               G if per_group else 1, int(bool(gate_first)), 0)
    return _Entry(dm, mamba_gated_norm_bwd_workspace_bytes(dm), dev)


def mamba_gated_norm_bwd_workspace_bytes(dims: mamba_gated_norm_dims) -> int:
    return int(lib().mamba_gated_norm_bwd_workspace_bytes(ctypes.byref(dims)))


def mamba_gated_norm_fwd(y, z, weight, eps=1e-5, gate_first=False, out=None):
    """RMS norm per group with a silu gate (mamba_gated_norm_fwd in include/mamba_scan.h).

    y, z: (rows, groups, dim) float32 or bfloat16, rows at any stride (z None: no gate); weight:
    (dim,) or (groups, dim) float32.  norm(y) * weight * silu(z), or norm(y * silu(z)) * weight with
    gate_first.  Returns out (rows, groups, dim).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_GATED_FWD, y, z, weight, bool(gate_first), out)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _gated_check(y, z, weight, gate_first, ((out, "out", "rows"),)))
    if out is None:
        out = m.empty(y)
    _call(_GATED_FWD, e, eps, 0, y, z, weight, out)
    return out


def mamba_gated_norm_bwd(y, z, weight, dout, eps=1e-5, gate_first=False, workspace=None,
                         grads=None):
    """Gradients of mamba_gated_norm_fwd: a dict with dy, dz (None without z) and dweight.  `grads`
    may hold preallocated output tensors under the same keys."""
    if dout is None:
        raise ValueError("dout is required")
    g = dict(grads or {})
    given = [g.get(name) for name in ("dy", "dz", "dweight")]
    m = _MARSHAL or _marshal()
    key = m.key(_GATED_BWD, y, z, weight, bool(gate_first), dout, *given)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _gated_check(y, z, weight, gate_first,
                                        ((dout, "dout", "rows"), (given[0], "dy", "rows"),
                                         (given[1], "dz", "rows"),
                                         (given[2], "dweight", "weight"))))
    dy, dz, dw = given
    if dy is None:
        dy = m.empty(y)
    if z is None:
        dz = None
    elif dz is None:
        dz = m.empty(y)
    if dw is None:
        dw = m.empty(weight)
    workspace, ws_len = _scratch(workspace, y, e)
    _call(_GATED_BWD, e, eps, ws_len, y, z, weight, dout, dy, dz, dw, workspace)
    return {"dy": dy, "dz": dz, "dweight": dw}


def _add_check(x, residual, vectors, others):
    """The entry of an add norm (extra: the residual's type).  `vectors`: (tensor or None, name) of
    (dim,) float32; `others`: (tensor or None, name, is of the residual's type)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() != 2 or x.device.type != "cuda":
        raise ValueError("x must be (rows, dim) on a HIP device")
    rows, d = x.shape
    io, dev = x.dtype, x.device
    code = _io_code(io)
    _check(x, "x", (rows, d), io, dev)
    # the stream's type is the residual's, or that of the first of its companions
    res = next((t.dtype for t, _, r in ((residual, "", True), *others)
                if r and isinstance(t, torch.Tensor)), io)
    res_code = _io_code(res)
    _check(residual, "residual", (rows, d), res, dev)
    if vectors[0][0] is None:
        raise ValueError("weight is required")
    for t, name in vectors:
        _check(t, name, (d,), torch.float32, dev)
    for t, name, of_res in others:
        _check(t, name, (rows, d), res if of_res else io, dev)
    dm = mamba_add_norm_dims(rows, d, code, res_code)
    return _Entry(dm, mamba_add_norm_bwd_workspace_bytes(dm), dev, extra=res)


def mamba_add_norm_bwd_workspace_bytes(dims: mamba_add_norm_dims) -> int:
    return int(lib().mamba_add_norm_bwd_workspace_bytes(ctypes.byref(dims)))


def mamba_add_norm_fwd(x, residual, weight, scale=None, post_weight=None, eps=1e-5, out=None,
                       residual_out=None):
    """The join of two blocks (mamba_add_norm_fwd in include/mamba_scan.h): r = residual + scale *
    x (or norm(x) * post_weight in place of x), out = norm(r) * weight.

    x: (rows, dim) float32 or bfloat16; residual: (rows, dim) of x's type or float32 (None: zero);
    weight, scale, post_weight: (dim,) float32.  Returns (out, r), r of the residual's type (of x's
    without one, or of residual_out's).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_ADD_FWD, x, residual, weight, scale, post_weight, out, residual_out)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _add_check(x, residual, ((weight, "weight"), (scale, "scale"),
                                                    (post_weight, "post_weight")),
                                      ((out, "out", False),
                                       (residual_out, "residual_out", True))))
    if out is None:
        out = m.empty(x)
    if residual_out is None:
        residual_out = m.empty(x if residual is None else residual)
    _call(_ADD_FWD, e, eps, 0, x, residual, weight, scale, post_weight, out, residual_out)
    return out, residual_out


_ADD_GRADS = ("dx", "dresidual", "dweight", "dscale", "dpost_weight")


def mamba_add_norm_bwd(x, residual, weight, dout, dresidual_out=None, scale=None, post_weight=None,
                       eps=1e-5, workspace=None, grads=None):
    """Gradients of mamba_add_norm_fwd for the loss sum(out * dout) + sum(r * dresidual_out): a dict
    with dx, dresidual (None without a residual), dweight, dscale and dpost_weight (None without
    theirs).  x and residual are the forward's inputs.  `grads` may hold preallocated output tensors
    under the same keys."""
    if dout is None:
        raise ValueError("dout is required")
    g = dict(grads or {})
    given = [g.get(name) for name in _ADD_GRADS]
    m = _MARSHAL or _marshal()
    key = m.key(_ADD_BWD, x, residual, weight, scale, post_weight, dout, dresidual_out, *given)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _add_check(
            x, residual, ((weight, "weight"), (scale, "scale"), (post_weight, "post_weight"),
                          *zip(given[2:], _ADD_GRADS[2:])),
            ((dout, "dout", False), (dresidual_out, "dresidual_out", True),
             (given[0], "dx", False), (given[1], "dresidual", True))))
    for name, like in zip(_ADD_GRADS, (x, residual, weight, scale, post_weight)):
        if like is None:
            g[name] = None
        elif g.get(name) is None:
            g[name] = m.empty(like)
    workspace, ws_len = _scratch(workspace, x, e)
    res = {name: g[name] for name in _ADD_GRADS}
    _call(_ADD_BWD, e, eps, ws_len, x, residual, weight, scale, post_weight, dout, dresidual_out,
          *res.values(), workspace)
    return res


# ---------------------------------------------------------------------------- norm of queries and keys

def _qk_check(q, k, q_weight, k_weight, positions, inv_freq, interleaved, others):
    """The entry of a norm of queries and keys; `others`: (tensor or None, name, "q", "k" or "weight")."""
    for t, name in ((q, "q"), (k, "k"), (q_weight, "q_weight"), (k_weight, "k_weight")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if q.dim() != 3 or q.device.type != "cuda" or q.layout != torch.strided:
        raise ValueError("q must be (rows, heads, dim) on a HIP device")
    io, dev = q.dtype, q.device
    code = _io_code(io)
    rows, Hq, d = q.shape
    if (k.dim() != 3 or k.dtype != io or k.device != dev or k.layout != torch.strided
            or k.shape[0] != rows or k.shape[2] != d):
        raise ValueError(f"k must be ({rows}, heads, {d}) {io} on {dev}")
    Hk = k.shape[1]
    rot = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a (rotary_dim / 2,) tensor")
        rot = 2 * inv_freq.shape[0]
        _check(inv_freq, "inv_freq", (rot // 2,), torch.float64, dev)
        if positions is None:
            raise ValueError("positions is required")
    _check(positions, "positions", (rows,), torch.int64, dev)
    _check(q_weight, "q_weight", (d,), torch.float32, dev)
    _check(k_weight, "k_weight", (d,), torch.float32, dev)
    for t, name, kind in others:
        if kind == "weight":
            _check(t, name, (d,), torch.float32, dev)
        else:
            _check(t, name, (rows, Hq if kind == "q" else Hk, d), io, dev)
    vec = 8 if code == MAMBA_BF16 else 4
    strides = []
    for t, name in ((q, "q"), (k, "k")):
        stride = _row_stride(t, name)
        if stride % vec:
            raise ValueError(f"{name} must have rows at a multiple of {vec} elements; its strides are "
                             f"{tuple(t.stride())}")
        strides.append(stride)
    dm = mamba_qk_norm_rope_dims(rows, Hq, Hk, d, rot, *strides, code, int(bool(interleaved)))
    return _Entry(dm, mamba_qk_norm_rope_bwd_workspace_bytes(dm), dev)


def mamba_qk_norm_rope_bwd_workspace_bytes(dims: mamba_qk_norm_rope_dims) -> int:
    return int(lib().mamba_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(dims)))


def mamba_qk_norm_rope_fwd(q, k, q_weight, k_weight, positions=None, inv_freq=None, eps=1e-5,
                           interleaved=False, q_out=None, k_out=None):
    """RMS norm of queries and keys per head and the rotation by position (mamba_qk_norm_rope_fwd in
    include/mamba_scan.h).

    q: (rows, Hq, dim), k: (rows, Hk, dim) float32 or bfloat16, rows at any stride of 16 bytes;
    q_weight, k_weight: (dim,) float32; positions: (rows,) int64; inv_freq: (rotary_dim / 2,) float64,
    radians per position (None: no rotation).  Value i turns with i + rotary_dim / 2, or with
    interleaved 2 i with 2 i + 1.  Returns (q_out, k_out).
    """
    m = _MARSHAL or _marshal()
    key = m.key(_QK_FWD, q, k, q_weight, k_weight, positions, inv_freq, bool(interleaved), q_out, k_out)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _qk_check(q, k, q_weight, k_weight, positions, inv_freq, interleaved,
                                     ((q_out, "q_out", "q"), (k_out, "k_out", "k"))))
    if q_out is None:
        q_out = m.empty(q)
    if k_out is None:
        k_out = m.empty(k)
    _call(_QK_FWD, e, eps, 0, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out)
    return q_out, k_out


_QK_GRADS = ("dq", "dk", "dq_weight", "dk_weight")


def mamba_qk_norm_rope_bwd(q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, eps=1e-5,
                           interleaved=False, workspace=None, grads=None):
    """Gradients of mamba_qk_norm_rope_fwd for the loss sum(q_out * dq_out) + sum(k_out * dk_out): a dict
    with dq, dk, dq_weight and dk_weight.  `grads` may hold preallocated output tensors under the same
    keys."""
    if dq_out is None or dk_out is None:
        raise ValueError("dq_out and dk_out are required")
    g = dict(grads or {})
    given = [g.get(name) for name in _QK_GRADS]
    m = _MARSHAL or _marshal()
    key = m.key(_QK_BWD, q, k, q_weight, k_weight, positions, inv_freq, bool(interleaved), dq_out, dk_out,
                *given)
    e = _CHECKED.get(key)
    if e is None:
        e = _remember(key, _qk_check(
            q, k, q_weight, k_weight, positions, inv_freq, interleaved,
            ((dq_out, "dq_out", "q"), (dk_out, "dk_out", "k"),
             *zip(given, _QK_GRADS, ("q", "k", "weight", "weight")))))
    for name, like in zip(_QK_GRADS, (q, k, q_weight, k_weight)):
        if g.get(name) is None:
            g[name] = m.empty(like)
    workspace, ws_len = _scratch(workspace, q, e)
    res = {name: g[name] for name in _QK_GRADS}
    _call(_QK_BWD, e, eps, ws_len, q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out,
          *res.values(), workspace)
    return res
