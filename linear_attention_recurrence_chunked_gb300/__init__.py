"""Thin Python binding of the GB300 causal linear-attention library.

Every function here marshals torch tensors into the C ABI of ``include/la.h``
and calls it; all arithmetic runs in the library's CUDA kernels.  There is no
CPU or PyTorch fallback: if the compiled library is missing, importing the
binding's functions raises.

Names follow the C entry points: ``la_based_prefill``, ``la_gdn_prefill``,
``la_decode_step`` (plus the workspace queries and status helpers).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

from . import _build

LA_OK = 0
LA_ERR_INVALID_ARGUMENT = 1
LA_ERR_UNSUPPORTED = 2
LA_ERR_WORKSPACE = 3
LA_ERR_CUDA = 4
LA_ERR_TIMEOUT = 5

LA_DTYPE_F32 = 0
LA_DTYPE_BF16 = 1
LA_VARIANT_TAYLOR = 0
LA_VARIANT_GDN = 1
LA_VARIANT_GATED = 2

TAYLOR_DFEAT = 16
TAYLOR_DV = 64
TAYLOR_D = 1 + TAYLOR_DFEAT + TAYLOR_DFEAT * TAYLOR_DFEAT
GDN_D = 128

_i64 = ctypes.c_int64


class LATensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", _i64), ("stride_h", _i64), ("stride_t", _i64)]


class BasedPrefillArgs(ctypes.Structure):
    _fields_ = [("B", _i64), ("H", _i64), ("N", _i64), ("d_feat", _i64), ("d_v", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("q", LATensor), ("k", LATensor), ("v", LATensor), ("y", LATensor),
                ("s_in", ctypes.c_void_p), ("z_in", ctypes.c_void_p),
                ("s_out", ctypes.c_void_p), ("z_out", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("decay", ctypes.c_void_p)]


class GdnPrefillArgs(ctypes.Structure):
    _fields_ = [("B", _i64), ("H", _i64), ("N", _i64), ("d_k", _i64), ("d_v", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("q", LATensor), ("k", LATensor), ("v", LATensor), ("o", LATensor),
                ("alpha", LATensor), ("beta", LATensor),
                ("q_scale", ctypes.c_float),
                ("S_in", ctypes.c_void_p), ("S_out", ctypes.c_void_p)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int), ("S", _i64), ("H", _i64), ("d_k", _i64), ("d_v", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("state", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("q_scale", ctypes.c_float), ("decay", ctypes.c_void_p)]


EXPORTED = ("la_based_prefill", "la_gdn_prefill", "la_gated_prefill", "la_decode_step", "la_based_prefill_workspace_size",
            "la_gdn_prefill_workspace_size", "la_gdn_prefill_workspace_size_min", "la_gdn_prefill_noalloc", "la_device_status",
            "la_state_rescale", "la_state_gather", "la_swa_decode_step", "la_notebank_scores", "la_notebank_address",
            "la_notebank_route", "la_conv_prefill", "la_conv_decode_step", "la_ssm_prefill_workspace_size", "la_ssm_prefill",
            "la_ssm_decode_step", "la_swa_prefill", "la_swa_biased_decode_step", "la_selftest_bounded_wait", "la_status_string", "la_abi_version",
            "la_last_cuda_error", "la_cuda_error_name")


class NotebankScoresArgs(ctypes.Structure):
    _fields_ = [("L", _i64), ("H", _i64), ("N", _i64), ("d", _i64), ("in_dtype", ctypes.c_int),
                ("k", LATensor), ("chunk", _i64), ("window", _i64),
                ("d_ch", ctypes.c_void_p), ("d_mean", ctypes.c_void_p), ("w", ctypes.c_void_p)]


class NotebankAddressArgs(ctypes.Structure):
    _fields_ = [("L", _i64), ("H", _i64), ("N", _i64), ("d", _i64), ("n_notes", _i64), ("in_dtype", ctypes.c_int),
                ("q", LATensor), ("d_ch", ctypes.c_void_p), ("coords", ctypes.c_void_p), ("spans", ctypes.c_void_p),
                ("t_star", ctypes.c_void_p), ("rho", ctypes.c_void_p)]


class NotebankRouteArgs(ctypes.Structure):
    _fields_ = [("n_notes", _i64), ("J", _i64), ("n_q", _i64), ("R", _i64),
                ("rho", ctypes.c_void_p), ("u", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("s", ctypes.c_void_p), ("winner", ctypes.c_void_p), ("votes", ctypes.c_void_p),
                ("top", ctypes.c_void_p)]


class SwaDecodeArgs(ctypes.Structure):
    _fields_ = [("S", _i64), ("H", _i64), ("d", _i64), ("window", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("scale", ctypes.c_float)]


class ConvPrefillArgs(ctypes.Structure):
    _fields_ = [("B", _i64), ("N", _i64), ("C", _i64), ("W", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
                ("x", LATensor), ("y", LATensor), ("w", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("state_in", ctypes.c_void_p), ("state_out", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("silu", ctypes.c_int32), ("fill", ctypes.c_int32)]


class ConvDecodeArgs(ctypes.Structure):
    _fields_ = [("S", _i64), ("C", _i64), ("W", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
                ("x", ctypes.c_void_p), ("x_stride", _i64), ("out", ctypes.c_void_p), ("out_stride", _i64),
                ("w", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("state_in", ctypes.c_void_p), ("state_out", ctypes.c_void_p), ("silu", ctypes.c_int32)]


class SsmPrefillArgs(ctypes.Structure):
    _fields_ = [("B", _i64), ("N", _i64), ("C", _i64), ("n", _i64), ("G", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("u", LATensor), ("delta", LATensor), ("z", LATensor), ("y", LATensor),
                ("Bm", LATensor), ("Cm", LATensor),
                ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("delta_bias", ctypes.c_void_p),
                ("h_in", ctypes.c_void_p), ("h_out", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("delta_softplus", ctypes.c_int32), ("fill", ctypes.c_int32)]


class SsmDecodeArgs(ctypes.Structure):
    _fields_ = [("S", _i64), ("C", _i64), ("n", _i64), ("G", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("u", LATensor), ("delta", LATensor), ("z", LATensor), ("out", LATensor),
                ("Bm", LATensor), ("Cm", LATensor),
                ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("delta_bias", ctypes.c_void_p),
                ("state_in", ctypes.c_void_p), ("state_out", ctypes.c_void_p), ("delta_softplus", ctypes.c_int32)]


class SwaPrefillArgs(ctypes.Structure):
    _fields_ = [("B", _i64), ("H", _i64), ("H_kv", _i64), ("Nq", _i64), ("Nk", _i64), ("d", _i64), ("window", _i64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("q", LATensor), ("k", LATensor), ("v", LATensor), ("o", LATensor),
                ("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("key_lo", ctypes.c_void_p), ("key_hi", ctypes.c_void_p), ("q_pos0", _i64), ("lens", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("fill", ctypes.c_int32)]


class SwaBiasedDecodeArgs(ctypes.Structure):
    _fields_ = [("base", SwaDecodeArgs), ("H_kv", _i64), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p)]


class LAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {la_status_string(status)} (status {status})"
        if status == LA_ERR_CUDA:
            lib = load_library()
            code = int(lib.la_last_cuda_error())
            msg += f"; CUDA error {code} ({lib.la_cuda_error_name(code).decode()})"
        super().__init__(msg)


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library(path: str | None = None):
    """Load the compiled library (build it first with ``_build.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built ({p} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    vp = ctypes.c_void_p
    lib.la_based_prefill.restype = ctypes.c_int
    lib.la_based_prefill.argtypes = [ctypes.POINTER(BasedPrefillArgs), vp, ctypes.c_size_t, vp]
    lib.la_gdn_prefill.restype = ctypes.c_int
    lib.la_gdn_prefill.argtypes = [ctypes.POINTER(GdnPrefillArgs), vp, ctypes.c_size_t, vp]
    lib.la_gated_prefill.restype = ctypes.c_int
    lib.la_gated_prefill.argtypes = [ctypes.POINTER(GdnPrefillArgs), vp, ctypes.c_size_t, vp]
    lib.la_gdn_prefill_noalloc.restype = ctypes.c_int
    lib.la_gdn_prefill_noalloc.argtypes = [ctypes.POINTER(GdnPrefillArgs), vp]
    lib.la_decode_step.restype = ctypes.c_int
    lib.la_decode_step.argtypes = [ctypes.POINTER(DecodeArgs), vp]
    lib.la_based_prefill_workspace_size.restype = ctypes.c_size_t
    lib.la_based_prefill_workspace_size.argtypes = [ctypes.POINTER(BasedPrefillArgs)]
    lib.la_gdn_prefill_workspace_size.restype = ctypes.c_size_t
    lib.la_gdn_prefill_workspace_size.argtypes = [ctypes.POINTER(GdnPrefillArgs)]
    lib.la_gdn_prefill_workspace_size_min.restype = ctypes.c_size_t
    lib.la_gdn_prefill_workspace_size_min.argtypes = [ctypes.POINTER(GdnPrefillArgs)]
    lib.la_swa_decode_step.restype = ctypes.c_int
    lib.la_swa_decode_step.argtypes = [ctypes.POINTER(SwaDecodeArgs), vp]
    lib.la_notebank_scores.restype = ctypes.c_int
    lib.la_notebank_scores.argtypes = [ctypes.POINTER(NotebankScoresArgs), vp]
    lib.la_notebank_address.restype = ctypes.c_int
    lib.la_notebank_address.argtypes = [ctypes.POINTER(NotebankAddressArgs), vp]
    lib.la_notebank_route.restype = ctypes.c_int
    lib.la_notebank_route.argtypes = [ctypes.POINTER(NotebankRouteArgs), vp]
    lib.la_conv_prefill.restype = ctypes.c_int
    lib.la_conv_prefill.argtypes = [ctypes.POINTER(ConvPrefillArgs), vp]
    lib.la_conv_decode_step.restype = ctypes.c_int
    lib.la_conv_decode_step.argtypes = [ctypes.POINTER(ConvDecodeArgs), vp]
    lib.la_ssm_prefill_workspace_size.restype = ctypes.c_size_t
    lib.la_ssm_prefill_workspace_size.argtypes = [ctypes.POINTER(SsmPrefillArgs)]
    lib.la_ssm_prefill.restype = ctypes.c_int
    lib.la_ssm_prefill.argtypes = [ctypes.POINTER(SsmPrefillArgs), vp, ctypes.c_size_t, vp]
    lib.la_ssm_decode_step.restype = ctypes.c_int
    lib.la_ssm_decode_step.argtypes = [ctypes.POINTER(SsmDecodeArgs), vp]
    lib.la_swa_prefill.restype = ctypes.c_int
    lib.la_swa_prefill.argtypes = [ctypes.POINTER(SwaPrefillArgs), vp]
    lib.la_swa_biased_decode_step.restype = ctypes.c_int
    lib.la_swa_biased_decode_step.argtypes = [ctypes.POINTER(SwaBiasedDecodeArgs), vp]
    lib.la_state_rescale.restype = ctypes.c_int
    lib.la_state_rescale.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, vp, ctypes.c_float, vp]
    lib.la_state_gather.restype = ctypes.c_int
    lib.la_state_gather.argtypes = [vp, vp, vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp]
    lib.la_device_status.restype = ctypes.c_int
    lib.la_device_status.argtypes = [vp, ctypes.c_int]
    lib.la_selftest_bounded_wait.restype = ctypes.c_int
    lib.la_selftest_bounded_wait.argtypes = [ctypes.c_int, ctypes.c_int64, vp]
    lib.la_status_string.restype = ctypes.c_char_p
    lib.la_status_string.argtypes = [ctypes.c_int]
    lib.la_last_cuda_error.restype = ctypes.c_int
    lib.la_last_cuda_error.argtypes = []
    lib.la_cuda_error_name.restype = ctypes.c_char_p
    lib.la_cuda_error_name.argtypes = [ctypes.c_int]
    lib.la_abi_version.restype = ctypes.c_int
    lib.la_abi_version.argtypes = []
    if path is None:
        _lib = lib
    return lib


def la_status_string(status: int) -> str:
    return load_library().la_status_string(int(status)).decode()


def la_abi_version() -> int:
    return int(load_library().la_abi_version())


# ---------------------------------------------------------------------------
# marshalling helpers


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return LA_DTYPE_F32
    if t == torch.bfloat16:
        return LA_DTYPE_BF16
    raise TypeError(f"unsupported dtype {t}; use float32 or bfloat16")


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _view4(t: torch.Tensor) -> LATensor:
    """[B,H,N,d] tensor -> strided view (the d axis must be contiguous)."""
    if t.dim() != 4:
        raise ValueError(f"expected a [B,H,N,d] tensor, got shape {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the feature axis must be contiguous")
    return LATensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _gate3(t: torch.Tensor) -> LATensor:
    """[B,H,N] fp32 gate -> view with its N axis as the token axis."""
    if t.dim() != 3 or t.dtype != torch.float32:
        raise ValueError("alpha/beta must be float32 [B,H,N]")
    return LATensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _check_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must live on a CUDA device")


def _workspace(nbytes: int, workspace, device):
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, nbytes


# ---------------------------------------------------------------------------
# entry points


def _based_args(q, k, v, y, s_in, z_in, s_out, z_out, eps, decay=None):
    B, H, N, F = q.shape
    return BasedPrefillArgs(B, H, N, F, v.shape[-1], _dtype_code(q.dtype), _dtype_code(y.dtype),
                            _view4(q), _view4(k), _view4(v), _view4(y),
                            _ptr(s_in), _ptr(z_in), _ptr(s_out), _ptr(z_out), float(eps), _ptr(decay))


def _check_decay(decay, H):
    if decay is not None and (decay.dtype != torch.float32 or decay.shape != (H,) or not decay.is_contiguous()):
        raise ValueError("decay must be a contiguous float32 tensor of shape [H]")


def la_based_prefill_workspace_size(q, k, v, y=None) -> int:
    y = y if y is not None else v
    a = _based_args(q, k, v, y, None, None, None, None, 0.0)
    return int(load_library().la_based_prefill_workspace_size(ctypes.byref(a)))


def la_based_prefill(q, k, v, y=None, s_in=None, z_in=None, s_out=None, z_out=None, eps: float = 0.0,
                     out_dtype=None, workspace=None, stream=None, decay=None):
    """Chunked Taylor (BASED) prefill.  Returns (y, s_out, z_out).

    q, k: [B,H,N,16], v: [B,H,N,64] (fp32 or bf16); states fp32
    s: [B,H,273,64], z: [B,H,273]; decay: None or fp32 [H], the per-head
    retention lambda (s_i = lambda s_{i-1} + phi(k_i) v_i^T, z likewise)."""
    lib = load_library()
    _check_cuda(q, k, v, y, s_in, z_in, s_out, z_out, decay)
    B, H, N, _ = q.shape
    _check_decay(decay, H)
    dv = v.shape[-1]
    if y is None:
        y = torch.empty((B, H, N, dv), dtype=out_dtype or q.dtype, device=q.device)
    if s_out is None:
        s_out = torch.empty((B, H, TAYLOR_D, dv), dtype=torch.float32, device=q.device)
    if z_out is None:
        z_out = torch.empty((B, H, TAYLOR_D), dtype=torch.float32, device=q.device)
    for name, t in (("s_in", s_in), ("z_in", z_in), ("s_out", s_out), ("z_out", z_out)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor")
    a = _based_args(q, k, v, y, s_in, z_in, s_out, z_out, eps, decay)
    need = int(lib.la_based_prefill_workspace_size(ctypes.byref(a)))
    ws, ws_bytes = _workspace(need, workspace, q.device)
    st = lib.la_based_prefill(ctypes.byref(a), _ptr(ws) if isinstance(ws, torch.Tensor) else ws, ws_bytes,
                              _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_based_prefill")
    return y, s_out, z_out


def _gdn_args(q, k, v, o, alpha, beta, S_in, S_out, q_scale):
    B, H, N, dk = q.shape
    return GdnPrefillArgs(B, H, N, dk, v.shape[-1], _dtype_code(q.dtype), _dtype_code(o.dtype),
                          _view4(q), _view4(k), _view4(v), _view4(o), _gate3(alpha), _gate3(beta),
                          float(q_scale), _ptr(S_in), _ptr(S_out))


def la_gdn_prefill_workspace_size(q, k, v, alpha, beta, o=None) -> int:
    o = o if o is not None else v
    a = _gdn_args(q, k, v, o, alpha, beta, None, None, 1.0)
    return int(load_library().la_gdn_prefill_workspace_size(ctypes.byref(a)))


def la_gdn_prefill_workspace_size_min(q, k, v, alpha, beta, o=None) -> int:
    """Smallest workspace la_gdn_prefill accepts (selects the one-kernel schedule)."""
    o = o if o is not None else v
    a = _gdn_args(q, k, v, o, alpha, beta, None, None, 1.0)
    return int(load_library().la_gdn_prefill_workspace_size_min(ctypes.byref(a)))


def _gdn_family_prefill(fn_name, q, k, v, alpha, beta, o, S_in, S_out, q_scale, out_dtype, workspace, stream):
    lib = load_library()
    _check_cuda(q, k, v, alpha, beta, o, S_in, S_out)
    B, H, N, _ = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, H, N, dv), dtype=out_dtype or q.dtype, device=q.device)
    if S_out is None:
        S_out = torch.empty((B, H, dv, q.shape[-1]), dtype=torch.float32, device=q.device)
    for name, t in (("S_in", S_in), ("S_out", S_out)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor")
    a = _gdn_args(q, k, v, o, alpha, beta, S_in, S_out, q_scale)
    need = int(lib.la_gdn_prefill_workspace_size(ctypes.byref(a)))
    ws, ws_bytes = _workspace(need, workspace, q.device)
    st = getattr(lib, fn_name)(ctypes.byref(a), _ptr(ws) if isinstance(ws, torch.Tensor) else ws, ws_bytes,
                               _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, fn_name)
    return o, S_out


def la_gdn_prefill(q, k, v, alpha, beta, o=None, S_in=None, S_out=None, q_scale: float = 1.0,
                   out_dtype=None, workspace=None, stream=None):
    """Chunked gated-delta-rule prefill.  Returns (o, S_out).

    q, k, v: [B,H,N,128] (fp32 or bf16); alpha, beta: fp32 [B,H,N];
    S: fp32 [B,H,128,128] (row = value index).  workspace: optional uint8
    device tensor; by default la_gdn_prefill_workspace_size bytes are
    allocated (the records schedule); a smaller one of at least
    la_gdn_prefill_workspace_size_min bytes selects the one-kernel schedule."""
    return _gdn_family_prefill("la_gdn_prefill", q, k, v, alpha, beta, o, S_in, S_out, q_scale, out_dtype,
                               workspace, stream)


def la_gated_prefill(q, k, v, alpha, beta, o=None, S_in=None, S_out=None, q_scale: float = 1.0,
                     out_dtype=None, workspace=None, stream=None):
    """Chunked scalar-gate prefill, S_t = alpha_t S_{t-1} + beta_t v_t k_t^T,
    o_t = S_t (q_scale q_t).  Arguments, workspace and result as la_gdn_prefill."""
    return _gdn_family_prefill("la_gated_prefill", q, k, v, alpha, beta, o, S_in, S_out, q_scale, out_dtype,
                               workspace, stream)


def la_gdn_prefill_noalloc(q, k, v, alpha, beta, o, S_out, S_in=None, q_scale: float = 1.0, stream=None):
    """la_gdn_prefill without a workspace, for callers that cannot allocate:
    the library's fixed 16 MiB device array serves as scratch (see
    include/la.h).  o and S_out must be preallocated by the caller.
    Returns (o, S_out)."""
    lib = load_library()
    _check_cuda(q, k, v, alpha, beta, o, S_in, S_out)
    a = _gdn_args(q, k, v, o, alpha, beta, S_in, S_out, q_scale)
    st = lib.la_gdn_prefill_noalloc(ctypes.byref(a), _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_gdn_prefill_noalloc")
    return o, S_out


def la_decode_step(variant: int, q, k, v, state, z=None, alpha=None, beta=None, out=None,
                   eps: float = 0.0, q_scale: float = 1.0, out_dtype=None, stream=None, decay=None):
    """One decode step, state (and z) updated in place.  Returns out [S,H,d_v].

    GDN and the scalar gate (LA_VARIANT_GATED): q, k, v [S,H,128], alpha, beta
    fp32 [S,H], state fp32 [S,H,128,128].
    Taylor: q, k [S,H,16], v [S,H,64], state fp32 [S,H,273,64], z fp32 [S,H,273];
    decay: None or fp32 [H] per-head retention, as in la_based_prefill."""
    lib = load_library()
    _check_cuda(q, k, v, state, z, alpha, beta, out, decay)
    for name, t in (("q", q), ("k", k), ("v", v), ("state", state), ("z", z), ("alpha", alpha),
                    ("beta", beta), ("out", out)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    S, H, dk = q.shape
    dv = v.shape[-1]
    _check_decay(decay, H)
    if out is None:
        out = torch.empty((S, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    a = DecodeArgs(int(variant), S, H, dk, dv, _dtype_code(q.dtype), _dtype_code(out.dtype),
                   _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(out), _ptr(state), _ptr(z),
                   float(eps), float(q_scale), _ptr(decay))
    st = lib.la_decode_step(ctypes.byref(a), _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_decode_step")
    return out


def _state_split(t, state_dims: int):
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError("states must be contiguous float32 tensors")
    if not 0 <= state_dims <= t.dim():
        raise ValueError("state_dims out of range")
    per = 1
    for d in t.shape[t.dim() - state_dims:]:
        per *= int(d)
    n = t.numel() // per if per else 0
    return n, per


def la_state_rescale(states, lam, state_dims: int = 2, stream=None):
    """S <- lambda S for every state in `states` (its last `state_dims` dims
    form one state: 2 for GDN S or Taylor s, 1 for Taylor z), in place.
    lam: a float, or a float32 device tensor with one factor per state.
    A factor of 0 resets the state to zeros.  Returns `states`."""
    lib = load_library()
    _check_cuda(states, lam if isinstance(lam, torch.Tensor) else None)
    n, per = _state_split(states, state_dims)
    lam_t = lam if isinstance(lam, torch.Tensor) else None
    if lam_t is not None and (lam_t.dtype != torch.float32 or not lam_t.is_contiguous() or lam_t.numel() != n):
        raise ValueError("lam must be a contiguous float32 tensor with one factor per state")
    st = lib.la_state_rescale(_ptr(states), n, per, _ptr(lam_t), 0.0 if lam_t is not None else float(lam),
                              _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_state_rescale")
    return states


def la_state_gather(src, index, state_dims: int = 2, dst=None, stream=None):
    """dst[i] = src[index[i]] over states (the last `state_dims` dims of src
    form one state); index: int64 device tensor.  Copies one state to
    several destinations, reorders, or keeps a branch point.  Returns dst,
    shaped [len(index), *state_shape]."""
    lib = load_library()
    _check_cuda(src, index, dst)
    n_src, per = _state_split(src, state_dims)
    if index.dtype != torch.int64 or not index.is_contiguous():
        raise ValueError("index must be a contiguous int64 tensor")
    shape = tuple(src.shape[src.dim() - state_dims:])
    if dst is None:
        dst = torch.empty((index.numel(), *shape), dtype=torch.float32, device=src.device)
    n_dst, per_d = _state_split(dst, state_dims)
    if per_d != per or n_dst != index.numel():
        raise ValueError("dst must hold len(index) states of the source's shape")
    st = lib.la_state_gather(_ptr(dst), _ptr(src), _ptr(index), n_dst, n_src, per, _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_state_gather")
    return dst


def la_swa_decode_step(q, k, v, k_cache, v_cache, pos, out=None, scale: float | None = None, out_dtype=None,
                       stream=None):
    """One sliding-window softmax-attention decode step (the window layers of
    BASED).  q, k, v: [S,H,d]; k_cache, v_cache: [S,H,window,d] ring buffers
    (token p in slot p % window), updated in place; pos: int64 [S] tokens
    already seen per sequence (not advanced here).  scale defaults to
    1/sqrt(d).  Returns out [S,H,d]."""
    lib = load_library()
    _check_cuda(q, k, v, k_cache, v_cache, pos, out)
    for name, t in (("q", q), ("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("pos", pos),
                    ("out", out)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if pos.dtype != torch.int64:
        raise ValueError("pos must be int64")
    S, H, d = q.shape
    window = k_cache.shape[2]
    if out is None:
        out = torch.empty((S, H, d), dtype=out_dtype or q.dtype, device=q.device)
    a = SwaDecodeArgs(S, H, d, window, _dtype_code(q.dtype), _dtype_code(out.dtype), _ptr(q), _ptr(k), _ptr(v),
                      _ptr(k_cache), _ptr(v_cache), _ptr(pos), _ptr(out),
                      float(scale if scale is not None else d ** -0.5))
    st = lib.la_swa_decode_step(ctypes.byref(a), _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_swa_decode_step")
    return out


NOTE_ADDR_DIMS = 16  # d_rho


def la_notebank_scores(k, chunk: int = 512, window: int = 48, stream=None):
    """NoteBank write-side scores (NoteBank Sec. 2 Eqs. (3), (8)).  k: [L, H, N, d]
    (the L x H channels of one document; fp32 or bf16, d a multiple of 32 up
    to 256).  Returns (d_ch [L,H,N], d_mean [N], w [N - window + 1]) fp32."""
    lib = load_library()
    _check_cuda(k)
    L, H, N, d = k.shape
    d_ch = torch.empty((L, H, N), dtype=torch.float32, device=k.device)
    d_mean = torch.empty((N,), dtype=torch.float32, device=k.device)
    w = torch.empty((max(N - window + 1, 0),), dtype=torch.float32, device=k.device)
    a = NotebankScoresArgs(L, H, N, d, _dtype_code(k.dtype), _view4(k), int(chunk), int(window),
                           _ptr(d_ch), _ptr(d_mean), _ptr(w) if w.numel() else None)
    st = lib.la_notebank_scores(ctypes.byref(a), _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_notebank_scores")
    return d_ch, d_mean, w


def la_notebank_address(d_ch, q, coords, spans, stream=None):
    """NoteBank note addresses (Eqs. (4), (9)): per note span and channel, the
    argmax of d_ch over the span and the query's 16 `coords` there as bf16.
    d_ch [L,H,N] fp32, q [L,H,N,d], coords int32 [L,H,16], spans int64 [n,2]
    (start, length), all on the device.  Returns (t_star int32 [n,L,H],
    rho bf16 [n,L,H,16])."""
    lib = load_library()
    _check_cuda(d_ch, q, coords, spans)
    L, H, N, d = q.shape
    n = spans.shape[0]
    if coords.dtype != torch.int32 or spans.dtype != torch.int64 or not coords.is_contiguous() or not spans.is_contiguous():
        raise ValueError("coords must be contiguous int32 and spans contiguous int64")
    t_star = torch.empty((n, L, H), dtype=torch.int32, device=q.device)
    rho = torch.empty((n, L, H, NOTE_ADDR_DIMS), dtype=torch.bfloat16, device=q.device)
    a = NotebankAddressArgs(L, H, N, d, n, _dtype_code(q.dtype), _view4(q), _ptr(d_ch), _ptr(coords), _ptr(spans),
                            _ptr(t_star), _ptr(rho))
    st = lib.la_notebank_address(ctypes.byref(a), _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_notebank_address")
    return t_star, rho


def la_notebank_route(rho, u, R: int, positions=None, want_scores: bool = False, stream=None):
    """NoteBank routing (Eq. (5)).  rho bf16 [n, J, 16] (notes in insertion
    order), u bf16 [J, n_q, 16] (question features), positions int64 [n] or
    None.  Returns (top int32 [R] in text order, -1 padded, winner int32 [J],
    votes int32 [n], s fp32 [n, J] or None)."""
    lib = load_library()
    _check_cuda(rho, u, positions)
    n, J = rho.shape[0], u.shape[0]
    for name, t in (("rho", rho), ("u", u)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor")
    dev = u.device
    winner = torch.empty((J,), dtype=torch.int32, device=dev)
    votes = torch.empty((n,), dtype=torch.int32, device=dev)
    top = torch.empty((R,), dtype=torch.int32, device=dev)
    s = torch.empty((n, J), dtype=torch.float32, device=dev) if want_scores else None
    a = NotebankRouteArgs(n, J, u.shape[1], int(R), _ptr(rho), _ptr(u), _ptr(positions), _ptr(s), _ptr(winner),
                          _ptr(votes), _ptr(top))
    st = lib.la_notebank_route(ctypes.byref(a), _stream_handle(stream))
    if st != LA_OK:
        raise LAError(st, "la_notebank_route")
    return top, winner, votes, s


# ---------------------------------------------------------------------------
# the other layers of a hybrid model: convolution, selective scan, window attention


_CODES = {torch.float32: LA_DTYPE_F32, torch.bfloat16: LA_DTYPE_BF16}


def _code(t: torch.dtype) -> int:
    c = _CODES.get(t)
    return _dtype_code(t) if c is None else c


def _refuse(index, name, t, shape, dtype, whole):
    if t.get_device() != index or index < 0:
        raise ValueError(f"all tensors must live on one CUDA device: {name} is on {t.device}")
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous" if whole else f"the last axis of {name} must be contiguous")


def _check(index, *expected):
    """expected: (name, tensor or None, shape, dtype, whole): every tensor on CUDA device `index`, of that shape and
    type, contiguous as a whole or along its last axis."""
    for name, t, shape, dtype, whole in expected:
        if t is None:
            continue
        if (index < 0 or t.get_device() != index or t.shape != shape or t.dtype is not dtype
                or not (t.is_contiguous() if whole else shape[-1] <= 1 or t.stride(-1) == 1 or not t.numel())):
            _refuse(index, name, t, shape, dtype, whole)


def _rows(t):
    """[B,N,C] tensor -> the words of a view (stride_h unused; the stride of an axis with one entry says nothing)."""
    if t is None:
        return 0, 0, 0, 0
    (B, N, _), (sb, st, _) = t.shape, t.stride()
    return t.data_ptr(), sb if B > 1 else 0, 0, st if N > 1 else 0


def _row(t):
    """[S,C] tensor -> the words of a view."""
    return (0, 0, 0, 0) if t is None else (t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 0, 0, 0)


def _heads(t):
    """[B,H,N,d] tensor -> the words of a view."""
    (B, H, N, _), (sb, sh, st, _) = t.shape, t.stride()
    return t.data_ptr(), sb if B > 1 else 0, sh if H > 1 else 0, st if N > 1 else 0


def _address(t):
    return 0 if t is None else t.data_ptr()


def _new_rows(x, shape, dtype):
    """An output beside x whose rows start on 16-byte boundaries whatever the last size is."""
    if shape[-1] % 8 == 0:
        return torch.empty(shape, dtype=dtype, device=x.device)
    return torch.empty((*shape[:-1], -(-shape[-1] // 8) * 8), dtype=dtype, device=x.device)[..., :shape[-1]]


# what a call with lens writes into outputs that were made for it (include/la.h)
_FILL_ROWS, _FILL_STATE = 1, 2


# The argument structs of include/la.h as words, for one pack() a call (the ctypes structures above describe the
# same bytes).
_CONV_PREFILL = struct.Struct("<4q3i4x8q5q2i")
_CONV_DECODE = struct.Struct("<3q3i4x8qi4x")
_SSM_PREFILL = struct.Struct("<5q2i24q6q2i")
_SSM_DECODE = struct.Struct("<4q2i24q5qi4x")
_SWA_PREFILL = struct.Struct("<7q2i16q2f3q1q3qi4x")
_SWA_BIASED_DECODE = struct.Struct("<4q2i7qf4xqf4xq")
_packed = {}


def _call(fn_name, index, args, *more):
    """Call an entry point with its packed arguments on the current stream of device `index`."""
    fn = _packed.get(fn_name)
    if fn is None or fn[0] is not _lib:
        f = load_library()[fn_name]  # a function object of its own: it takes the packed bytes
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_char_p, *([ctypes.c_void_p, ctypes.c_size_t] if more else []), ctypes.c_void_p]
        fn = _packed[fn_name] = (_lib, f)
    handle = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = fn[1](args, *more, handle)
    else:
        with torch.cuda.device(index):
            st = fn[1](args, *more, handle)
    if st != LA_OK:
        raise LAError(st, fn_name)


def _on_stream(fn):
    """With `stream` (a torch stream or a cudaStream_t) the whole call runs on it: the kernels, and the memory that
    outputs and workspaces take.  Tensors of the caller's stream stay allocated until that work is done, outputs until
    the caller's stream has used them."""
    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        x = args[0] if args else kwargs[first]
        if not x.is_cuda:
            return fn(*args, **kwargs)
        if not isinstance(stream, torch.cuda.Stream):
            handle = _stream_handle(stream)
            # NULL and cudaStreamLegacy are the default stream; as an external stream torch takes neither for it
            stream = torch.cuda.default_stream(x.device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device=x.device)
        if stream.device != x.device:
            raise ValueError(f"the stream is of {stream.device}, the tensors of {x.device}")
        own = torch.cuda.current_stream(x.device)
        with torch.cuda.stream(stream):
            out = fn(*args, **kwargs)
        if own != stream:
            taken = [t for t in (*args, *kwargs.values()) if isinstance(t, torch.Tensor)]
            for t in taken:
                t.record_stream(stream)
            for t in out if isinstance(out, tuple) else (out,):
                if not any(t is i for i in taken):
                    t.record_stream(own)
        return out
    return call


@_on_stream
def la_conv_prefill(x, w, bias=None, state_in=None, lens=None, silu: bool = True, y=None, state_out=None,
                    out_dtype=None, *, stream=None):
    """Short causal depthwise convolution of a prompt.  Returns (y, state_out).

    x: [B,N,C] (fp32 or bf16, channels contiguous, rows 16-byte aligned); w:
    [C,W], W in 2..4, and bias [C] or None, both fp32 or both bf16; state:
    [B,W-1,C] in x's dtype, the last inputs, oldest first (None: zeros; state_out
    may be state_in).  lens: None or int64 [B] on the device: later tokens are
    padding, their rows of y stay as they were (zeros in a y made here)."""
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be [B,N,C] and w [C,W]")
    index, xt, wt = x.get_device(), x.dtype, w.dtype
    B, N, C = x.shape
    W = w.shape[1]
    fill = 0
    if y is None:
        y = _new_rows(x, (B, N, C), out_dtype or xt)
        fill = _FILL_ROWS
    held = (B, W - 1, C)
    _check(index, ("x", x, (B, N, C), xt, False), ("w", w, (C, W), wt, True), ("bias", bias, (C,), wt, True),
           ("lens", lens, (B,), torch.int64, True), ("state_in", state_in, held, xt, True),
           ("state_out", state_out, held, xt, True), ("y", y, (B, N, C), y.dtype, False))
    if state_out is None:
        state_out = torch.empty((B, max(W - 1, 0), C), dtype=xt, device=x.device)
        fill |= _FILL_STATE
    _call("la_conv_prefill", index,
          _CONV_PREFILL.pack(B, N, C, W, _code(xt), _code(y.dtype), _code(wt), *_rows(x), *_rows(y), w.data_ptr(),
                             _address(bias), _address(state_in), state_out.data_ptr(), _address(lens), bool(silu), fill))
    return y, state_out


@_on_stream
def la_conv_decode_step(x, w, state, bias=None, silu: bool = True, out=None, state_out=None, out_dtype=None,
                        *, stream=None):
    """The convolution's step for one token of each sequence.  x: [S,C] (rows
    16-byte aligned); w, bias as in la_conv_prefill; state: [S,W-1,C], updated in
    place unless state_out is given.  Returns out [S,C]."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [S,C] and w [C,W]")
    index, xt, wt = x.get_device(), x.dtype, w.dtype
    S, C = x.shape
    W = w.shape[1]
    state_out = state if state_out is None else state_out
    if out is None:
        out = _new_rows(x, (S, C), out_dtype or xt)
    held = (S, W - 1, C)
    _check(index, ("x", x, (S, C), xt, False), ("w", w, (C, W), wt, True), ("bias", bias, (C,), wt, True),
           ("state", state, held, xt, True), ("state_out", state_out, held, xt, True),
           ("out", out, (S, C), out.dtype, False))
    _call("la_conv_decode_step", index,
          _CONV_DECODE.pack(S, C, W, _code(xt), _code(out.dtype), _code(wt), *_row(x)[:2], *_row(out)[:2],
                            w.data_ptr(), _address(bias), state.data_ptr(), state_out.data_ptr(), bool(silu)))
    return out


def _ssm_prefill_args(u, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus, h_in, lens, y, h_out, fill=0):
    B, N, C = u.shape
    return _SSM_PREFILL.pack(B, N, C, A.shape[1], Bm.shape[1], _code(u.dtype), _code(y.dtype), *_rows(u),
                             *_rows(delta), *_rows(z), *_rows(y), *_heads(Bm), *_heads(Cm), A.data_ptr(), _address(D),
                             _address(delta_bias), _address(h_in), _address(h_out), _address(lens),
                             bool(delta_softplus), fill)


def _ssm_workspace_size(args) -> int:
    f = _packed.get("la_ssm_prefill_workspace_size")
    if f is None or f[0] is not _lib:
        fn = load_library()["la_ssm_prefill_workspace_size"]
        fn.restype, fn.argtypes = ctypes.c_size_t, [ctypes.c_char_p]
        f = _packed["la_ssm_prefill_workspace_size"] = (_lib, fn)
    return f[1](args)


def la_ssm_prefill_workspace_size(u, delta, A, Bm, Cm) -> int:
    return _ssm_workspace_size(_ssm_prefill_args(u, delta, A, Bm, Cm, None, None, None, True, None, None, u, None))


@_on_stream
def la_ssm_prefill(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, delta_softplus: bool = True, h_in=None,
                   lens=None, y=None, h_out=None, out_dtype=None, workspace=None, *, stream=None):
    """Selective state space scan of a prompt.  Returns (y, h_out).

        dt = softplus(delta + delta_bias)   (delta + delta_bias without delta_softplus)
        h <- exp(dt A) h + dt u B;   y = (C h + D u) silu(z)

    u, delta, z: [B,N,C] (fp32 or bf16, rows 16-byte aligned); A: fp32 [C,n];
    Bm, Cm: [B,G,N,n] in u's dtype (channel c reads group c // (C // G)); D,
    delta_bias: fp32 [C] or None; h: fp32 [B,C,n] (h_out may be h_in); lens as in
    la_conv_prefill; workspace: uint8 device tensor of at least
    la_ssm_prefill_workspace_size bytes, allocated here by default."""
    if u.dim() != 3 or A.dim() != 2 or Bm.dim() != 4:
        raise ValueError("u must be [B,N,C], A [C,n] and Bm, Cm [B,G,N,n]")
    index, ut, f32 = u.get_device(), u.dtype, torch.float32
    B, N, C = rows = tuple(u.shape)
    n, G = A.shape[1], Bm.shape[1]
    fill = 0
    if y is None:
        y = _new_rows(u, rows, out_dtype or ut)
        fill = _FILL_ROWS
    _check(index, ("u", u, rows, ut, False), ("delta", delta, rows, ut, False), ("z", z, rows, ut, False),
           ("Bm", Bm, (B, G, N, n), ut, False), ("Cm", Cm, (B, G, N, n), ut, False), ("A", A, (C, n), f32, True),
           ("D", D, (C,), f32, True), ("delta_bias", delta_bias, (C,), f32, True), ("h_in", h_in, (B, C, n), f32, True),
           ("h_out", h_out, (B, C, n), f32, True), ("lens", lens, (B,), torch.int64, True),
           ("y", y, rows, y.dtype, False))
    if h_out is None:
        h_out = torch.empty((B, C, n), dtype=f32, device=u.device)
        fill |= _FILL_STATE
    a = _ssm_prefill_args(u, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus, h_in, lens, y, h_out, fill)
    ws, ws_bytes = _workspace(_ssm_workspace_size(a), workspace, u.device)
    if workspace is not None and workspace.get_device() != index:
        raise ValueError("workspace must live on the device of the inputs")
    _call("la_ssm_prefill", index, a, ws.data_ptr() if isinstance(ws, torch.Tensor) else ws, ws_bytes)
    return y, h_out


@_on_stream
def la_ssm_decode_step(u, delta, A, Bm, Cm, state, D=None, z=None, delta_bias=None, delta_softplus: bool = True,
                       out=None, state_out=None, out_dtype=None, *, stream=None):
    """The scan's step for one token of each sequence.  u, delta, z: [S,C]; Bm,
    Cm: [S,G,n]; state: fp32 [S,C,n], updated in place unless state_out is given;
    the rest as in la_ssm_prefill.  Returns out [S,C]."""
    if u.dim() != 2 or A.dim() != 2 or Bm.dim() != 3:
        raise ValueError("u must be [S,C], A [C,n] and Bm, Cm [S,G,n]")
    index, ut, f32 = u.get_device(), u.dtype, torch.float32
    S, C = rows = tuple(u.shape)
    n, G = A.shape[1], Bm.shape[1]
    state_out = state if state_out is None else state_out
    if out is None:
        out = torch.empty(rows, dtype=out_dtype or ut, device=u.device)
    _check(index, ("u", u, rows, ut, False), ("delta", delta, rows, ut, False), ("z", z, rows, ut, False),
           ("Bm", Bm, (S, G, n), ut, False), ("Cm", Cm, (S, G, n), ut, False), ("A", A, (C, n), f32, True),
           ("D", D, (C,), f32, True), ("delta_bias", delta_bias, (C,), f32, True), ("state", state, (S, C, n), f32, True),
           ("state_out", state_out, (S, C, n), f32, True), ("out", out, rows, out.dtype, False))
    many, groups = S > 1, G > 1
    _call("la_ssm_decode_step", index,
          _SSM_DECODE.pack(S, C, n, G, _code(ut), _code(out.dtype), *_row(u), *_row(delta), *_row(z), *_row(out),
                           Bm.data_ptr(), Bm.stride(0) if many else 0, Bm.stride(1) if groups else 0, 0,
                           Cm.data_ptr(), Cm.stride(0) if many else 0, Cm.stride(1) if groups else 0, 0,
                           A.data_ptr(), _address(D), _address(delta_bias), state.data_ptr(), state_out.data_ptr(),
                           bool(delta_softplus)))
    return out


@_on_stream
def la_swa_prefill(q, k, v, window: int = 0, scale: float | None = None, softcap: float = 0.0, slopes=None,
                   key_lo=None, key_hi=None, q_pos0: int | None = None, lens=None, o=None, k_cache=None, v_cache=None,
                   out_dtype=None, *, stream=None):
    """Softmax attention of a prompt's queries.  Returns o [B,H,Nq,d].

    q: [B,H,Nq,d], k, v: [B,H_kv,Nk,d] (fp32 or bf16; H a multiple of H_kv; d a
    multiple of 8 up to 128).  Query i stands at key position p = q_pos0 + i
    (default: the last Nq of Nk) and sees the keys from max(key_lo[b,i], p -
    window + 1) to key_hi[b,i] - 1 (int32 [B,Nq]; default: every key up to p;
    window 0: unbounded); a query that sees nothing gives zeros.  Scores: softcap
    tanh(scale q.k / softcap) (0: no cap) - slopes[h] |p - j| (fp32 [H] or None).
    lens: None or int64 [B]: later keys are not seen and later queries' rows of o
    stay as they were.  k_cache, v_cache: [B,H_kv,window,d] rings to fill for
    la_swa_decode_step and la_swa_biased_decode_step (window <= 256)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,H,Nq,d] and k, v [B,H_kv,Nk,d]")
    index, qt, i32 = q.get_device(), q.dtype, torch.int32
    B, H, Nq, d = queries = tuple(q.shape)
    keys = tuple(k.shape)
    Hkv, Nk, window = keys[1], keys[2], int(window)
    fill = 0
    if o is None:
        o = torch.empty(queries, dtype=out_dtype or qt, device=q.device)
        fill = _FILL_ROWS
    _check(index, ("q", q, queries, qt, False), ("k", k, (B, Hkv, Nk, d), qt, False), ("v", v, (B, Hkv, Nk, d), qt, False),
           ("slopes", slopes, (H,), torch.float32, True), ("key_lo", key_lo, (B, Nq), i32, True),
           ("key_hi", key_hi, (B, Nq), i32, True), ("lens", lens, (B,), torch.int64, True),
           ("k_cache", k_cache, (B, Hkv, window, d), qt, True), ("v_cache", v_cache, (B, Hkv, window, d), qt, True),
           ("o", o, queries, o.dtype, False))
    _call("la_swa_prefill", index,
          _SWA_PREFILL.pack(B, H, Hkv, Nq, Nk, d, window, _code(qt), _code(o.dtype), *_heads(q), *_heads(k), *_heads(v),
                            *_heads(o), scale if scale is not None else d ** -0.5, softcap, _address(slopes),
                            _address(key_lo), _address(key_hi), q_pos0 if q_pos0 is not None else Nk - Nq,
                            _address(lens), _address(k_cache), _address(v_cache), fill))
    return o


@_on_stream
def la_swa_biased_decode_step(q, k, v, k_cache, v_cache, pos, softcap: float = 0.0, slopes=None, out=None,
                              scale: float | None = None, out_dtype=None, *, stream=None):
    """la_swa_decode_step with grouped heads, capped scores and a distance bias:
    q: [S,H,d]; k, v: [S,H_kv,d]; k_cache, v_cache: [S,H_kv,window,d]; pos: int64
    [S]; softcap and slopes as in la_swa_prefill.  Returns out [S,H,d]."""
    if q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [S,H,d], k, v [S,H_kv,d] and the caches [S,H_kv,window,d]")
    index, qt = q.get_device(), q.dtype
    S, H, d = heads = tuple(q.shape)
    Hkv, window = k.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty(heads, dtype=out_dtype or qt, device=q.device)
    ring = (S, Hkv, window, d)
    _check(index, ("q", q, heads, qt, True), ("k", k, (S, Hkv, d), qt, True), ("v", v, (S, Hkv, d), qt, True),
           ("k_cache", k_cache, ring, qt, True), ("v_cache", v_cache, ring, qt, True), ("pos", pos, (S,), torch.int64, True),
           ("slopes", slopes, (H,), torch.float32, True), ("out", out, heads, out.dtype, True))
    _call("la_swa_biased_decode_step", index,
          _SWA_BIASED_DECODE.pack(S, H, d, window, _code(qt), _code(out.dtype), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                  k_cache.data_ptr(), v_cache.data_ptr(), pos.data_ptr(), out.data_ptr(),
                                  scale if scale is not None else d ** -0.5, Hkv, softcap, _address(slopes)))
    return out


def la_device_status(stream=None, clear: bool = True) -> int:
    return int(load_library().la_device_status(_stream_handle(stream), 1 if clear else 0))


def la_selftest_bounded_wait(arrive: bool, limit_ns: int, stream=None) -> int:
    """Launch the bounded-wait self-test (see include/la.h); returns the launch status."""
    return int(load_library().la_selftest_bounded_wait(1 if arrive else 0, int(limit_ns), _stream_handle(stream)))
