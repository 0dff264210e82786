"""Python binding of libtriattn (ctypes; argument marshalling only).

Every step of the computation runs in the CUDA kernels behind the C ABI in
``include/triattn.h``.  This module only checks tensor dtypes and shapes,
allocates outputs with torch (device memory), passes raw pointers and the
current CUDA stream, and raises on a non-OK status.  There is no fallback:
if the shared library is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import operator
import os
import struct
import threading
import warnings
from typing import Optional

import torch

from . import build as _build

_LIB = None
_HOST = None
_LOCK = threading.Lock()

STATUS = {
    0: "TRIATTN_OK",
    1: "TRIATTN_ERR_INVALID_ARG",
    2: "TRIATTN_ERR_UNSUPPORTED",
    3: "TRIATTN_ERR_WORKSPACE",
    4: "TRIATTN_ERR_CUDA",
    5: "TRIATTN_ERR_TIMEOUT",
}
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(6)

EXPORTED = ("triattn_status_string", "triattn_fwd_workspace_bytes", "triattn_bwd_workspace_bytes", "tri_attn_fwd",
            "tri_attn_bwd",
            "triattn_device_status", "triattn_set_wait_limit_ns", "triattn_trace_enable", "triattn_trace_read",
            "triattn_test_set_starve", "tri_attn_bwd_noalloc", "triattn_bwd_atomic_workspace_bytes",
            "tri_attn_bwd_atomic_ablation", "tri_attn_dbias_combine", "triattn_module_ctx_bytes",
            "triattn_module_workspace_bytes", "tri_attn_module_fwd", "tri_attn_module_bwd",
            "triattn_trimul_ctx_bytes", "triattn_trimul_workspace_bytes", "triattn_trimul_fwd",
            "triattn_trimul_bwd", "triattn_gemm_workspace_bytes", "triattn_gemm", "tri_attn_fwd_strided",
            "tri_attn_bwd_strided", "triattn_transition_workspace_bytes", "triattn_transition_fwd",
            "triattn_transition_bwd", "triattn_grad_norm_workspace_bytes", "triattn_grad_norm",
            "triattn_clip_grad_norm", "triattn_qk_norm_workspace_bytes", "triattn_qk_norm_fwd", "triattn_qk_norm_bwd",
            "triattn_relpos_workspace_bytes", "triattn_relpos_fwd", "triattn_relpos_bwd",
            "triattn_orthogonalize_workspace_bytes", "triattn_orthogonalize")

FLAG_DBIAS_FP32 = 1
FLAG_GRADS_BF16 = 2
FLAG_DOUT_FP32 = 4

NOALLOC_SCRATCH_BYTES = 64 << 20


class TraceEntry(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double),
                ("min_ms", ctypes.c_double), ("max_ms", ctypes.c_double)]


class TriAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N_o", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("flags", ctypes.c_uint)]


class Layout(ctypes.Structure):
    """triattn_layout: row (b, o, h, n) of a [B, N_o, H, N, D] tensor starts
    slice * (b N_o + o) + head * h + row * n elements from its base."""
    _fields_ = [("slice", ctypes.c_longlong), ("head", ctypes.c_longlong), ("row", ctypes.c_longlong)]


class ModuleShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("C", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("flags", ctypes.c_uint)]


class TriMulShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("C_z", ctypes.c_int), ("C_h", ctypes.c_int),
                ("direction", ctypes.c_int), ("flags", ctypes.c_uint)]


class TransitionShape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_longlong), ("C", ctypes.c_int), ("H", ctypes.c_int), ("activation", ctypes.c_int),
                ("flags", ctypes.c_uint)]


class QKNormShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N_o", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("w_heads", ctypes.c_int), ("rotary", ctypes.c_int), ("eps", ctypes.c_float),
                ("theta", ctypes.c_double), ("flags", ctypes.c_uint)]


class RelposShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("F", ctypes.c_int), ("layout", ctypes.c_int),
                ("kind", ctypes.c_int), ("buckets", ctypes.c_int), ("max_distance", ctypes.c_int),
                ("flags", ctypes.c_uint)]


class Tensor(ctypes.Structure):
    """triattn_tensor: one gradient of a list (device pointer, elements, dtype)."""
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_longlong), ("dtype", ctypes.c_int)]


ACTIVATIONS = {"silu": 0, "sigmoid": 1, "gelu": 2}
TRIMUL_DIRECTIONS = {"outgoing": 0, "incoming": 1}
ROTARY = {"none": 0, "half": 1, "interleaved": 2}
RELPOS_LAYOUTS = {"heads": 0, "pairs": 1}
BUCKETS = {"clip": 0, "log": 1}


def _declare(lib):
    vp, sp = ctypes.c_void_p, ctypes.POINTER(Shape)
    lib.triattn_status_string.argtypes = [ctypes.c_int]
    lib.triattn_status_string.restype = ctypes.c_char_p
    lib.triattn_bwd_workspace_bytes.argtypes = [sp]
    lib.triattn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_fwd_workspace_bytes.argtypes = [sp]
    lib.triattn_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.tri_attn_fwd.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.tri_attn_fwd.restype = ctypes.c_int
    lib.tri_attn_bwd.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lp = ctypes.POINTER(Layout)
    lib.tri_attn_fwd_strided.argtypes = [sp, vp, vp, vp, lp, vp, vp, vp, vp, vp, lp, vp, ctypes.c_size_t, vp]
    lib.tri_attn_fwd_strided.restype = ctypes.c_int
    lib.tri_attn_bwd_strided.argtypes = ([sp, vp, vp, vp, lp, vp, vp, vp, vp, lp, vp, vp, lp, vp, vp, vp, lp, vp, vp,
                                          ctypes.c_size_t, vp])
    lib.tri_attn_bwd_strided.restype = ctypes.c_int
    lib.tri_attn_bwd.restype = ctypes.c_int
    lib.triattn_device_status.argtypes = [vp]
    lib.triattn_device_status.restype = ctypes.c_int
    lib.triattn_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.triattn_set_wait_limit_ns.restype = None
    lib.triattn_trace_enable.argtypes = [ctypes.c_int]
    lib.triattn_trace_enable.restype = None
    lib.triattn_trace_read.argtypes = [ctypes.POINTER(TraceEntry), ctypes.c_int]
    lib.triattn_trace_read.restype = ctypes.c_int
    lib.triattn_test_set_starve.argtypes = [ctypes.c_int]
    lib.triattn_test_set_starve.restype = None
    lib.tri_attn_bwd_noalloc.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.tri_attn_bwd_noalloc.restype = ctypes.c_int
    lib.triattn_bwd_atomic_workspace_bytes.argtypes = [sp, ctypes.c_int]
    lib.triattn_bwd_atomic_workspace_bytes.restype = ctypes.c_size_t
    lib.tri_attn_bwd_atomic_ablation.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                                 vp, ctypes.c_size_t, vp]
    lib.tri_attn_bwd_atomic_ablation.restype = ctypes.c_int
    lib.tri_attn_dbias_combine.argtypes = [sp, vp, ctypes.c_int, vp, vp]
    lib.tri_attn_dbias_combine.restype = ctypes.c_int
    mp = ctypes.POINTER(ModuleShape)
    lib.triattn_module_ctx_bytes.argtypes = [mp]
    lib.triattn_module_ctx_bytes.restype = ctypes.c_size_t
    lib.triattn_module_workspace_bytes.argtypes = [mp]
    lib.triattn_module_workspace_bytes.restype = ctypes.c_size_t
    lib.tri_attn_module_fwd.argtypes = [mp] + [vp] * 9 + [ctypes.c_size_t, vp]
    lib.tri_attn_module_fwd.restype = ctypes.c_int
    lib.tri_attn_module_bwd.argtypes = [mp] + [vp] * 13 + [ctypes.c_size_t, vp]
    lib.tri_attn_module_bwd.restype = ctypes.c_int
    tp = ctypes.POINTER(TriMulShape)
    lib.triattn_trimul_ctx_bytes.argtypes = [tp]
    lib.triattn_trimul_ctx_bytes.restype = ctypes.c_size_t
    lib.triattn_trimul_workspace_bytes.argtypes = [tp]
    lib.triattn_trimul_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_trimul_fwd.argtypes = [tp] + [vp] * 11 + [ctypes.c_size_t, vp]
    lib.triattn_trimul_fwd.restype = ctypes.c_int
    lib.triattn_trimul_bwd.argtypes = [tp] + [vp] * 16 + [ctypes.c_size_t, vp]
    lib.triattn_trimul_bwd.restype = ctypes.c_int
    rp = ctypes.POINTER(TransitionShape)
    lib.triattn_transition_workspace_bytes.argtypes = [rp]
    lib.triattn_transition_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_transition_fwd.argtypes = [rp] + [vp] * 8
    lib.triattn_transition_fwd.restype = ctypes.c_int
    lib.triattn_transition_bwd.argtypes = [rp] + [vp] * 13 + [ctypes.c_size_t, vp]
    lib.triattn_transition_bwd.restype = ctypes.c_int
    ll = ctypes.c_longlong
    lib.triattn_grad_norm_workspace_bytes.argtypes = [ll]
    lib.triattn_grad_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_grad_norm.argtypes = [vp, ll, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]
    lib.triattn_grad_norm.restype = ctypes.c_int
    lib.triattn_clip_grad_norm.argtypes = [vp, vp, ll, ctypes.c_int, ctypes.c_float, vp, vp, ctypes.c_size_t, vp]
    lib.triattn_clip_grad_norm.restype = ctypes.c_int
    qp = ctypes.POINTER(QKNormShape)
    lib.triattn_qk_norm_workspace_bytes.argtypes = [qp]
    lib.triattn_qk_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_qk_norm_fwd.argtypes = [qp, vp, vp, lp, vp, vp, vp, vp, vp, lp, vp]
    lib.triattn_qk_norm_fwd.restype = ctypes.c_int
    lib.triattn_qk_norm_bwd.argtypes = ([qp, vp, vp, lp, vp, vp, vp, vp, vp, lp, vp, vp, lp, vp, vp, vp,
                                         ctypes.c_size_t, vp])
    lib.triattn_qk_norm_bwd.restype = ctypes.c_int
    bp = ctypes.POINTER(RelposShape)
    lib.triattn_relpos_workspace_bytes.argtypes = [bp]
    lib.triattn_relpos_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_relpos_fwd.argtypes = [bp] + [vp] * 6
    lib.triattn_relpos_fwd.restype = ctypes.c_int
    lib.triattn_relpos_bwd.argtypes = [bp] + [vp] * 5 + [ctypes.c_size_t, vp]
    lib.triattn_relpos_bwd.restype = ctypes.c_int
    lib.triattn_orthogonalize_workspace_bytes.argtypes = [vp, ll]
    lib.triattn_orthogonalize_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_orthogonalize.argtypes = [vp, vp, ll, ctypes.c_int, vp, ctypes.c_float, vp, ctypes.c_size_t, vp]
    lib.triattn_orthogonalize.restype = ctypes.c_int
    lib.triattn_gemm_workspace_bytes.argtypes = [ctypes.c_int] * 4
    lib.triattn_gemm_workspace_bytes.restype = ctypes.c_size_t
    lib.triattn_gemm.argtypes = ([ctypes.c_int] * 5 + [vp, ll, vp, ll, vp, ll, ctypes.c_int, ctypes.c_int, ll, ll, ll,
                                 vp, ctypes.c_size_t, vp])
    lib.triattn_gemm.restype = ctypes.c_int
    return lib


def library_path() -> str:
    return _build.lib_path()


def load(path: Optional[str] = None):
    """Load libtriattn (built in-tree by ``build.build()``); raises if absent."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    with _LOCK:
        if _LIB is None:
            p = path or library_path()
            if not os.path.exists(p):
                raise RuntimeError(f"libtriattn is not built ({p} missing): run __graft_entry__.build()")
            lib = _declare(ctypes.CDLL(p))
            _load_host(lib)
            _LIB = lib
    return _LIB


class _General:
    """Stands where the native part is not there: every call goes the general path."""

    @staticmethod
    def _leave(*args):
        return None

    qk_norm_fwd = qk_norm_bwd = relpos_fwd = relpos_bwd = matrix_tables = _leave


def _load_host(lib):
    """The binding's native part (csrc/host.cpp), which takes the library's functions
    by address: usual calls of some entry points and the tables of long lists.  It is
    built for one torch and one Python; without it these calls take some 10 us more."""
    global _HOST
    p = _build.host_path()
    try:
        loader = importlib.machinery.ExtensionFileLoader("triattn_host", p)
        host = importlib.util.module_from_spec(importlib.util.spec_from_loader("triattn_host", loader))
        loader.exec_module(host)
    except ImportError as e:
        warnings.warn(f"the binding's native part is not used ({e}): run __graft_entry__.build()", RuntimeWarning)
        _HOST = _General
        return
    names = ("qk_norm_workspace_bytes", "qk_norm_fwd", "qk_norm_bwd", "relpos_workspace_bytes", "relpos_fwd",
             "relpos_bwd")
    host.bind(*(ctypes.cast(getattr(lib, f"triattn_{n}"), ctypes.c_void_p).value for n in names))
    _HOST = host


def _host():
    if _HOST is None:
        load()
    return _HOST


def shape_of(q: torch.Tensor) -> Shape:
    if q.dim() != 5:
        raise ValueError("q must be [B, N_o, H, N, D]")
    B, No, H, N, D = q.shape
    return Shape(B, No, N, H, D, 0)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(t: torch.Tensor, name: str, shape, dtype=torch.bfloat16):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _raise(code: int, where: str):
    if code != OK:
        raise TriAttnError(code, where)


def bwd_workspace_bytes(q_or_shape) -> int:
    s = q_or_shape if isinstance(q_or_shape, Shape) else shape_of(q_or_shape)
    return int(load().triattn_bwd_workspace_bytes(ctypes.byref(s)))


def fwd_workspace_bytes(q_or_shape) -> int:
    s = q_or_shape if isinstance(q_or_shape, Shape) else shape_of(q_or_shape)
    return int(load().triattn_fwd_workspace_bytes(ctypes.byref(s)))


def tri_attn_fwd(q, k, v, bias, mask=None, *, save_residual: bool = True, out=None, workspace=None, stream=None):
    """Forward.  Returns (o [B,N_o,H,N,D] bf16, lse [B,N_o,H,N] fp32,
    o_resid bf16 or None).  ``out`` may pass preallocated (o, lse, o_resid),
    ``workspace`` a uint8 device buffer of ``fwd_workspace_bytes`` bytes
    (allocated per call otherwise)."""
    s = shape_of(q)
    B, No, H, N, D = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, (B, No, H, N, D))
    _check(bias, "bias", (B, H, N, N))
    if mask is not None:
        _check(mask, "mask", (B, No, N))
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((B, No, H, N), dtype=torch.float32, device=q.device)
        resid = torch.empty_like(q) if save_residual else None
    else:
        o, lse, resid = out
    if workspace is None:
        need = fwd_workspace_bytes(s)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 0 else None
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = load().tri_attn_fwd(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(bias), _ptr(mask), _ptr(o),
                               _ptr(lse), _ptr(resid), _ptr(workspace), ctypes.c_size_t(nbytes), _stream_ptr(stream))
    _raise(code, "tri_attn_fwd")
    return o, lse, resid


def tri_attn_bwd(q, k, v, bias, mask, o, o_resid, lse, do, *, workspace=None, out=None, stream=None,
                 dbias_fp32: bool = False):
    """Backward.  ``o_resid=None`` turns the residual compensation off.
    Returns (dq, dk, dv, dbias) in bf16; with ``dbias_fp32`` dbias is the FP32
    sum over this call's outer slices (a shard's part, see tri_attn_dbias_combine)."""
    s = shape_of(q)
    if dbias_fp32:
        s.flags = FLAG_DBIAS_FP32
    B, No, H, N, D = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _check(t, name, (B, No, H, N, D))
    if o_resid is not None:
        _check(o_resid, "o_resid", (B, No, H, N, D))
    _check(bias, "bias", (B, H, N, N))
    _check(lse, "lse", (B, No, H, N), torch.float32)
    if mask is not None:
        _check(mask, "mask", (B, No, N))
    need = bwd_workspace_bytes(s)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        dbias = torch.empty(bias.shape, dtype=torch.float32 if dbias_fp32 else torch.bfloat16, device=q.device)
    else:
        dq, dk, dv, dbias = out
    _check(dbias, "dbias", tuple(bias.shape), torch.float32 if dbias_fp32 else torch.bfloat16)
    code = load().tri_attn_bwd(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(bias), _ptr(mask), _ptr(o),
                               _ptr(o_resid), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbias),
                               _ptr(workspace), ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                               _stream_ptr(stream))
    _raise(code, "tri_attn_bwd")
    return dq, dk, dv, dbias


def layout_of(t: torch.Tensor) -> Layout:
    """The row layout of a [B, N_o, H, N, D] view whose D features are
    contiguous and whose b stride is N_o times its o stride (e.g. the heads of
    pair rows: ``P.view(B, N, N, ld)[..., c:c + H*D].unflatten(-1, (H, D))
    .permute(0, 1, 3, 2, 4)``)."""
    if t.dim() != 5 or t.stride(4) != 1:
        raise ValueError("expected a [B, N_o, H, N, D] view with contiguous features")
    if t.shape[0] > 1 and t.stride(0) != t.shape[1] * t.stride(1):
        raise ValueError("the b stride must be N_o times the o stride")
    return Layout(t.stride(1), t.stride(2), t.stride(3))


def _check_view(t, name, shape, lay: Layout):
    if t is None or not t.is_cuda or t.dtype != torch.bfloat16 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a bf16 CUDA view of shape {tuple(shape)}")
    got = layout_of(t)
    if (got.slice, got.head, got.row) != (lay.slice, lay.head, lay.row):
        raise ValueError(f"{name} does not share the layout of its group")


def tri_attn_fwd_strided(q, k, v, bias, mask, o, lse, o_resid=None, *, workspace=None, stream=None):
    """Forward on views: q, k, v share one row layout, o and o_resid another
    (both [B, N_o, H, N, D] views, written in place); lse [B, N_o, H, N] fp32
    contiguous.  Bitwise the same results as tri_attn_fwd on copies."""
    s = shape_of(q)
    B, No, H, N, D = q.shape
    lq, lo = layout_of(q), layout_of(o)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_view(t, name, (B, No, H, N, D), lq)
    for name, t in (("o", o), ("o_resid", o_resid)):
        if t is not None:
            _check_view(t, name, (B, No, H, N, D), lo)
    _check(bias, "bias", (B, H, N, N))
    _check(lse, "lse", (B, No, H, N), torch.float32)
    if mask is not None:
        _check(mask, "mask", (B, No, N))
    if workspace is None:
        need = fwd_workspace_bytes(s)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 0 else None
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = load().tri_attn_fwd_strided(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(lq), _ptr(bias),
                                       _ptr(mask), _ptr(o), _ptr(lse), _ptr(o_resid), ctypes.byref(lo),
                                       _ptr(workspace), ctypes.c_size_t(nbytes), _stream_ptr(stream))
    _raise(code, "tri_attn_fwd_strided")
    return o, lse, o_resid


def tri_attn_bwd_strided(q, k, v, bias, mask, o, o_resid, lse, do, dq, dk, dv, dbias, *, workspace=None,
                         stream=None):
    """Backward on views: q, k, v share one row layout, o and o_resid a
    second, do a third and dq, dk, dv a fourth; dq, dk, dv and dbias
    ([B, H, N, N] bf16) written in place."""
    s = shape_of(q)
    B, No, H, N, D = q.shape
    lq, lo, ldo, lg = layout_of(q), layout_of(o), layout_of(do), layout_of(dq)
    for name, t, lay in (("q", q, lq), ("k", k, lq), ("v", v, lq), ("dq", dq, lg), ("dk", dk, lg), ("dv", dv, lg),
                         ("o", o, lo), ("o_resid", o_resid, lo), ("do", do, ldo)):
        if t is not None:
            _check_view(t, name, (B, No, H, N, D), lay)
    _check(bias, "bias", (B, H, N, N))
    _check(dbias, "dbias", (B, H, N, N))
    _check(lse, "lse", (B, No, H, N), torch.float32)
    if mask is not None:
        _check(mask, "mask", (B, No, N))
    if workspace is None:
        workspace = torch.empty(bwd_workspace_bytes(s), dtype=torch.uint8, device=q.device)
    code = load().tri_attn_bwd_strided(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(lq), _ptr(bias),
                                       _ptr(mask), _ptr(o), _ptr(o_resid), ctypes.byref(lo), _ptr(lse), _ptr(do),
                                       ctypes.byref(ldo), _ptr(dq), _ptr(dk), _ptr(dv), ctypes.byref(lg),
                                       _ptr(dbias), _ptr(workspace),
                                       ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                                       _stream_ptr(stream))
    _raise(code, "tri_attn_bwd_strided")
    return dq, dk, dv, dbias


ATOMIC_DQ, ATOMIC_DBIAS, ATOMIC_DBIAS_DQ, BULK_DQ, BULK_DQ_ATOMIC_DBIAS = 1, 2, 3, 4, 6


def bwd_atomic_workspace_bytes(q_or_shape, atomic_mask: int) -> int:
    """Workspace of the atomic ablation (0 for an invalid shape or mask)."""
    s = q_or_shape if isinstance(q_or_shape, Shape) else shape_of(q_or_shape)
    return int(load().triattn_bwd_atomic_workspace_bytes(ctypes.byref(s), int(atomic_mask)))


def tri_attn_bwd_atomic_ablation(q, k, v, bias, mask, o, o_resid, lse, do, atomic_mask=ATOMIC_DBIAS_DQ, *,
                                 workspace=None, out=None, stream=None):
    """Ablation only (not the library's backward): the backward with FP32
    atomics for dQ (``atomic_mask=1``), dbias (2) or both (3), or TMA bulk
    reductions for dQ (4; 6 with atomic dbias), instead of the ordered
    single-writer partials.  The gradients added that way are not bitwise
    reproducible between calls.  Returns (dq, dk, dv, dbias) in bf16."""
    s = shape_of(q)
    B, No, H, N, D = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _check(t, name, (B, No, H, N, D))
    if o_resid is not None:
        _check(o_resid, "o_resid", (B, No, H, N, D))
    _check(bias, "bias", (B, H, N, N))
    _check(lse, "lse", (B, No, H, N), torch.float32)
    if mask is not None:
        _check(mask, "mask", (B, No, N))
    need = bwd_atomic_workspace_bytes(s, atomic_mask)
    if need == 0:
        raise TriAttnError(ERR_INVALID_ARG, "tri_attn_bwd_atomic_ablation")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        dbias = torch.empty_like(bias)
    else:
        dq, dk, dv, dbias = out
    code = load().tri_attn_bwd_atomic_ablation(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(bias), _ptr(mask),
                                               _ptr(o), _ptr(o_resid), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                                               _ptr(dv), _ptr(dbias), int(atomic_mask), _ptr(workspace),
                                               ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                                               _stream_ptr(stream))
    _raise(code, "tri_attn_bwd_atomic_ablation")
    return dq, dk, dv, dbias


def tri_attn_dbias_combine(parts, *, out=None, stream=None):
    """dbias of an outer axis split across GPUs: ``parts`` is [R, B, H, N, N]
    FP32 (each written by tri_attn_bwd(..., dbias_fp32=True) on one shard,
    gathered in rank order); returns bf16 [B, H, N, N], the parts added in
    ascending r in FP32 and rounded once."""
    if parts.dim() != 5 or parts.dtype != torch.float32 or not parts.is_cuda or not parts.is_contiguous():
        raise ValueError("parts must be a contiguous CUDA float32 tensor [R, B, H, N, N]")
    R, B, H, N, N2 = parts.shape
    if N != N2:
        raise ValueError("parts must be [R, B, H, N, N]")
    s = Shape(B, N, N, H, 16, 0)
    dbias = out if out is not None else torch.empty((B, H, N, N), dtype=torch.bfloat16, device=parts.device)
    _check(dbias, "dbias", (B, H, N, N))
    code = load().tri_attn_dbias_combine(ctypes.byref(s), _ptr(parts), int(R), _ptr(dbias), _stream_ptr(stream))
    _raise(code, "tri_attn_dbias_combine")
    return dbias


def device_status(stream=None) -> int:
    """Synchronise the stream and return (then clear) the device status code."""
    return int(load().triattn_device_status(_stream_ptr(stream)))


def set_wait_limit_ns(ns: int) -> None:
    load().triattn_set_wait_limit_ns(ctypes.c_ulonglong(int(ns)))


def trace_enable(on: bool = True) -> None:
    """Start (clearing old records) or stop per-kernel CUDA-event tracing."""
    load().triattn_trace_enable(1 if on else 0)


def trace_read() -> dict:
    """Per-kernel totals of the traced launches: {name: {launches, total_ms,
    mean_ms, min_ms, max_ms}} (synchronises the recorded events)."""
    buf = (TraceEntry * 64)()
    n = load().triattn_trace_read(buf, 64)
    if n < 0:
        raise TriAttnError(ERR_CUDA, "triattn_trace_read")
    out = {}
    for e in buf[:n]:
        name = e.kernel.decode()
        out[name] = {"launches": e.launches, "total_ms": e.total_ms, "mean_ms": e.total_ms / max(e.launches, 1),
                     "min_ms": e.min_ms, "max_ms": e.max_ms}
    return out


def test_set_starve(on: bool) -> None:
    """Test hook: starve the MMA warp of the forward, of small matrices' orthogonalisation and of the
    table's gradient from pair features, so that its bounded wait runs out."""
    load().triattn_test_set_starve(1 if on else 0)


def module_sizes(B: int, N: int, C: int, H: int, D: int):
    """(ctx bytes, workspace bytes) of the module; (0, 0) for an unsupported shape."""
    s = ModuleShape(B, N, C, H, D, 0)
    lib = load()
    return int(lib.triattn_module_ctx_bytes(ctypes.byref(s))), int(lib.triattn_module_workspace_bytes(ctypes.byref(s)))


def _module_shape(z, H, D):
    if z.dim() != 4 or z.shape[1] != z.shape[2]:
        raise ValueError("z must be [B, N, N, C]")
    B, N, _, C = z.shape
    return ModuleShape(B, N, C, H, D, 0)


def _bytes(t):
    return ctypes.c_size_t(t.numel() * t.element_size())


def tri_attn_module_fwd(z, mask, ln_w, ln_b, w_in, w_o, H: int, D: int, *, ctx=None, workspace=None, out=None,
                        stream=None):
    """Module forward: LayerNorm, projections into q, k, v and the bias, the
    core, output projection.  Returns (out [B, N, N, C] bf16, ctx) where ctx
    is the uint8 buffer the backward needs."""
    s = _module_shape(z, H, D)
    B, N, C = s.B, s.N, s.C
    F = 3 * H * D + H
    _check(z, "z", (B, N, N, C))
    _check(ln_w, "ln_w", (C,), torch.float32)
    _check(ln_b, "ln_b", (C,), torch.float32)
    _check(w_in, "w_in", (C, F))
    _check(w_o, "w_o", (H * D, C))
    if mask is not None:
        _check(mask, "mask", (B, N, N))
    nctx, nws = module_sizes(B, N, C, H, D)
    if nctx == 0:
        raise TriAttnError(ERR_UNSUPPORTED, "tri_attn_module_fwd")
    if ctx is None:
        ctx = torch.empty(nctx, dtype=torch.uint8, device=z.device)
    if workspace is None:
        workspace = torch.empty(nws, dtype=torch.uint8, device=z.device)
    if out is None:
        out = torch.empty_like(z)
    _check(out, "out", (B, N, N, C))
    code = load().tri_attn_module_fwd(ctypes.byref(s), _ptr(z), _ptr(mask), _ptr(ln_w), _ptr(ln_b), _ptr(w_in),
                                      _ptr(w_o), _ptr(out), _ptr(ctx), _ptr(workspace), _bytes(workspace),
                                      _stream_ptr(stream))
    _raise(code, "tri_attn_module_fwd")
    return out, ctx


def tri_attn_module_bwd(z, mask, ln_w, w_in, w_o, ctx, d_out, H: int, D: int, *, workspace=None, out=None,
                        stream=None):
    """Module backward of <out, d_out>.  Returns (dz bf16, d_ln_w, d_ln_b,
    d_w_in, d_w_o fp32)."""
    s = _module_shape(z, H, D)
    B, N, C = s.B, s.N, s.C
    F = 3 * H * D + H
    _check(z, "z", (B, N, N, C))
    _check(d_out, "d_out", (B, N, N, C))
    _check(ln_w, "ln_w", (C,), torch.float32)
    _check(w_in, "w_in", (C, F))
    _check(w_o, "w_o", (H * D, C))
    if mask is not None:
        _check(mask, "mask", (B, N, N))
    nctx, nws = module_sizes(B, N, C, H, D)
    if nctx == 0:
        raise TriAttnError(ERR_UNSUPPORTED, "tri_attn_module_bwd")
    _check(ctx, "ctx", (nctx,), torch.uint8)
    if workspace is None:
        workspace = torch.empty(nws, dtype=torch.uint8, device=z.device)
    if out is None:
        f32 = dict(dtype=torch.float32, device=z.device)
        out = (torch.empty_like(z), torch.empty(C, **f32), torch.empty(C, **f32), torch.empty((C, F), **f32),
               torch.empty((H * D, C), **f32))
    dz, dlw, dlb, dwi, dwo = out
    code = load().tri_attn_module_bwd(ctypes.byref(s), _ptr(z), _ptr(mask), _ptr(ln_w), _ptr(w_in), _ptr(w_o),
                                      _ptr(ctx), _ptr(d_out), _ptr(dz), _ptr(dlw), _ptr(dlb), _ptr(dwi), _ptr(dwo),
                                      _ptr(workspace), _bytes(workspace), _stream_ptr(stream))
    _raise(code, "tri_attn_module_bwd")
    return dz, dlw, dlb, dwi, dwo


def trimul_shape(B: int, N: int, Cz: int, Ch: int, direction: str) -> TriMulShape:
    if direction not in TRIMUL_DIRECTIONS:
        raise ValueError(f"direction must be one of {tuple(TRIMUL_DIRECTIONS)}")
    return TriMulShape(B, N, Cz, Ch, TRIMUL_DIRECTIONS[direction], 0)


def trimul_sizes(B: int, N: int, Cz: int, Ch: int, direction: str = "outgoing"):
    """(ctx bytes, workspace bytes) of the triangle multiplicative update; (0, 0)
    for an unsupported shape."""
    s = trimul_shape(B, N, Cz, Ch, direction)
    lib = load()
    return int(lib.triattn_trimul_ctx_bytes(ctypes.byref(s))), int(lib.triattn_trimul_workspace_bytes(ctypes.byref(s)))


def _trimul_check(z, mask, ln_in_w, w_p, ln_out_w, w_o):
    if z.dim() != 4 or z.shape[1] != z.shape[2]:
        raise ValueError("z must be [B, N, N, C_z]")
    B, N, _, Cz = z.shape
    if w_o.dim() != 2:
        raise ValueError("w_o must be [C_h, C_z]")
    Ch = w_o.shape[0]
    _check(z, "z", (B, N, N, Cz))
    _check(ln_in_w, "ln_in_w", (Cz,), torch.float32)
    _check(w_p, "w_p", (Cz, 4 * Ch + Cz))
    _check(ln_out_w, "ln_out_w", (Ch,), torch.float32)
    _check(w_o, "w_o", (Ch, Cz))
    if mask is not None:
        _check(mask, "mask", (B, N, N))
    return B, N, Cz, Ch


def triattn_trimul_fwd(z, mask, ln_in_w, ln_in_b, w_p, ln_out_w, ln_out_b, w_o, direction: str, *, ctx=None,
                       workspace=None, out=None, stream=None):
    """Triangle multiplicative update forward ("outgoing" or "incoming").
    Returns (out [B, N, N, C_z] bf16, ctx) where ctx is the uint8 buffer the
    backward needs."""
    B, N, Cz, Ch = _trimul_check(z, mask, ln_in_w, w_p, ln_out_w, w_o)
    _check(ln_in_b, "ln_in_b", (Cz,), torch.float32)
    _check(ln_out_b, "ln_out_b", (Ch,), torch.float32)
    s = trimul_shape(B, N, Cz, Ch, direction)
    nctx, nws = trimul_sizes(B, N, Cz, Ch, direction)
    if nctx == 0:
        raise TriAttnError(ERR_UNSUPPORTED, "triattn_trimul_fwd")
    ctx = torch.empty(nctx, dtype=torch.uint8, device=z.device) if ctx is None else ctx
    workspace = torch.empty(nws, dtype=torch.uint8, device=z.device) if workspace is None else workspace
    out = torch.empty_like(z) if out is None else out
    _check(out, "out", (B, N, N, Cz))
    code = load().triattn_trimul_fwd(ctypes.byref(s), _ptr(z), _ptr(mask), _ptr(ln_in_w), _ptr(ln_in_b), _ptr(w_p),
                                     _ptr(ln_out_w), _ptr(ln_out_b), _ptr(w_o), _ptr(out), _ptr(ctx),
                                     _ptr(workspace), _bytes(workspace), _stream_ptr(stream))
    _raise(code, "triattn_trimul_fwd")
    return out, ctx


def triattn_trimul_bwd(z, mask, ln_in_w, w_p, ln_out_w, w_o, ctx, d_out, direction: str, *, workspace=None,
                       out=None, stream=None):
    """Backward of <out, d_out>.  Returns (dz bf16, d_ln_in_w, d_ln_in_b, d_w_p,
    d_ln_out_w, d_ln_out_b, d_w_o fp32)."""
    B, N, Cz, Ch = _trimul_check(z, mask, ln_in_w, w_p, ln_out_w, w_o)
    _check(d_out, "d_out", (B, N, N, Cz))
    s = trimul_shape(B, N, Cz, Ch, direction)
    nctx, nws = trimul_sizes(B, N, Cz, Ch, direction)
    if nctx == 0:
        raise TriAttnError(ERR_UNSUPPORTED, "triattn_trimul_bwd")
    _check(ctx, "ctx", (nctx,), torch.uint8)
    workspace = torch.empty(nws, dtype=torch.uint8, device=z.device) if workspace is None else workspace
    if out is None:
        f32 = dict(dtype=torch.float32, device=z.device)
        out = (torch.empty_like(z), torch.empty(Cz, **f32), torch.empty(Cz, **f32),
               torch.empty((Cz, 4 * Ch + Cz), **f32), torch.empty(Ch, **f32), torch.empty(Ch, **f32),
               torch.empty((Ch, Cz), **f32))
    dz, dliw, dlib, dwp, dlow, dlob, dwo = out
    code = load().triattn_trimul_bwd(ctypes.byref(s), _ptr(z), _ptr(mask), _ptr(ln_in_w), _ptr(w_p), _ptr(ln_out_w),
                                     _ptr(w_o), _ptr(ctx), _ptr(d_out), _ptr(dz), _ptr(dliw), _ptr(dlib), _ptr(dwp),
                                     _ptr(dlow), _ptr(dlob), _ptr(dwo), _ptr(workspace), _bytes(workspace),
                                     _stream_ptr(stream))
    _raise(code, "triattn_trimul_bwd")
    return out


def _current_stream_ptr(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the stream's address without a Stream object around it, where torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream_ptr)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class _Here:
    """A context that changes nothing."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on_stream(device, stream):
    """(context, stream pointer) of a call on `device`: inside the context the
    device is current and allocations belong to the stream that the call runs
    on, so that a workspace freed at the end of the call is not handed to
    another stream while its kernels still run."""
    if stream is None:
        index = device.index
        if _current_device() == index:
            return _HERE, _raw_stream(index)
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


# After a call that wrote tensors of the caller's through their addresses: autograd
# has to see that one it saved is no longer what it was (a list costs 50 ns per tensor).
_written = torch.autograd.graph.increment_version


def transition_shape(rows: int, C: int, H: int, activation: str = "silu", grads_bf16: bool = False) -> TransitionShape:
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}")
    return TransitionShape(rows, C, H, ACTIVATIONS[activation], FLAG_GRADS_BF16 if grads_bf16 else 0)


def transition_workspace_bytes(rows: int, C: int, H: int) -> int:
    """Workspace of the transition's backward; 0 for an unsupported shape."""
    s = transition_shape(rows, C, H)
    return int(load().triattn_transition_workspace_bytes(ctypes.byref(s)))


def _fits(t, device: int, shape, dtype) -> bool:
    return t is not None and t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous()


def _transition_check(z, mask, ln_w, ln_b, w_in, w_o):
    if z.dim() < 1 or w_o.dim() != 2:
        raise ValueError("z must be [..., C] and w_o [H, C]")
    lead, C, H = z.shape[:-1], z.shape[-1], w_o.shape[0]
    # one look at every tensor, what is wrong is found out below: a call on a few
    # rows takes the GPU 5 us, so the host's 12 are what counts there
    dev, bf16, f32 = z.get_device(), torch.bfloat16, torch.float32
    if not (dev >= 0 and z.dtype is bf16 and z.is_contiguous() and _fits(ln_w, dev, (C,), f32)
            and _fits(ln_b, dev, (C,), f32) and _fits(w_in, dev, (C, 2 * H), bf16) and _fits(w_o, dev, (H, C), bf16)
            and (mask is None or _fits(mask, dev, lead, bf16))):
        _check(z, "z", z.shape)
        _check(ln_w, "ln_w", (C,), torch.float32)
        _check(ln_b, "ln_b", (C,), torch.float32)
        _check(w_in, "w_in", (C, 2 * H))
        _check(w_o, "w_o", (H, C))
        if mask is not None:
            _check(mask, "mask", lead)
        _same_device(z.device, mask=mask, ln_w=ln_w, ln_b=ln_b, w_in=w_in, w_o=w_o)
    return lead.numel(), C, H


def triattn_transition_fwd(z, mask, ln_w, ln_b, w_in, w_o, activation: str = "silu", *, out=None, stream=None):
    """Transition (gated feed-forward block) forward over the rows of z
    [..., C] bf16: out = mask * ((act(a) * b) w_o), [a | b] = LayerNorm(z) w_in.
    ``mask`` [...] bf16 (1 keeps a row, 0 leaves it out) or None; ``activation``
    "silu", "sigmoid" or "gelu" (tanh form).  Returns out [..., C] bf16."""
    M, C, H = _transition_check(z, mask, ln_w, ln_b, w_in, w_o)
    s = transition_shape(M, C, H, activation)
    here, sp = _on_stream(z.device, stream)
    given = out
    with here:
        if out is None:
            out = torch.empty_like(z)
        else:
            _check(out, "out", z.shape)
            _same_device(z.device, out=out)
        code = load().triattn_transition_fwd(ctypes.byref(s), z.data_ptr(), None if mask is None else mask.data_ptr(),
                                             ln_w.data_ptr(), ln_b.data_ptr(), w_in.data_ptr(), w_o.data_ptr(),
                                             out.data_ptr(), sp)
    _raise(code, "triattn_transition_fwd")
    if given is not None:
        _written(out)
    return out


def triattn_transition_bwd(z, mask, ln_w, ln_b, w_in, w_o, d_out, activation: str = "silu", *,
                           grads_bf16: bool = False, workspace=None, out=None, stream=None):
    """Backward of <out, d_out>; the forward's intermediates are computed
    again.  Returns (dz bf16, d_ln_w, d_ln_b, d_w_in, d_w_o), the parameter
    gradients FP32, or with ``grads_bf16`` BF16 (one rounding of the FP32 sums)."""
    M, C, H = _transition_check(z, mask, ln_w, ln_b, w_in, w_o)
    if not _fits(d_out, z.get_device(), z.shape, torch.bfloat16):
        _check(d_out, "d_out", z.shape)
        _same_device(z.device, d_out=d_out)
    s = transition_shape(M, C, H, activation, grads_bf16)
    lib = load()
    need = lib.triattn_transition_workspace_bytes(ctypes.byref(s))
    if need == 0:
        raise TriAttnError(ERR_UNSUPPORTED, "triattn_transition_bwd")
    dt = torch.bfloat16 if grads_bf16 else torch.float32
    here, sp = _on_stream(z.device, stream)
    given = out
    with here:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=z.device)
        else:
            _same_device(z.device, workspace=workspace)
        if out is None:
            out = (torch.empty_like(z),) + tuple(torch.empty_like(t, dtype=dt) for t in (ln_w, ln_b, w_in, w_o))
            dz, dlw, dlb, dwi, dwo = out
        else:
            dz, dlw, dlb, dwi, dwo = out
            _check(dz, "dz", z.shape)
            for name, t, shape in (("d_ln_w", dlw, (C,)), ("d_ln_b", dlb, (C,)), ("d_w_in", dwi, (C, 2 * H)),
                                   ("d_w_o", dwo, (H, C))):
                _check(t, name, shape, dt)
            _same_device(z.device, dz=dz, d_ln_w=dlw, d_ln_b=dlb, d_w_in=dwi, d_w_o=dwo)
        code = lib.triattn_transition_bwd(ctypes.byref(s), z.data_ptr(), None if mask is None else mask.data_ptr(),
                                          ln_w.data_ptr(), ln_b.data_ptr(), w_in.data_ptr(), w_o.data_ptr(),
                                          d_out.data_ptr(), dz.data_ptr(), dlw.data_ptr(), dlb.data_ptr(),
                                          dwi.data_ptr(), dwo.data_ptr(), workspace.data_ptr(), _bytes(workspace), sp)
    _raise(code, "triattn_transition_bwd")
    if given is not None:
        _written([dz, dlw, dlb, dwi, dwo])
    return dz, dlw, dlb, dwi, dwo


def _address(t):
    return None if t is None else t.data_ptr()


def _rows_pair(a, b, names, shape, dev: int):
    """The layout that two [B, N_o, H, N, D] views share, None where both are contiguous."""
    bf16 = torch.bfloat16
    if (a.dtype is bf16 and b.dtype is bf16 and a.shape == shape and b.shape == shape and dev >= 0
            and a.get_device() == dev and b.get_device() == dev):
        if a.is_contiguous() and b.is_contiguous():
            return None
        if a.stride() == b.stride():
            return layout_of(a)
    lay = layout_of(a)
    for name, t in zip(names, (a, b)):
        _check_view(t, name, shape, lay)
    _same_device(torch.device("cuda", dev), **dict(zip(names, (a, b))))
    return lay


def qk_norm_shape(shape, w, rotary: str = "half", theta: float = 10000.0, eps: float = 1e-6) -> QKNormShape:
    """Of q's shape and its weight, [H, D] or [D]."""
    return QKNormShape.from_buffer_copy(_qk_norm_plan(tuple(shape), w.dim() == 1, rotary, theta, eps)[0])


@functools.lru_cache(maxsize=256)
def _qk_norm_plan(shape, shared, rotary, theta, eps):
    """(struct, its reference, the weights' shape, the positions' shape, the
    backward's workspace) of a call of these sizes."""
    if len(shape) != 5:
        raise ValueError("q must be [B, N_o, H, N, D]")
    if rotary not in ROTARY:
        raise ValueError(f"rotary must be one of {tuple(ROTARY)}")
    B, No, H, N, D = shape
    s = QKNormShape(B, No, N, H, D, 1 if shared else H, ROTARY[rotary], eps, theta, 0)
    ref = ctypes.byref(s)
    return s, ref, (D,) if shared else (H, D), (B, N), load().triattn_qk_norm_workspace_bytes(ref)


def _qk_norm_check(q, k, w_q, w_k, positions, rotary, theta, eps):
    """(shape's reference, the backward's workspace, q's layout) of valid arguments.
    The tests of a usual call stand in one line each: the host's time is what a
    small call takes."""
    shape, dev, f32, bf16 = q.shape, q.get_device(), torch.float32, torch.bfloat16
    _, ref, w_shape, p_shape, need = _qk_norm_plan(shape, w_q.dim() == 1, rotary, theta, eps)
    if (q.dtype is bf16 and k.dtype is bf16 and k.shape == shape and dev >= 0 and k.get_device() == dev
            and q.is_contiguous() and k.is_contiguous()):
        lay = None
    else:
        lay = _rows_pair(q, k, ("q", "k"), shape, dev)
    if not (w_q.dtype is f32 and w_k.dtype is f32 and w_q.shape == w_shape and w_k.shape == w_shape
            and w_q.get_device() == dev and w_k.get_device() == dev and w_q.is_contiguous() and w_k.is_contiguous()
            and (positions is None or _fits(positions, dev, p_shape, torch.int32))):
        _check(w_q, "w_q", w_shape, f32)
        _check(w_k, "w_k", w_shape, f32)
        if positions is not None:
            _check(positions, "positions", p_shape, torch.int32)
        _same_device(q.device, w_q=w_q, w_k=w_k, positions=positions)
    return ref, need, lay


def _rows_like(q, lay):
    """A contiguous tensor of q's shape."""
    return torch.empty_like(q) if lay is None else torch.empty(q.shape, dtype=q.dtype, device=q.device)


def _ref(lay):
    return None if lay is None else ctypes.byref(lay)


def triattn_qk_norm_fwd(q, k, w_q, w_k, positions=None, rotary: str = "half", *, theta: float = 10000.0,
                        eps: float = 1e-6, out=None, stream=None):
    """Norms of queries and keys for each head with the position rotation:
    y = R(pos) (w[h] * x rsqrt(mean x^2 + eps)) for every row of q and k
    [B, N_o, H, N, D] bf16 (contiguous, or views as tri_attn_fwd_strided takes
    them).  ``w_q``, ``w_k`` [H, D] or [D] fp32; ``positions`` [B, N] int32 (the
    token's index if None); ``rotary`` "half", "interleaved" or "none".  Returns
    (q, k) normed, contiguous, or written into the views ``out``."""
    if out is None and stream is None:
        done = _host().qk_norm_fwd(q, k, w_q, w_k, positions, ROTARY.get(rotary, -1), theta, eps)
        if done is not None:
            return done
    ref, _, lay = _qk_norm_check(q, k, w_q, w_k, positions, rotary, theta, eps)
    here, sp = _on_stream(q.device, stream)
    given, lo = out, None
    with here:
        if out is None:
            out = _rows_like(q, lay), _rows_like(q, lay)
        else:
            lo = _rows_pair(*out, ("q_out", "k_out"), q.shape, q.get_device())
        qo, ko = out
        code = load().triattn_qk_norm_fwd(ref, q.data_ptr(), k.data_ptr(), _ref(lay), w_q.data_ptr(),
                                          w_k.data_ptr(), _address(positions), qo.data_ptr(), ko.data_ptr(), _ref(lo),
                                          sp)
    _raise(code, "triattn_qk_norm_fwd")
    if given is not None:
        _written([qo, ko])
    return qo, ko


def triattn_qk_norm_bwd(q, k, w_q, w_k, d_q_out, d_k_out, positions=None, rotary: str = "half", *,
                        theta: float = 10000.0, eps: float = 1e-6, workspace=None, out=None, stream=None):
    """Backward of <q_out, d_q_out> + <k_out, d_k_out>; the norms are computed
    again from q and k.  Returns (dq, dk bf16, d_w_q, d_w_k fp32); ``out`` may
    pass them preallocated, dq and dk also as views, or d_q_out and d_k_out
    themselves."""
    if out is None and stream is None and workspace is None:
        done = _host().qk_norm_bwd(q, k, w_q, w_k, d_q_out, d_k_out, positions, ROTARY.get(rotary, -1), theta, eps)
        if done is not None:
            return done
    ref, need, lay = _qk_norm_check(q, k, w_q, w_k, positions, rotary, theta, eps)
    ld = _rows_pair(d_q_out, d_k_out, ("d_q_out", "d_k_out"), q.shape, q.get_device())
    if need == 0:
        raise TriAttnError(ERR_UNSUPPORTED, "triattn_qk_norm_bwd")
    here, sp = _on_stream(q.device, stream)
    given, lg = out, None
    with here:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            _same_device(q.device, workspace=workspace)
        if out is None:
            dq, dk, dwq, dwk = (_rows_like(q, lay), _rows_like(q, lay), torch.empty_like(w_q), torch.empty_like(w_k))
        else:
            dq, dk, dwq, dwk = out
            lg = _rows_pair(dq, dk, ("dq", "dk"), q.shape, q.get_device())
            _check(dwq, "d_w_q", w_q.shape, torch.float32)
            _check(dwk, "d_w_k", w_k.shape, torch.float32)
            _same_device(q.device, d_w_q=dwq, d_w_k=dwk)
        code = load().triattn_qk_norm_bwd(ref, q.data_ptr(), k.data_ptr(), _ref(lay), w_q.data_ptr(),
                                       w_k.data_ptr(), _address(positions), d_q_out.data_ptr(), d_k_out.data_ptr(),
                                       _ref(ld), dq.data_ptr(), dk.data_ptr(), _ref(lg), dwq.data_ptr(),
                                       dwk.data_ptr(), workspace.data_ptr(), _bytes(workspace), sp)
    _raise(code, "triattn_qk_norm_bwd")
    if given is not None:
        _written([dq, dk, dwq, dwk])
    return dq, dk, dwq, dwk


def relpos_shape(B: int, N: int, F: int, buckets: int, layout: str = "heads", kind: str = "clip",
                 max_distance: int = 32, dout_fp32: bool = False) -> RelposShape:
    return RelposShape.from_buffer_copy(_relpos_plan(B, N, F, buckets, layout, kind, max_distance, dout_fp32)[0])


@functools.lru_cache(maxsize=256)
def _relpos_plan(B, N, F, buckets, layout, kind, max_distance, dout_fp32):
    """(struct, its reference, the planes' or features' shape, the backward's
    workspace) of a call of these sizes."""
    if layout not in RELPOS_LAYOUTS:
        raise ValueError(f"layout must be one of {tuple(RELPOS_LAYOUTS)}")
    if kind not in BUCKETS:
        raise ValueError(f"kind must be one of {tuple(BUCKETS)}")
    s = RelposShape(B, N, F, RELPOS_LAYOUTS[layout], BUCKETS[kind], buckets, max_distance,
                    FLAG_DOUT_FP32 if dout_fp32 else 0)
    ref = ctypes.byref(s)
    shape = (B, F, N, N) if layout == "heads" else (B, N, N, F)
    return s, ref, shape, load().triattn_relpos_workspace_bytes(ref)


def _relpos_ids(positions, chains, B, N, device):
    dev, i32 = device.index, torch.int32
    if ((positions is None or _fits(positions, dev, (B, N), i32))
            and (chains is None or _fits(chains, dev, (B, N), i32))):
        return
    for name, t in (("positions", positions), ("chains", chains)):
        if t is not None:
            _check(t, name, (B, N), torch.int32)
    _same_device(device, positions=positions, chains=chains)


def triattn_relpos_fwd(table, base=None, positions=None, chains=None, *, layout: str = "heads", kind: str = "clip",
                       max_distance: int = 32, out=None, stream=None):
    """Learned relative position bias: out = base + table[bucket(i, j)], planes
    [B, F, N, N] ("heads": the core's bias) or pair features [B, N, N, F]
    ("pairs"), bf16.  ``table`` [buckets, F] fp32; ``base`` of out's shape or
    None (then positions or out give B and N); ``positions`` [B, N] int32 (the
    token's index if None); ``chains`` [B, N] int32 or None: pairs of different
    chains take the table's last row, which it has for them.  ``kind`` "clip":
    2 max_distance + 1 rows; "log": an even number of rows, logarithmic from a
    quarter of them to max_distance.  ``out`` may be base."""
    if out is None and stream is None:
        done = _host().relpos_fwd(table, base, positions, chains, RELPOS_LAYOUTS.get(layout, -1), BUCKETS.get(kind, -1),
                                  max_distance)
        if done is not None:
            return done
    if table.dim() != 2:
        raise ValueError("table must be [buckets, F]")
    K, F = table.shape
    device = table.device
    like = base if base is not None else out
    if like is not None:
        if like.dim() != 4:
            raise ValueError("base must be [B, F, N, N] or [B, N, N, F]")
        B, N = like.shape[0], like.shape[2]
    elif positions is not None and positions.dim() == 2:
        B, N = positions.shape
    else:
        raise ValueError("base, out or positions [B, N] must be given")
    _, ref, shape, need = _relpos_plan(B, N, F, K, layout, kind, max_distance, False)
    if need == 0 and out is None and base is None:  # before an output of any size is allocated
        raise TriAttnError(ERR_UNSUPPORTED, "triattn_relpos_fwd")
    dev = table.get_device()
    if not (_fits(table, dev, (K, F), torch.float32) and dev >= 0
            and (base is None or _fits(base, dev, shape, torch.bfloat16))):
        _check(table, "table", (K, F), torch.float32)
        if base is not None:
            _check(base, "base", shape)
            _same_device(device, base=base)
    _relpos_ids(positions, chains, B, N, device)
    here, sp = _on_stream(device, stream)
    given = out
    with here:
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=device)
        else:
            _check(out, "out", shape)
            _same_device(device, out=out)
        code = load().triattn_relpos_fwd(ref, table.data_ptr(), _address(base), _address(positions),
                                         _address(chains), out.data_ptr(), sp)
    _raise(code, "triattn_relpos_fwd")
    if given is not None:
        _written(out)
    return out


def triattn_relpos_bwd(d_out, buckets: int, positions=None, chains=None, *, layout: str = "heads", kind: str = "clip",
                       max_distance: int = 32, workspace=None, out=None, stream=None):
    """Gradient of the table of ``buckets`` rows: d_table [buckets, F] fp32 from
    d_out [B, F, N, N] (bf16, or fp32 as tri_attn_bwd(..., dbias_fp32=True)
    gives it) or [B, N, N, F] (bf16).  The gradient of base is d_out itself."""
    if out is None and stream is None and workspace is None:
        done = _host().relpos_bwd(d_out, buckets, positions, chains, RELPOS_LAYOUTS.get(layout, -1),
                                  BUCKETS.get(kind, -1), max_distance)
        if done is not None:
            return done
    if d_out.dim() != 4:
        raise ValueError("d_out must be [B, F, N, N] or [B, N, N, F]")
    B, N = d_out.shape[0], d_out.shape[2]
    F = d_out.shape[1] if layout == "heads" else d_out.shape[3]
    f32 = d_out.dtype is torch.float32 and layout == "heads"
    _, ref, shape, need = _relpos_plan(B, N, F, buckets, layout, kind, max_distance, f32)
    _check(d_out, "d_out", shape, torch.float32 if f32 else torch.bfloat16)
    device = d_out.device
    _relpos_ids(positions, chains, B, N, device)
    if need == 0:
        raise TriAttnError(ERR_UNSUPPORTED, "triattn_relpos_bwd")
    here, sp = _on_stream(device, stream)
    given = out
    with here:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            _same_device(device, workspace=workspace)
        if out is None:
            out = torch.empty((buckets, F), dtype=torch.float32, device=device)
        else:
            _check(out, "d_table", (buckets, F), torch.float32)
            _same_device(device, d_table=out)
        code = load().triattn_relpos_bwd(ref, d_out.data_ptr(), _address(positions), _address(chains),
                                      out.data_ptr(), workspace.data_ptr(), _bytes(workspace), sp)
    _raise(code, "triattn_relpos_bwd")
    if given is not None:
        _written(out)
    return out


GRAD_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_dtype_of = operator.attrgetter("dtype")


def _dense(t) -> bool:
    """Whether the elements of a strided tensor fill one block of memory, each once."""
    n = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda p: p[1]):
        if size != 1:
            if stride != n:
                return False
            n *= size
    return True


def _tensor_table(tensors, name, device):
    """The triattn_tensor array of a list as bytes (address, elements and dtype,
    eight each), its elements and dtypes, and whether all are contiguous.
    Column by column: a model has thousands of gradients, and the host's time
    per tensor is what counts."""
    n = len(tensors)
    try:
        numel = list(map(torch.Tensor.numel, tensors))
        kinds = list(map(GRAD_DTYPES.__getitem__, map(_dtype_of, tensors)))
        rows = [0] * (3 * n)
        rows[0::3], rows[1::3], rows[2::3] = map(torch.Tensor.data_ptr, tensors), numel, kinds
        table = struct.pack(f"{3 * n}q", *rows)
        plain = (all(map(torch.Tensor.is_contiguous, tensors))
                 and set(map(torch.Tensor.get_device, tensors)) <= {device.index})
    except (KeyError, RuntimeError):
        table = numel = kinds = None
        plain = False
    if not plain:
        for i, t in enumerate(tensors):
            if t.dtype not in GRAD_DTYPES or t.device != device or t.layout != torch.strided:
                raise ValueError(f"{name}[{i}] must be a strided bfloat16 or float32 tensor on {device}")
            if not t.is_contiguous() and t.numel() and not _dense(t):
                raise ValueError(f"{name}[{i}] must fill one block of memory")
        if table is None:
            raise ValueError(f"{name} holds a tensor without an address")
    return table, numel, kinds, plain


def _grad_call(tensors, norm_type):
    tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    kinds = {2.0: 0, float("inf"): 1}
    if float(norm_type) not in kinds:
        raise ValueError("norm_type must be 2 or inf")
    device = tensors[0].device if tensors else torch.device("cuda", torch.cuda.current_device())
    if device.type != "cuda":
        raise ValueError("the gradients must be CUDA tensors")
    return tensors, kinds[float(norm_type)], device


def triattn_grad_norm(tensors, norm_type: float = 2.0, *, stream=None):
    """Norm of all elements of ``tensors`` (BF16 and FP32 CUDA tensors, mixed):
    2 or inf.  Returns a 0-dim FP32 tensor; nothing waits for the device."""
    tensors, kind, device = _grad_call(tensors, norm_type)
    n = len(tensors)
    table, _, _, _ = _tensor_table(tensors, "tensors", device)
    here, sp = _on_stream(device, stream)
    lib = load()
    with here:
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws = torch.empty(lib.triattn_grad_norm_workspace_bytes(n), dtype=torch.uint8, device=device)
        code = lib.triattn_grad_norm(table, n, kind, norm.data_ptr(), ws.data_ptr(), ws.numel(), sp)
    _raise(code, "triattn_grad_norm")
    return norm


def triattn_clip_grad_norm(tensors, max_norm: float, norm_type: float = 2.0, *, out=None, stream=None):
    """Scale ``tensors`` (BF16 and FP32 CUDA tensors, mixed) by
    min(1, max_norm / (norm + 1e-6)), in place, or into ``out`` (a list of
    tensors of the same dtypes and sizes, in the same memory order, that share
    no memory with ``tensors``).  Returns the norm before clipping as a 0-dim
    FP32 tensor; nothing waits for the device.  A tensor may not be listed
    twice.  A captured call keeps the tensors' addresses."""
    tensors, kind, device = _grad_call(tensors, norm_type)
    n = len(tensors)
    table, numel, kinds, plain = _tensor_table(tensors, "tensors", device)
    into = None
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != n:
            raise ValueError(f"out has {len(out)} tensors, expected {n}")
        into, numel_out, kinds_out, plain_out = _tensor_table(out, "out", device)
        if not (numel == numel_out and kinds == kinds_out and plain and plain_out):
            for i, (a, b) in enumerate(zip(tensors, out)):
                if (a.numel() != b.numel() or a.dtype != b.dtype
                        or not (plain and plain_out) and (a.shape != b.shape or a.stride() != b.stride())):
                    raise ValueError(f"out[{i}] does not match tensors[{i}]")
    here, sp = _on_stream(device, stream)
    lib = load()
    with here:
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws = torch.empty(lib.triattn_grad_norm_workspace_bytes(n), dtype=torch.uint8, device=device)
        code = lib.triattn_clip_grad_norm(table, into, n, kind, float(max_norm), norm.data_ptr(), ws.data_ptr(),
                                          ws.numel(), sp)
    _raise(code, "triattn_clip_grad_norm")
    _written(tensors if out is None else out)
    return norm


def _matrix_table(tensors, name, device, of=None):
    """The triattn_matrix array of a list of 2-D tensors as bytes (address, rows,
    columns, stride and dtype, eight each), and their shapes; as outputs, of the
    shapes ``of``.  For the lists that the native part does not take."""
    rows = []
    for i, t in enumerate(tensors):
        if of is not None and (t.shape != of[i] or t.dtype is not torch.bfloat16):
            raise ValueError(f"{name}[{i}] must be a bfloat16 tensor of the shape of tensors[{i}]")
        if t.dim() != 2 or t.dtype not in GRAD_DTYPES or t.device != device or t.layout != torch.strided:
            raise ValueError(f"{name}[{i}] must be a 2-D bfloat16 or float32 tensor on {device}")
        r, c = t.shape
        stride = t.stride(0) if r > 1 else c
        if (c > 1 and t.stride(1) != 1) or (stride < c and t.numel()):
            raise ValueError(f"{name}[{i}] must have contiguous rows")
        rows += (t.data_ptr(), r, c, stride, GRAD_DTYPES[t.dtype])
    return struct.pack(f"{len(rows)}q", *rows), [t.shape for t in tensors]


ORTHOGONALIZE = (3.4445, -4.7750, 2.0315)


def triattn_orthogonalize(tensors, steps: int = 5, *, coefficients=ORTHOGONALIZE, eps: float = 1e-7, out=None,
                          workspace=None, stream=None):
    """Orthogonalise a list of matrices (2-D BF16 or FP32 CUDA tensors, mixed,
    with contiguous rows) by Newton-Schulz products: X = G / (|G| + eps), then
    ``steps`` times X <- a X + (b A + c A^2) X, A = X X^T.  Returns the list of
    results (BF16, of the same shapes), or writes them into ``out``, whose tensors
    may be those of ``tensors``; nothing waits for the device.  A captured call
    keeps the tensors' addresses."""
    tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    if len(coefficients) != 3:
        raise ValueError("coefficients must be three numbers")
    device = tensors[0].device if tensors else torch.device("cuda", torch.cuda.current_device())
    if device.type != "cuda":
        raise ValueError("the matrices must be CUDA tensors")
    n = len(tensors)
    here, sp = _on_stream(device, stream)
    given = out
    lib = load()
    with here:
        if out is not None:
            out = [out] if isinstance(out, torch.Tensor) else list(out)
            if len(out) != n:
                raise ValueError(f"out has {len(out)} tensors, expected {n}")
        tables = _host().matrix_tables(tensors, out, device.index)
        table, into = tables if tables is not None else (_matrix_table(tensors, "tensors", device)[0], None)
        if out is None:
            out = [torch.empty(t.shape, dtype=torch.bfloat16, device=device) for t in tensors]
        if into is None:
            into, _ = _matrix_table(out, "out", device, [t.shape for t in tensors])
        need = lib.triattn_orthogonalize_workspace_bytes(table, n)
        if need == 0:
            raise TriAttnError(ERR_UNSUPPORTED, "triattn_orthogonalize")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            _same_device(device, workspace=workspace)
        code = lib.triattn_orthogonalize(table, into, n, int(steps), struct.pack("3f", *map(float, coefficients)),
                                         float(eps), workspace.data_ptr(), _bytes(workspace), sp)
    _raise(code, "triattn_orthogonalize")
    if given is not None:
        _written(out)
    return out


def gemm(a, b, *, ta: bool = False, tb: bool = False, out_f32: bool = False, out=None, stream=None):
    """The library's tensor-core GEMM: op(a) @ op(b) for BF16 CUDA tensors,
    2-D or 3-D (batched, leading dimension), contiguous; op transposes the
    last two dimensions when ta / tb.  FP32 accumulation; BF16 output, or
    FP32 with ``out_f32``."""
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16 or not (a.is_cuda and b.is_cuda):
        raise ValueError("a and b must be CUDA bfloat16 tensors")
    if a.dim() != b.dim() or a.dim() not in (2, 3) or not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous, both 2-D or both 3-D")
    batched = a.dim() == 3
    a3, b3 = (a, b) if batched else (a[None], b[None])
    batch = a3.shape[0]
    M, K = (a3.shape[2], a3.shape[1]) if ta else (a3.shape[1], a3.shape[2])
    Kb, N = (b3.shape[2], b3.shape[1]) if tb else (b3.shape[1], b3.shape[2])
    if K != Kb or b3.shape[0] != batch:
        raise ValueError("shapes do not match")
    dt = torch.float32 if out_f32 else torch.bfloat16
    c = out if out is not None else torch.empty((batch, M, N), dtype=dt, device=a.device)
    lib = load()
    need = int(lib.triattn_gemm_workspace_bytes(M, N, K, batch))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=a.device)
    code = lib.triattn_gemm(int(ta), int(tb), M, N, K, _ptr(a3), a3.shape[2], _ptr(b3), b3.shape[2], _ptr(c), N,
                            int(out_f32), batch, a3.shape[1] * a3.shape[2], b3.shape[1] * b3.shape[2], M * N,
                            _ptr(ws), ctypes.c_size_t(ws.numel()), _stream_ptr(stream))
    _raise(code, "triattn_gemm")
    return c if batched else c[0]


class TriAttnFunction(torch.autograd.Function):
    """Autograd wrapper: forward saves o, lse and the residual; backward runs
    the compensated key-tile-parallel backward."""

    @staticmethod
    def forward(ctx, q, k, v, bias, mask=None):
        o, lse, resid = tri_attn_fwd(q, k, v, bias, mask, save_residual=True)
        ctx.save_for_backward(q, k, v, bias, o, lse, resid)
        ctx.mask = mask
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, bias, o, lse, resid = ctx.saved_tensors
        dq, dk, dv, dbias = tri_attn_bwd(q, k, v, bias, ctx.mask, o, resid, lse, do.contiguous())
        return dq, dk, dv, dbias, None


def triangle_attention(q, k, v, bias, mask=None):
    """Differentiable triangular attention (BF16 in, BF16 out)."""
    return TriAttnFunction.apply(q, k, v, bias, mask)
