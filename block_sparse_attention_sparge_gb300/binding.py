"""Thin ctypes binding over ``libsparge.so`` (argument marshalling only).

Every step of the hot path runs in the library's CUDA kernels; this module
only allocates outputs with torch, passes raw device pointers, sizes and the
current CUDA stream, and turns a negative status into ``SpargeError``.  There
is no CPU fallback: if the library is missing or no GPU is present, calls
raise.
"""

from __future__ import annotations

import array
import ctypes
import functools
import math
import os
import struct

import torch

from . import _build

__all__ = [
    "SpargeError",
    "Shape",
    "load_library",
    "library_path",
    "status_string",
    "sparge_pool",
    "sparge_mask",
    "sparge_mask_from_prob",
    "sparge_attn_fwd",
    "sparge_attn_bwd",
    "RopeAxes",
    "sparge_heads_fwd",
    "sparge_heads_bwd",
    "sparge_resnorm_fwd",
    "sparge_resnorm_bwd",
    "sparge_clip_grads",
    "sparge_cross_fwd",
    "sparge_cross_bwd",
    "sparge_orthogonalize",
    "sparge_muon_step",
    "sparge_debug_wait_probe",
    "num_blocks",
    "SPARGE_OK",
    "SPARGE_ERR_INVALID_ARG",
    "SPARGE_ERR_UNSUPPORTED",
    "SPARGE_ERR_MISALIGNED",
    "SPARGE_ERR_WORKSPACE",
    "SPARGE_ERR_CUDA",
    "SPARGE_ERR_TIMEOUT",
]

SPARGE_OK = 0
SPARGE_ERR_INVALID_ARG = -1
SPARGE_ERR_UNSUPPORTED = -2
SPARGE_ERR_MISALIGNED = -3
SPARGE_ERR_WORKSPACE = -4
SPARGE_ERR_CUDA = -5
SPARGE_ERR_TIMEOUT = -6

BLOCK_Q = 128
BLOCK_KV = 64


class SpargeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("block_q", ctypes.c_int32), ("block_kv", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("turn", ctypes.c_uint64 * 64), ("axis", ctypes.c_uint8 * 64)]


class HeadsPart(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64 * 3),
                ("weight", ctypes.c_void_p), ("y", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("dx_stride", ctypes.c_int64 * 3), ("dweight", ctypes.c_void_p),
                ("H", ctypes.c_int32), ("plain", ctypes.c_int32)]


class Heads(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("x_type", ctypes.c_int32), ("weight_type", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("n_parts", ctypes.c_int32),
                ("rope", ctypes.c_void_p), ("grid", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("pos_batch", ctypes.c_int32), ("part", HeadsPart * 3)]


class Resnorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("C", ctypes.c_int32), ("x_type", ctypes.c_int32),
                ("branch_type", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("unit_offset", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("branch", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p),
                ("gate_groups", ctypes.c_int32), ("scale_groups", ctypes.c_int32),
                ("shift_groups", ctypes.c_int32),
                ("gate_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("shift_stride", ctypes.c_int64), ("post_weight", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("h", ctypes.c_void_p), ("stats", ctypes.c_void_p),
                ("dy", ctypes.c_void_p), ("dh", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("dbranch", ctypes.c_void_p), ("dgate", ctypes.c_void_p),
                ("dscale", ctypes.c_void_p), ("dshift", ctypes.c_void_p),
                ("dpost", ctypes.c_void_p)]


_HEADS_TENSOR = (ctypes.c_void_p, ctypes.c_int64 * 3)


class Cross(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Bk", ctypes.c_int32), ("H", ctypes.c_int32),
                ("Hk", ctypes.c_int32), ("N", ctypes.c_int32), ("M", ctypes.c_int32),
                ("d", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("kv_len", ctypes.c_void_p),
                *((n + s, t) for n in ("q", "k", "v", "o")
                  for s, t in zip(("", "_stride"), _HEADS_TENSOR)),
                ("lse", ctypes.c_void_p),
                *((n + s, t) for n in ("dout", "dq", "dk", "dv")
                  for s, t in zip(("", "_stride"), _HEADS_TENSOR)),
                ("status", ctypes.c_void_p)]


class Matrix(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("grad_type", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("grad", ctypes.c_void_p),
                ("grad_stride", ctypes.c_int64), ("momentum", ctypes.c_void_p),
                ("momentum_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("keep", ctypes.c_float), ("step", ctypes.c_float)]


class Ortho(ctypes.Structure):
    _fields_ = [("mats", ctypes.c_void_p), ("n", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("eps", ctypes.c_float), ("mu", ctypes.c_float), ("nesterov", ctypes.c_int32),
                ("update", ctypes.c_int32), ("half", ctypes.c_int32), ("status", ctypes.c_void_p)]


_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_I = ctypes.c_int
_SHP = ctypes.POINTER(Shape)

_SIGNATURES = {
    "sparge_version": ([], _I),
    "sparge_status_string": ([_I], ctypes.c_char_p),
    "sparge_pool": ([_SHP, _P, _P, _P, _P, _P], _I),
    "sparge_mask_workspace_bytes": ([_SHP, ctypes.POINTER(_SZ)], _I),
    "sparge_mask": ([_SHP, _P, _P, _F, _F, _F, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "sparge_mask_from_prob": ([_SHP, _P, _F, _F, _P, _P, _P, _P, _P, _P], _I),
    "sparge_mask_noalloc": ([_SHP, _P, _P, _F, _F, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "sparge_attn_fwd": ([_SHP, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P], _I),
    "sparge_attn_bwd_workspace_bytes": ([_SHP, ctypes.POINTER(_SZ)], _I),
    "sparge_attn_bwd": ([_SHP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ,
                         _P, _P], _I),
    "sparge_rope_init": ([ctypes.POINTER(Rope), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                          ctypes.c_double, ctypes.POINTER(ctypes.c_double), ctypes.c_int32], _I),
    "sparge_heads_fwd": ([_P, _P], _I),
    "sparge_heads_bwd_workspace_bytes": ([_P, ctypes.POINTER(_SZ)], _I),
    "sparge_heads_bwd": ([_P, _P, _SZ, _P], _I),
    "sparge_resnorm_fwd": ([_P, _P], _I),
    "sparge_resnorm_bwd_workspace_bytes": ([_P, ctypes.POINTER(_SZ)], _I),
    "sparge_resnorm_bwd": ([_P, _P, _SZ, _P], _I),
    "sparge_clip_workspace_bytes": ([ctypes.c_int32, ctypes.POINTER(_SZ)], _I),
    "sparge_clip_grads": ([_P, _P, ctypes.c_int32, _F, _F, _P, _P, _SZ, _P], _I),
    "sparge_cross_fwd_workspace_bytes": ([_P, ctypes.POINTER(_SZ)], _I),
    "sparge_cross_fwd": ([_P, _P, _SZ, _P], _I),
    "sparge_cross_bwd_workspace_bytes": ([_P, ctypes.POINTER(_SZ)], _I),
    "sparge_cross_bwd": ([_P, _P, _SZ, _P], _I),
    "sparge_orthogonalize_workspace_bytes": ([_P, ctypes.POINTER(_SZ)], _I),
    "sparge_orthogonalize_check": ([_P], _I),
    "sparge_orthogonalize": ([_P, _P, _SZ, _P], _I),
    "sparge_status_copy_async": ([_P, _P, _P], _I),
    "sparge_read_status": ([_P, _P, ctypes.POINTER(ctypes.c_int32)], _I),
    "sparge_debug_wait_probe": ([_P, ctypes.c_uint64, _P], _I),
}

_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = True):
    """Loads libsparge.so (building it first if it is absent or stale and nvcc
    is available).  Raises if it cannot be loaded: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if build_if_missing and (not os.path.exists(path) or _build.is_stale()):
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"libsparge.so not found at {path}; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return load_library(build_if_missing=False).sparge_status_string(int(code)).decode()
    except Exception:  # pragma: no cover - only while the library is unavailable
        return f"status {code}"


def _check(code: int, where: str):
    if code != SPARGE_OK:
        raise SpargeError(code, where)


def num_blocks(n: int, b: int) -> int:
    return (n + b - 1) // b


def _shape(q: torch.Tensor, block_q=BLOCK_Q, block_kv=BLOCK_KV) -> Shape:
    if q.dim() != 4:
        raise ValueError("expected a [B, H, N, d] tensor")
    B, H, N, d = q.shape
    return Shape(B, H, N, d, block_q, block_kv)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda_bf16(*ts):
    for t in ts:
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise ValueError("expected contiguous bf16 CUDA tensors")


def _read_status(status: torch.Tensor) -> int:
    lib = load_library()
    host = ctypes.c_int32(0)
    _check(lib.sparge_read_status(_ptr(status), _stream(status.device), ctypes.byref(host)),
           "sparge_read_status")
    return host.value


def _finish(status: torch.Tensor, check_status: bool, where: str):
    if check_status:
        code = _read_status(status)
        if code != SPARGE_OK:
            raise SpargeError(code, where + " (device)")


def sparge_pool(q: torch.Tensor, k: torch.Tensor, block_q=BLOCK_Q, block_kv=BLOCK_KV):
    """Block means (fp32) of Q over q-blocks and of K over kv-blocks."""
    _need_cuda_bf16(q, k)
    lib = load_library()
    shp = _shape(q, block_q, block_kv)
    B, H, N, d = q.shape
    qbar = torch.empty((B, H, num_blocks(N, block_q), d), dtype=torch.float32, device=q.device)
    kbar = torch.empty((B, H, num_blocks(N, block_kv), d), dtype=torch.float32, device=q.device)
    _check(lib.sparge_pool(ctypes.byref(shp), _ptr(q), _ptr(k), _ptr(qbar), _ptr(kbar),
                           _stream(q.device)), "sparge_pool")
    return qbar, kbar


def _mask_outputs(B, H, mq, mk, device, want_csc):
    out = {
        "bitmask": torch.empty((B, H, mq, (mk + 31) // 32), dtype=torch.int32, device=device),
        "row_idx": torch.empty((B, H, mq, mk), dtype=torch.int32, device=device),
        "row_cnt": torch.empty((B, H, mq), dtype=torch.int32, device=device),
        "col_idx": None,
        "col_cnt": None,
    }
    if want_csc:
        out["col_idx"] = torch.empty((B, H, mk, mq), dtype=torch.int32, device=device)
        out["col_cnt"] = torch.empty((B, H, mk), dtype=torch.int32, device=device)
    return out


def sparge_mask(q, k, k_frac: float, p: float, softmax_scale: float = 0.0, want_csc=True,
                want_prob=False, want_logit=False, block_q=BLOCK_Q, block_kv=BLOCK_KV,
                workspace=None, out=None):
    """Hybrid Top-k + Top-p block mask.  Returns a dict with ``bitmask``
    (int32 view of the uint32 words), ``row_idx``, ``row_cnt`` and, when asked
    for, ``col_idx``, ``col_cnt``, ``prob``, ``logit``."""
    _need_cuda_bf16(q, k)
    lib = load_library()
    shp = _shape(q, block_q, block_kv)
    B, H, N, d = q.shape
    mq, mk = num_blocks(N, block_q), num_blocks(N, block_kv)
    res = out if out is not None else _mask_outputs(B, H, mq, mk, q.device, want_csc)
    res.setdefault("prob", None)
    res.setdefault("logit", None)
    if want_prob and res["prob"] is None:
        res["prob"] = torch.empty((B, H, mq, mk), dtype=torch.float32, device=q.device)
    if want_logit and res["logit"] is None:
        res["logit"] = torch.empty((B, H, mq, mk), dtype=torch.float32, device=q.device)
    if workspace is None:
        nbytes = ctypes.c_size_t(0)
        _check(lib.sparge_mask_workspace_bytes(ctypes.byref(shp), ctypes.byref(nbytes)),
               "sparge_mask_workspace_bytes")
        workspace = torch.empty(nbytes.value, dtype=torch.uint8, device=q.device)
    _check(lib.sparge_mask(ctypes.byref(shp), _ptr(q), _ptr(k), float(k_frac), float(p),
                           float(softmax_scale), _ptr(res["bitmask"]), _ptr(res["row_idx"]),
                           _ptr(res["row_cnt"]), _ptr(res["col_idx"]), _ptr(res["col_cnt"]),
                           _ptr(res["prob"]), _ptr(res["logit"]), _ptr(workspace),
                           workspace.numel(), None, _stream(q.device)), "sparge_mask")
    return res


def sparge_mask_from_prob(prob: torch.Tensor, k_frac: float, p: float, N: int, d: int = 128,
                          want_csc=True, block_q=BLOCK_Q, block_kv=BLOCK_KV):
    """Hybrid selection on a given fp32 pooled probability map [B, H, Mq, Mk]."""
    if not (prob.is_cuda and prob.dtype == torch.float32 and prob.is_contiguous()):
        raise ValueError("prob must be a contiguous fp32 CUDA tensor")
    lib = load_library()
    B, H, mq, mk = prob.shape
    if mq != num_blocks(N, block_q) or mk != num_blocks(N, block_kv):
        raise ValueError("prob shape does not match N and the block sizes")
    shp = Shape(B, H, N, d, block_q, block_kv)
    res = _mask_outputs(B, H, mq, mk, prob.device, want_csc)
    _check(lib.sparge_mask_from_prob(ctypes.byref(shp), _ptr(prob), float(k_frac), float(p),
                                     _ptr(res["bitmask"]), _ptr(res["row_idx"]),
                                     _ptr(res["row_cnt"]), _ptr(res["col_idx"]),
                                     _ptr(res["col_cnt"]), _stream(prob.device)),
           "sparge_mask_from_prob")
    return res


def sparge_attn_fwd(q, k, v, row_idx, row_cnt, softmax_scale: float = 0.0, check_status=False,
                    out=None, lse=None, status=None, block_kv=BLOCK_KV):
    """Block-sparse attention forward; returns (O bf16, LSE fp32).  The lists
    index kv-blocks of ``block_kv`` tokens (64 or 128)."""
    _need_cuda_bf16(q, k, v)
    lib = load_library()
    shp = _shape(q, BLOCK_Q, block_kv)
    B, H, N, d = q.shape
    o = out if out is not None else torch.empty_like(q)
    lse = lse if lse is not None else torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=q.device)
    _check(lib.sparge_attn_fwd(ctypes.byref(shp), _ptr(q), _ptr(k), _ptr(v), _ptr(row_idx),
                               _ptr(row_cnt), float(softmax_scale), _ptr(o), _ptr(lse), _ptr(st),
                               _stream(q.device)), "sparge_attn_fwd")
    _finish(st, check_status, "sparge_attn_fwd")
    return o, lse


def sparge_attn_bwd(q, k, v, o, lse, dout, row_idx, row_cnt, col_idx, col_cnt,
                    softmax_scale: float = 0.0, check_status=False, workspace=None, out=None,
                    status=None, block_kv=BLOCK_KV):
    """Gradients (dQ, dK, dV) of the block-sparse attention, mask held fixed."""
    _need_cuda_bf16(q, k, v, o, dout)
    lib = load_library()
    shp = _shape(q, BLOCK_Q, block_kv)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        dq, dk, dv = out
    if workspace is None:
        nbytes = ctypes.c_size_t(0)
        _check(lib.sparge_attn_bwd_workspace_bytes(ctypes.byref(shp), ctypes.byref(nbytes)),
               "sparge_attn_bwd_workspace_bytes")
        workspace = torch.empty(nbytes.value, dtype=torch.uint8, device=q.device)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=q.device)
    _check(lib.sparge_attn_bwd(ctypes.byref(shp), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                               _ptr(dout), _ptr(row_idx), _ptr(row_cnt), _ptr(col_idx),
                               _ptr(col_cnt), float(softmax_scale), _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(workspace), workspace.numel(), _ptr(st), _stream(q.device)),
           "sparge_attn_bwd")
    _finish(st, check_status, "sparge_attn_bwd")
    return dq, dk, dv


# ------------------------------------------------- around the attention
#
# The arguments of these calls are packed into the C structs in one go (the
# ctypes classes above describe the same layout, field by field): at small sizes
# a call is as long as the host takes to make it.
_HEADS = struct.Struct("@6ifi3Pi4x" + "P3q3P3qP2i" * 3)
_NO_PART = (0,) * 13
_RESNORM = struct.Struct("@q5if5P3i4x3q12P")
_MATRIX = struct.Struct("@4i" + "Pq" * 3 + "2f")
_ORTHO = struct.Struct("@P2i5f3iP")
_CROSS = struct.Struct("@7ifP" + "P3q" * 4 + "P" + "P3q" * 4 + "P")

_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_HEADS_NORMS = {None: 0, "token": 1, "head": 2}
_NORMS = {None: 0, "layer": 1, "rms": 2}


def _type_of(t: torch.Tensor, what: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bf16 or fp32")
    return code


def _cuda_index(first, *others) -> int:
    """The index of the CUDA device that all of the given tensors are on."""
    index = first.get_device()
    if index < 0 or not first.is_cuda:
        raise ValueError("expected CUDA tensors on one device")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("expected CUDA tensors on one device")
    return index


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _call(fn, where: str, index: int, *args):
    """One library call on the device's current stream."""
    # (torch.cuda.current_stream(index).cuda_stream without building the Stream)
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        code = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            code = fn(*args, stream)
    if code != SPARGE_OK:
        raise SpargeError(code, where)


def _workspace(fn, where: str, args, device, given):
    """(pointer, bytes, and the tensor that holds them)"""
    nbytes = _SZ(0)
    _check(fn(args, ctypes.byref(nbytes)), where + "_workspace_bytes")
    if given is None:
        if nbytes.value == 0:
            return 0, 0, None
        given = torch.empty(nbytes.value, dtype=torch.uint8, device=device)
    elif given.device != device:
        raise ValueError("expected CUDA tensors on one device")
    return given.data_ptr(), given.numel() * given.element_size(), given


class RopeAxes:
    """Rotary positions over up to three axes (time, height, width): the first
    ``pairs[0]`` channel pairs of a head turn with axis 0, the next with axis 1,
    then axis 2; pairs behind them do not turn.  Pair i of an axis with n pairs
    turns by ``scale * theta ** (-i / n)`` radians per unit of position.  Pairs
    are channels (2j, 2j + 1), or (j, j + d / 2) if not ``interleaved``."""

    def __init__(self, d: int, pairs, theta: float = 10000.0, scale=(1.0, 1.0, 1.0),
                 interleaved: bool = True):
        pairs, scale = tuple(pairs), tuple(scale)
        if not (1 <= len(pairs) <= 3 and len(scale) >= len(pairs)):
            raise ValueError("expected pairs (and a scale) for one to three axes")
        self.d, self.pairs, self.theta = int(d), pairs, float(theta)
        self.scale, self.interleaved = scale[:len(pairs)], bool(interleaved)
        pad = 3 - len(pairs)
        self.plan = Rope()
        _check(load_library().sparge_rope_init(
            ctypes.byref(self.plan), self.d, (ctypes.c_int32 * 3)(*pairs, *[0] * pad),
            self.theta, (ctypes.c_double * 3)(*self.scale, *[1.0] * pad), int(self.interleaved)),
            "sparge_rope_init")

    @property
    def address(self) -> int:
        return ctypes.addressof(self.plan)


def _token_strides(t, B, N, H):
    sb, sn, sh, sc = t.stride()
    if sc != 1:
        raise ValueError("the channels of a head must be contiguous")
    return sb if B > 1 else 0, sn if N > 1 else 0, sh if H > 1 else 0


def _heads_head(B, N, d, x_type, n_parts, rope, grid, pos, norm, weights, eps, index):
    """The leading fields of the packed struct, after their checks."""
    if norm not in _HEADS_NORMS:
        raise ValueError("norm must be None, 'token' or 'head'")
    plan = 0
    if rope is not None:
        if rope.d != d:
            raise ValueError("the rope's head width differs from the tensors'")
        plan = rope.address
    if grid is not None:
        if (grid.dtype != torch.int32 or grid.shape != (B, 3) or not grid.is_contiguous()
                or grid.get_device() != index):
            raise ValueError("grid must be a contiguous int32 [B, 3] tensor on the same device")
    if pos is not None:
        if (pos.dtype != torch.int32 or pos.dim() != 3 or pos.shape[0] not in (1, B)
                or pos.shape[1:] != (N, 3) or not pos.is_contiguous()
                or pos.get_device() != index):
            raise ValueError("pos must be a contiguous int32 [B, N, 3] or [1, N, 3] tensor on the "
                             "same device")
    if (rope is None) != (grid is None and pos is None) or (grid is not None and pos is not None):
        raise ValueError("a rope needs grid or pos, one of the two")
    w_type = None
    for w in weights:
        if w is not None:
            if norm is None or w.get_device() != index or w_type not in (None, w.dtype):
                raise ValueError("norm weights need a norm, and share one type and the device")
            w_type = w.dtype
    if w_type is not None and w_type not in _TYPES:
        raise ValueError("a norm weight must be bf16 or fp32")
    return (B, N, d, x_type, _TYPES.get(w_type, 0), _HEADS_NORMS[norm], eps, n_parts, plan,
            _addr(grid), _addr(pos), 0 if pos is None else pos.shape[0])


def _apart(starts):
    """(The library compares the whole places; this is the plainest mistake.)"""
    if len(set(starts)) != len(starts):
        raise ValueError("the outputs must not overlap")


def _norm_weight(w, norm, H, d):
    if w is None:
        return 0
    if w.shape != ((H * d,) if norm == "token" else (d,)) or not w.is_contiguous():
        raise ValueError("a norm weight is contiguous, [H * d] for 'token' and [d] for 'head'")
    return w.data_ptr()


def sparge_heads_fwd(q=None, k=None, v=None, rope: RopeAxes | None = None, grid=None, pos=None,
                     norm: str | None = None, q_weight=None, k_weight=None, eps: float = 1e-6,
                     out=None):
    """Projections to the attention's layout: each of q, k and v is bf16 or
    fp32 [B, N, H, d] of any batch, token and head stride (multiples of 16
    bytes: slices of a fused projection need no copy) and comes back as bf16
    [B, H, N, d].  Q and K pass
    an RMS norm over the token's H * d channels (``"token"``) or over each head
    (``"head"``), then ``rope``: with ``grid`` (int32 [B, 3]: frames, height,
    width of each sample; tokens behind them do not turn) or ``pos`` (int32
    [B, N, 3]).  Returns (q, k, v), None for what was not given; ``out``, where
    they are written, must not share memory with one another or an input."""
    first = q if q is not None else k if k is not None else v
    if first is None:
        raise ValueError("nothing to lay out")
    index = _cuda_index(first, q, k, v)
    if first.dim() != 4:
        raise ValueError("expected [B, N, H, d] tensors")
    B, N, _, d = first.shape
    dtype, device = first.dtype, first.device
    res, parts, starts, given = [None, None, None], (), [], []
    for i, (t, w) in enumerate(((q, q_weight), (k, k_weight), (v, None))):
        if t is None:
            if w is not None:
                raise ValueError("a norm weight without its tensor")
            continue
        H = t.shape[2] if t.dim() == 4 else 0
        if t.shape != (B, N, H, d) or t.dtype != dtype:
            raise ValueError("q, k and v share their type, batch, length and head width")
        y = out[i] if out is not None else None
        if y is None:
            y = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=device)
        elif (y.shape != (B, H, N, d) or y.dtype != torch.bfloat16 or not y.is_contiguous()
              or y.get_device() != index):
            raise ValueError("out must be contiguous bf16 [B, H, N, d] tensors on the same device")
        else:
            given.append(y)
        at = y.data_ptr()
        parts += (t.data_ptr(), *_token_strides(t, B, N, H), _norm_weight(w, norm, H, d),
                  at, 0, 0, 0, 0, 0, H, i == 2)
        starts.append(at)
        res[i] = y
    if given:
        _apart(starts)
    n = len(parts) // 13
    args = _HEADS.pack(*_heads_head(B, N, d, _type_of(first, "q, k and v"), n, rope, grid, pos,
                                    norm, (q_weight, k_weight), eps, index),
                       *parts, *_NO_PART * (3 - n))
    _call(load_library().sparge_heads_fwd, "sparge_heads_fwd", index, args)
    if given:
        torch.autograd.graph.increment_version(given)
    return tuple(res)


def sparge_heads_bwd(dq=None, dk=None, dv=None, q=None, k=None, rope: RopeAxes | None = None,
                     grid=None, pos=None, norm: str | None = None, q_weight=None, k_weight=None,
                     eps: float = 1e-6, out=None, dtype=None, workspace=None):
    """Gradients of ``sparge_heads_fwd`` from those of its results (bf16
    [B, H, N, d]); q and k are the forward's inputs, needed under a norm.
    Returns (dq, dk, dv, dq_weight, dk_weight): [B, N, H, d] in the inputs'
    type (``dtype`` where neither q nor k is given), written into ``out`` where
    that is given (slices of one buffer, say; no shared memory with one another
    or an input, q and k themselves apart), and the weights' gradients."""
    first = dq if dq is not None else dk if dk is not None else dv
    if first is None:
        raise ValueError("no gradient given")
    index = _cuda_index(first, dq, dk, dv, q, k)
    if first.dim() != 4:
        raise ValueError("expected [B, H, N, d] gradients")
    B, _, N, d = first.shape
    device = first.device
    outs = out if out is not None else (None, None, None)
    typed = [t.dtype for t in (q, k, *outs) if t is not None]
    dtype = typed[0] if typed else (dtype or torch.bfloat16)
    if dtype not in _TYPES or any(t != dtype for t in typed):
        raise ValueError("q, k and out share one type, bf16 or fp32")
    res, parts, starts, given = [None] * 5, (), [], []
    for i, (g, x, w) in enumerate(((dq, q, q_weight), (dk, k, k_weight), (dv, None, None))):
        if g is None:
            if w is not None:
                raise ValueError("a norm weight without its gradient")
            continue
        H = g.shape[1] if g.dim() == 4 else 0
        if g.shape != (B, H, N, d) or g.dtype != torch.bfloat16 or not g.is_contiguous():
            raise ValueError("gradients are contiguous bf16 [B, H, N, d] tensors")
        xp, xs, wp, dw = 0, (0, 0, 0), 0, 0
        if norm is not None and i < 2:
            if x is None or x.shape != (B, N, H, d):
                raise ValueError("a norm's gradient needs its input, [B, N, H, d]")
            xp, xs = x.data_ptr(), _token_strides(x, B, N, H)
            if w is not None:
                wp = _norm_weight(w, norm, H, d)
                res[3 + i] = torch.empty_like(w)
                dw = res[3 + i].data_ptr()
        dx = outs[i]
        if dx is None:
            dx = torch.empty((B, N, H, d), dtype=dtype, device=device)
        elif dx.shape != (B, N, H, d) or dx.get_device() != index:
            raise ValueError("out must be [B, N, H, d] tensors on the same device")
        elif 0 in dx.stride() and any(st == 0 and n_ > 1
                                      for st, n_ in zip(dx.stride(), dx.shape)):
            raise ValueError("out must not repeat elements")
        else:
            given.append(dx)
        at = dx.data_ptr()
        parts += (xp, *xs, wp, g.data_ptr(), at, *_token_strides(dx, B, N, H), dw, H, i == 2)
        starts.append(at)
        res[i] = dx
    if given:
        _apart(starts)
    n = len(parts) // 13
    args = _HEADS.pack(*_heads_head(B, N, d, _TYPES[dtype], n, rope, grid, pos, norm,
                                    (q_weight, k_weight), eps, index),
                       *parts, *_NO_PART * (3 - n))
    lib = load_library()
    ws, size, _hold = _workspace(lib.sparge_heads_bwd_workspace_bytes, "sparge_heads_bwd", args,
                                 device, workspace)
    _call(lib.sparge_heads_bwd, "sparge_heads_bwd", index, args, ws, size)
    if given:
        torch.autograd.graph.increment_version(given)
    return tuple(res)


def _modulation(m, what, B, N, C):
    """(pointer, groups, stride) of a gate, scale or shift: [C] for all tokens,
    or [B, F, C] with a row for each run of N / F tokens of a sample."""
    if m is None:
        return 0, 1, 0
    if m.dtype != torch.float32 or m.stride(-1) != 1:
        raise ValueError(f"{what} must be fp32 with contiguous channels")
    if m.shape == (C,):
        return m.data_ptr(), 1, 0
    if m.dim() != 3 or m.shape[2] != C or m.shape[0] not in (1, B):
        raise ValueError(f"{what} must be [C] or [B, F, C]")
    b, f = m.shape[:2]
    if b * f == 1:
        return m.data_ptr(), 1, 0
    if b != B or f < 1 or N % f:
        raise ValueError(f"{what} [B, F, C]: F must divide the tokens of a sample")
    if f == 1:
        return m.data_ptr(), b, m.stride(0)
    if b > 1 and m.stride(0) != f * m.stride(1):
        raise ValueError(f"the rows of {what} must be evenly spaced")
    return m.data_ptr(), b * f, m.stride(1)


def _resnorm_head(x, branch, gate, scale, shift, norm, unit_offset, post_weight, eps, h_type):
    """The leading fields of the packed struct, after their checks."""
    if norm not in _NORMS:
        raise ValueError("norm must be None, 'layer' or 'rms'")
    if x.dim() not in (2, 3) or not x.is_contiguous():
        raise ValueError("x must be a contiguous [B, N, C] or [N, C] tensor")
    shape = x.shape
    C = shape[-1]
    B, N = (1, shape[0]) if len(shape) == 2 else shape[:2]
    if branch is not None and (branch.shape != shape or not branch.is_contiguous()):
        raise ValueError("branch must be contiguous, of x's shape")
    if post_weight is not None and (post_weight.shape != (C,) or not post_weight.is_contiguous()
                                    or post_weight.dtype != torch.float32):
        raise ValueError("post_weight must be contiguous fp32 [C]")
    gp, gg, gs = _modulation(gate, "gate", B, N, C)
    cp, cg, cs = _modulation(scale, "scale", B, N, C)
    sp, sg, ss = _modulation(shift, "shift", B, N, C)
    return (B * N, C, _type_of(x, "x"), h_type, _NORMS[norm], unit_offset, eps, x.data_ptr(),
            _addr(branch), gp, cp, sp, gg, cg, sg, gs, cs, ss, _addr(post_weight))


def sparge_resnorm_fwd(x, branch=None, gate=None, scale=None, shift=None,
                       norm: str | None = "layer", unit_offset: bool = True, post_weight=None,
                       eps: float = 1e-6, h_dtype=None, want_stats: bool = True):
    """Residual join and norm: y = x + gate * branch, h = norm(y) * (1 + scale)
    + shift (``scale`` itself without ``unit_offset``); with ``post_weight`` the
    branch passes an RMS norm first.  x and branch are contiguous [B, N, C]
    (bf16 x: bf16 branch); gate, scale and shift fp32, [C] for all tokens or
    [B, F, C] with a row for each run of N / F tokens.  Returns (y, h, stats):
    y is x where there is no branch, h (of the branch's type, or ``h_dtype``)
    is None without a norm, stats (fp32 [3, tokens]) is what the backward
    needs."""
    index = _cuda_index(x, branch, gate, scale, shift, post_weight)
    if branch is not None:
        h_type = _type_of(branch, "branch")
        if h_dtype is not None and h_dtype != branch.dtype:
            raise ValueError("h has the branch's type")
        h_dtype = branch.dtype
    else:
        h_dtype = h_dtype or x.dtype
        if h_dtype not in _TYPES:
            raise ValueError("h must be bf16 or fp32")
        h_type = _TYPES[h_dtype]
    head = _resnorm_head(x, branch, gate, scale, shift, norm, bool(unit_offset), post_weight, eps,
                         h_type)
    y, h, stats = x, None, None
    if branch is not None:
        y = torch.empty_like(x)
    if norm is not None:
        h = torch.empty_like(x, dtype=h_dtype)
    if want_stats and (norm is not None or post_weight is not None):
        stats = torch.empty((3, head[0]), dtype=torch.float32, device=x.device)
    args = _RESNORM.pack(*head, y.data_ptr(), _addr(h), _addr(stats), 0, 0, 0, 0, 0, 0, 0, 0)
    _call(load_library().sparge_resnorm_fwd, "sparge_resnorm_fwd", index, args)
    return y, h, stats


def sparge_resnorm_bwd(dy, dh, x, branch=None, gate=None, scale=None, shift=None, stats=None,
                       norm: str | None = "layer", unit_offset: bool = True, post_weight=None,
                       want_mods: bool = True, workspace=None):
    """Gradients of ``sparge_resnorm_fwd``: returns (dx, dbranch, dgate, dscale,
    dshift, dpost), None for what was not given.  ``dy`` or ``dh`` may be None
    (zero).  ``want_mods=False`` leaves the four sums out."""
    index = _cuda_index(x, branch, gate, scale, shift, post_weight, dy, dh, stats)
    like = branch if branch is not None else dh if dh is not None else x
    head = _resnorm_head(x, branch, gate, scale, shift, norm, bool(unit_offset), post_weight, 0.0,
                         _type_of(like, "branch and dh"))
    for t, ref, what in ((dy, x, "dy"), (dh, like, "dh")):
        if t is not None and (t.shape != x.shape or t.dtype != ref.dtype
                              or not t.is_contiguous()):
            raise ValueError(f"{what} must be contiguous, of x's shape and its own result's type")
    if stats is not None and (stats.dtype != torch.float32 or stats.numel() != 3 * head[0]
                              or not stats.is_contiguous()):
        raise ValueError("stats must be the forward's fp32 [3, tokens]")
    device = x.device
    dx = torch.empty_like(x)
    dbranch = torch.empty_like(branch) if branch is not None else None
    sums = [torch.empty(m.shape, dtype=torch.float32, device=device)
            if want_mods and m is not None else None for m in (gate, scale, shift, post_weight)]
    args = _RESNORM.pack(*head, 0, 0, _addr(stats), _addr(dy), _addr(dh), dx.data_ptr(),
                         _addr(dbranch), *(_addr(t) for t in sums))
    lib = load_library()
    ws, size, _hold = _workspace(lib.sparge_resnorm_bwd_workspace_bytes, "sparge_resnorm_bwd",
                                 args, device, workspace)
    _call(lib.sparge_resnorm_bwd, "sparge_resnorm_bwd", index, args, ws, size)
    return (dx, dbranch, *sums)


def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill its memory without gaps or repeats."""
    step = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size != 1:
            if stride != step:
                return False
            step *= size
    return True


def _tensor_lists(grads, outs, index):
    """The C list of the gradients and the pointers of the outputs (None: in
    place).  One plain loop: with hundreds of tensors it is most of the call."""
    rows, ptrs = [], []
    code = _TYPES.get
    for t, o in zip(grads, grads if outs is None else outs):
        dtype, n = t.dtype, t.numel()
        kind = code(dtype)
        if kind is None or t.get_device() != index:
            raise ValueError("gradients must be bf16 or fp32 CUDA tensors on one device")
        if o is not t and (o.dtype is not dtype or o.numel() != n or o.get_device() != index):
            raise ValueError("out must match the gradients in type, size and device")
        if not (t.is_contiguous() and o.is_contiguous()) and n > 0:
            if not _dense(t):
                raise ValueError("gradients must have no gaps or repeated elements")
            if o.shape != t.shape or o.stride() != t.stride():
                raise ValueError("out must match the gradients in shape and strides")
        rows += (t.data_ptr(), n, kind)
        if outs is not None:
            ptrs.append(o.data_ptr())
    # sparge_tensor: pointer, int64, int32 and padding
    return array.array("q", rows), array.array("q", ptrs) if outs is not None else None


@functools.lru_cache(maxsize=64)
def _clip_workspace_bytes(n: int) -> int:
    nbytes = _SZ(0)
    _check(load_library().sparge_clip_workspace_bytes(n, ctypes.byref(nbytes)),
           "sparge_clip_workspace_bytes")
    return nbytes.value


def sparge_clip_grads(grads, max_norm: float | None, out=None, eps: float = 1e-6, workspace=None):
    """Global 2-norm of a list of gradients (fp32 scalar tensor, returned
    without waiting for the GPU), and g * min(1, max_norm / (norm + eps)) in
    place or into ``out``.  ``max_norm=None``: the norm alone.  Tensors may mix
    bf16 and fp32; a tensor must not be listed twice or overlap another."""
    grads = list(grads)
    if not grads:
        raise ValueError("expected at least one gradient")
    if max_norm is not None and not (math.isfinite(max_norm) and max_norm >= 0):
        raise ValueError("max_norm must be finite and not negative")
    index = _cuda_index(grads[0])
    device, n = grads[0].device, len(grads)
    if out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError("expected one output for each gradient")
    table, outs = _tensor_lists(grads, out, index)
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(_clip_workspace_bytes(n), dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError("expected CUDA tensors on one device")
    norm = torch.empty((), dtype=torch.float32, device=device)
    _call(lib.sparge_clip_grads, "sparge_clip_grads", index, table.buffer_info()[0],
          outs.buffer_info()[0] if outs is not None else None, n,
          -1.0 if max_norm is None else float(max_norm), eps, norm.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if max_norm is not None:
        torch.autograd.graph.increment_version(grads if out is None else out)
    return norm


# ------------------------------------------------ attention over a context
_NO_TENSOR = (0, 0, 0, 0)


def _heads_tensor(t, what, shape, index):
    """(pointer, batch stride, head stride, token stride) of a bf16 tensor
    [batch, heads, tokens, d] in any order of the first three."""
    if t.dtype is not torch.bfloat16 or t.get_device() != index or t.shape != shape:
        raise ValueError(f"{what} must be a bf16 {list(shape)} tensor on the same device")
    sb, sh, sn, sc = t.stride()
    if sc != 1:
        raise ValueError(f"the channels of {what} must be contiguous")
    return t.data_ptr(), sb, sh, sn


def _cross_head(q, k, v, kv_len, softmax_scale, index):
    """The leading fields of the packed struct, after their checks."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected [batch, heads, tokens, d] tensors")
    B, H, N, d = q.shape
    Bk, Hk, M, _ = k.shape
    if kv_len is not None and (kv_len.dtype is not torch.int32 or kv_len.shape != (B,)
                               or kv_len.get_device() != index or not kv_len.is_contiguous()):
        raise ValueError("kv_len must be a contiguous int32 [B] tensor on the same device")
    keys = torch.Size((Bk, Hk, M, d))
    return (B, Bk, H, Hk, N, M, d, softmax_scale, _addr(kv_len),
            *_heads_tensor(q, "q", q.shape, index), *_heads_tensor(k, "k", keys, index),
            *_heads_tensor(v, "v", keys, index))


def _cross_lse(lse, q, index):
    if (lse.dtype is not torch.float32 or lse.shape != q.shape[:3] or lse.get_device() != index
            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor on the same device")
    return lse.data_ptr()


def _cross_status(status, check_status, device):
    if status is None and check_status:
        status = torch.zeros(1, dtype=torch.int32, device=device)
    return status


def sparge_cross_fwd(q, k, v, kv_len=None, softmax_scale: float = 0.0, check_status=False,
                     out=None, lse=None, status=None, workspace=None):
    """Attention over a context: softmax(scale q k^T) v with bf16 q [B, H, N, d],
    k and v [Bk, Hk, M, d]; Hk divides H (query head h reads key head
    h // (H // Hk)), Bk is B, or 1 for one context of all samples.  The first
    three dimensions may lie in any order (strides of multiples of 16 bytes): a
    transposed view of projections [B, N, H, d] needs no copy.  ``kv_len`` (int32
    [B]): the valid context tokens of each sample, all without it; what lies
    behind them is not used, and a sample of length 0 gets O = 0, LSE = -inf.
    Returns (O, of q's shape and, unless ``out`` is given, dense; LSE fp32
    [B, H, N])."""
    index = _cuda_index(q, k, v)
    device = q.device
    head = _cross_head(q, k, v, kv_len, softmax_scale, index)
    o = out if out is not None else torch.empty(q.shape, dtype=torch.bfloat16, device=device)
    given = [t for t in (out, lse) if t is not None]
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=device)
    status = _cross_status(status, check_status, device)
    args = _CROSS.pack(*head, *_heads_tensor(o, "out", q.shape, index),
                       _cross_lse(lse, q, index), *_NO_TENSOR * 4, _addr(status))
    lib = load_library()
    ws, size, _hold = _workspace(lib.sparge_cross_fwd_workspace_bytes, "sparge_cross_fwd", args,
                                 device, workspace)
    _call(lib.sparge_cross_fwd, "sparge_cross_fwd", index, args, ws, size)
    if given:
        torch.autograd.graph.increment_version(given)
    if check_status:
        _finish(status, True, "sparge_cross_fwd")
    return o, lse


def sparge_cross_bwd(q, k, v, o, lse, dout, kv_len=None, softmax_scale: float = 0.0,
                     check_status=False, workspace=None, out=None, status=None):
    """Gradients (dQ, dK, dV) of ``sparge_cross_fwd``: o and lse as it returned
    them, dout of o's shape.  dK and dV are summed over the heads of a group and,
    with one context, over the samples; they are 0 behind the samples' lengths.
    With more than 64 context tokens they are less exact where the values' mean is
    large beside their spread (``include/sparge.h`` has the figures).
    ``out``: three tensors to write them into, of any order of the first three
    dimensions (slices of one buffer, say)."""
    index = _cuda_index(q, k, v, o, lse, dout)
    device = q.device
    head = _cross_head(q, k, v, kv_len, softmax_scale, index)
    if out is None:
        outs = [torch.empty(t.shape, dtype=torch.bfloat16, device=device) for t in (q, k, v)]
    else:
        outs = list(out)
        if len(outs) != 3:
            raise ValueError("out must be three tensors")
    status = _cross_status(status, check_status, device)
    args = _CROSS.pack(*head, *_heads_tensor(o, "o", q.shape, index), _cross_lse(lse, q, index),
                       *_heads_tensor(dout, "dout", q.shape, index),
                       *(x for t, like, what in zip(outs, (q, k, v), ("dq", "dk", "dv"))
                         for x in _heads_tensor(t, what, like.shape, index)), _addr(status))
    lib = load_library()
    ws, size, _hold = _workspace(lib.sparge_cross_bwd_workspace_bytes, "sparge_cross_bwd", args,
                                 device, workspace)
    _call(lib.sparge_cross_bwd, "sparge_cross_bwd", index, args, ws, size)
    if out is not None:
        torch.autograd.graph.increment_version(outs)
    if check_status:
        _finish(status, True, "sparge_cross_bwd")
    return tuple(outs)


# ------------------------------------------------ orthogonalised updates
_NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def _matrix(t, what, shape, flipped, index):
    """(pointer, elements between rows) of a matrix, or with ``flipped`` of its
    transposed form."""
    if t.shape != shape or t.get_device() != index or t.dtype not in _TYPES:
        raise ValueError(f"{what} must be bf16 or fp32 matrices of their gradient's shape and device")
    (sr, sc), (r, c) = t.stride(), shape
    if flipped:
        sr, sc, r, c = sc, sr, c, r
    if sc != 1 and c > 1:
        raise ValueError(f"{what}: the values of a matrix's rows (or, for all of its tensors, of "
                         "its columns) must be contiguous")
    return t.data_ptr(), sr if r > 1 else c


def _is_flipped(t) -> bool:
    """Whether t's columns lie contiguous and its rows do not."""
    return t.stride(1) != 1 and t.shape[1] > 1 and (t.stride(0) == 1 or t.shape[0] == 1)


def _orthogonalize(grads, outs, momenta, factors, steps, coefficients, eps, mu, nesterov, half,
                   workspace, status, check_status, where):
    index = _cuda_index(grads[0])
    device = grads[0].device
    a, b, c = coefficients
    rows = {False: [], True: []}
    for i, (g, o) in enumerate(zip(grads, outs)):
        if g.dim() != 2:
            raise ValueError("expected matrices")
        shape, flipped = g.shape, _is_flipped(g)
        n, m = reversed(shape) if flipped else shape
        mom = momenta[i] if momenta is not None else None
        if mom is not None and mom.dtype is not torch.float32:
            raise ValueError("momenta must be fp32")
        keep, step = factors[i] if factors is not None else (0.0, 0.0)
        packed = _MATRIX.pack(
            n, m, _TYPES.get(g.dtype, -1), _TYPES.get(o.dtype, -1),
            *_matrix(g, "gradients", shape, flipped, index),
            *(_matrix(mom, "momenta", shape, flipped, index) if mom is not None else (0, 0)),
            *_matrix(o, "results", shape, flipped, index), keep, step)
        rows[o.dtype is torch.bfloat16 if half is None else bool(half)].append(packed)
    lib = load_library()
    status = _cross_status(status, check_status, device)

    def pack(part, fast):
        table = ctypes.create_string_buffer(b"".join(part))
        return table, _ORTHO.pack(ctypes.addressof(table), len(part), steps, a, b, c, eps, mu,
                                  bool(nesterov), factors is not None, fast, _addr(status))

    calls = [pack(part, fast) for fast, part in rows.items() if part]
    if len(calls) > 1:
        # One list to its caller: refused, if at all, before the first of two calls. (With
        # a workspace too small for either, that is the one that needs more.)
        _table, args = pack(rows[False] + rows[True], False)
        _check(lib.sparge_orthogonalize_check(args), where)
        need = _SZ(0)

        def bytes_of(call):
            _check(lib.sparge_orthogonalize_workspace_bytes(call[1], ctypes.byref(need)), where)
            return need.value

        calls.sort(key=bytes_of, reverse=True)
    ws, size, _hold = _workspace(lib.sparge_orthogonalize_workspace_bytes, "sparge_orthogonalize",
                                 calls[0][1], device, workspace)
    for _table, args in calls:
        _call(lib.sparge_orthogonalize, where, index, args, ws, size)
    if check_status:
        _finish(status, True, where)


def sparge_orthogonalize(mats, out=None, steps: int = 5, coefficients=_NEWTON_SCHULZ,
                         eps: float = 1e-7, half: bool | None = None, workspace=None,
                         status=None, check_status=False):
    """Matrices to nearly orthogonal ones of the same singular vectors: X = G / (|G|
    + eps), then ``steps`` times X <- a X + (b A + c A A) X with A = X X^T (the
    transposed form for tall ones).  ``mats``: a list of bf16 or fp32 matrices of any
    sizes up to 65536, of any row stride (or, transposed, column stride); results of
    the same types, or written to ``out`` (a matrix may be its own).  ``half``: the
    products take fp16 values (results off by some 2^-9 of their size) or pairs of
    them (some 2^-20, three times the work); None: as the results are bf16 or
    fp32.  Both are further off where a few directions are strong and the others
    10^3 and more below them, up to 2^-4 for fp16 values and a short side up to 16:
    ``include/sparge.h`` has the figures."""
    mats = list(mats)
    if not mats:
        raise ValueError("expected at least one matrix")
    if out is None:
        outs = [torch.empty(m.shape[::-1], dtype=m.dtype, device=m.device).t()
                if m.dim() == 2 and _is_flipped(m) else
                torch.empty(m.shape, dtype=m.dtype, device=m.device) for m in mats]
    else:
        outs = list(out)
        if len(outs) != len(mats):
            raise ValueError("expected one result for each matrix")
    _orthogonalize(mats, outs, None, None, steps, coefficients, eps, 0.0, False, half, workspace,
                   status, check_status, "sparge_orthogonalize")
    if out is not None:
        torch.autograd.graph.increment_version(outs)
    return outs


def sparge_muon_step(weights, grads, momenta, lr: float, momentum: float = 0.95,
                     nesterov: bool = True, weight_decay: float = 0.0, rms: float | None = None,
                     steps: int = 5, coefficients=_NEWTON_SCHULZ, eps: float = 1e-7,
                     half: bool | None = None, workspace=None, status=None, check_status=False,
                     inputs_first: bool = False):
    """One optimiser step on matrices, in place: m <- momentum * m + g; U = g +
    momentum * m (``nesterov``) or m; w <- (1 - lr * weight_decay) * w - lr * gain *
    O, O the orthogonalised U (``sparge_orthogonalize``).  gain is sqrt(max(1, outputs /
    inputs)) of weights [outputs, inputs], or with ``inputs_first`` [inputs, outputs] (those
    of ``x @ w``), or with ``rms`` what gives the update about that root mean square:
    rms * sqrt(max(rows, columns)).  Weights and gradients are bf16 or fp32, momenta
    fp32 (``momenta`` None: U = g).  ``half`` None: as the weights are bf16 or fp32."""
    weights, grads = list(weights), list(grads)
    momenta = list(momenta) if momenta is not None else None
    if not weights:
        raise ValueError("expected at least one matrix")
    if len(grads) != len(weights) or (momenta is not None and len(momenta) != len(weights)):
        raise ValueError("expected one gradient and one momentum for each weight")
    factors = []
    for w in weights:
        if w.dim() != 2 or 0 in w.shape:
            raise ValueError("expected matrices")
        r, c = w.shape
        if inputs_first:
            r, c = c, r
        gain = math.sqrt(max(1.0, r / c)) if rms is None else rms * math.sqrt(max(r, c))
        factors.append((1.0 - lr * weight_decay, lr * gain))
    _orthogonalize(grads, weights, momenta, factors, steps, coefficients, eps, momentum, nesterov,
                   half, workspace, status, check_status, "sparge_muon_step")
    torch.autograd.graph.increment_version(weights if momenta is None else weights + momenta)


def sparge_debug_wait_probe(timeout_ns: int = 10_000_000, device="cuda") -> int:
    """Runs the bounded-wait probe kernel; returns the device status it wrote."""
    lib = load_library()
    st = torch.zeros(1, dtype=torch.int32, device=device)
    _check(lib.sparge_debug_wait_probe(_ptr(st), int(timeout_ns), _stream(st.device)),
           "sparge_debug_wait_probe")
    return _read_status(st)
