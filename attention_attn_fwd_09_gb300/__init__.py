"""Python binding for libattn.so: fused exact attention on GB300 (sm_103a).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  If the compiled
library is missing this module raises at import time; there is no fallback.

Names match the C ABI in include/attn.h: ``attn_fwd``, ``attn_fwd_kv``,
``attn_fwd_varlen`` and ``attn_bwd_varlen`` (packed sequences of different lengths), ``attn_bwd``,
``attn_bwd_noalloc``, ``attn_quantize_fp8`` and ``attn_fwd_fp8`` (e4m3 inputs with
per-block scales), ``attn_rope`` and ``attn_rope_bwd`` (rotary positions),
``attn_kv_append_fp8`` and ``attn_fwd_kv_fp8`` (a paged e4m3 key/value cache and the attention
over it), the ``*_workspace_size`` queries, ``attn_last_error`` and the
test/tuning knobs.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (or python -m "
                      "attention_attn_fwd_09_gb300._build) first")

_lib = ctypes.CDLL(LIB_PATH)
_p, _i, _f, _ll, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t
_lib.attn_fwd.argtypes = [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p]
_lib.attn_fwd.restype = _i
_lib.attn_fwd_kv.argtypes = [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p]
_lib.attn_fwd_kv.restype = _i
_lib.attn_fwd_kv_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.attn_fwd_kv_workspace_size.restype = _sz
_lib.attn_fwd_varlen.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p]
_lib.attn_fwd_varlen.restype = _i
_lib.attn_fwd_varlen_workspace_size.argtypes = [_i, _i, _i, _i, _i]
_lib.attn_fwd_varlen_workspace_size.restype = _sz
_lib.attn_bwd_varlen.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p,
                                 _sz, _p]
_lib.attn_bwd_varlen.restype = _i
_lib.attn_bwd_varlen_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
_lib.attn_bwd_varlen_workspace_size.restype = _sz
_lib.attn_set_fwd_persistent.argtypes = [_i]
_lib.attn_set_fwd_persistent.restype = _i
_lib.attn_set_fwd_one_tile.argtypes = [_i]
_lib.attn_set_fwd_one_tile.restype = _i
_lib.attn_set_decode_one_tile.argtypes = [_i]
_lib.attn_set_decode_one_tile.restype = _i
_lib.attn_set_bwd_query_tile.argtypes = [_i]
_lib.attn_set_bwd_query_tile.restype = _i
_lib.attn_set_varlen_order.argtypes = [_i]
_lib.attn_set_varlen_order.restype = _i
_lib.attn_bwd.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p]
_lib.attn_bwd.restype = _i
_lib.attn_bwd_noalloc.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _i, _p]
_lib.attn_bwd_noalloc.restype = _i
_lib.attn_bwd_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.attn_bwd_workspace_size.restype = _sz
_lib.attn_last_error.argtypes = []
_lib.attn_last_error.restype = ctypes.c_char_p
_lib.attn_version.argtypes = []
_lib.attn_version.restype = ctypes.c_char_p
_lib.attn_set_debug_knobs.argtypes = [_f, _i, _ll, _i]
_lib.attn_set_debug_knobs.restype = _i
_lib.attn_get_debug_knobs.argtypes = [ctypes.POINTER(_f), ctypes.POINTER(_i), ctypes.POINTER(_ll), ctypes.POINTER(_i)]
_lib.attn_get_debug_knobs.restype = _i
_lib.attn_device_status.argtypes = [_i]
_lib.attn_device_status.restype = _i
_lib.attn_rescale_counter.argtypes = [_i, ctypes.POINTER(ctypes.c_ulonglong)]
_lib.attn_rescale_counter.restype = _i
_lib.attn_set_test_hooks.argtypes = [_i]
_lib.attn_set_test_hooks.restype = _i
_lib.attn_quantize_fp8.argtypes = [_p, _p, _p, _i, _i, _i, _i, _p]
_lib.attn_quantize_fp8.restype = _i
_lib.attn_fwd_fp8.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p]
_lib.attn_fwd_fp8.restype = _i
_lib.attn_rope.argtypes = [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, ctypes.POINTER(_ll), _p]
_lib.attn_rope.restype = _i
_lib.attn_rope_bwd.argtypes = _lib.attn_rope.argtypes
_lib.attn_rope_bwd.restype = _i
_lib.attn_kv_append_fp8.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                    ctypes.POINTER(_ll), _p]
_lib.attn_kv_append_fp8.restype = _i
_lib.attn_fwd_kv_fp8.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _p,
                                 _sz, _p]
_lib.attn_fwd_kv_fp8.restype = _i
_lib.attn_fwd_kv_fp8_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.attn_fwd_kv_fp8_workspace_size.restype = _sz
_lib.attn_exp2_sw.argtypes = [_p, _p, _ll, _i, _p]
_lib.attn_exp2_sw.restype = _i

STATUS = {0: "ATTN_OK", -1: "ATTN_ERR_INVALID_ARG", -2: "ATTN_ERR_UNSUPPORTED", -3: "ATTN_ERR_MISALIGNED",
          -4: "ATTN_ERR_WORKSPACE", -5: "ATTN_ERR_CUDA", -6: "ATTN_ERR_TIMEOUT"}


class AttnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


def attn_last_error() -> str:
    return (_lib.attn_last_error() or b"").decode()


def attn_version() -> str:
    return _lib.attn_version().decode()


def _check(rc: int):
    if rc != 0:
        raise AttnError(rc, attn_last_error())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dev_bf16(name, t, shape):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected a contiguous CUDA bf16 tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")


def _dev_f32(name, t, shape):
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected a contiguous CUDA fp32 tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")


def _bwd_tensors(q, k, v, o, lse, do, dq, dk, dv):
    """Checks the backward's inputs and outputs ([B,Hq,N,d] / [B,Hkv,N,d] bf16, lse [B,Hq,N]
    fp32, all on one device) and allocates the outputs not given."""
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    for name, t, shp in (("q", q, (B, Hq, N, d)), ("k", k, (B, Hkv, N, d)), ("v", v, (B, Hkv, N, d)),
                         ("o", o, (B, Hq, N, d)), ("do", do, (B, Hq, N, d))):
        _dev_bf16(name, t, shp)
    _dev_f32("lse", lse, (B, Hq, N))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _dev_bf16("dq", dq, (B, Hq, N, d))
    _dev_bf16("dk", dk, (B, Hkv, N, d))
    _dev_bf16("dv", dv, (B, Hkv, N, d))
    for name, t in (("k", k), ("v", v), ("o", o), ("lse", lse), ("do", do), ("dq", dq), ("dk", dk), ("dv", dv)):
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    return B, Hq, Hkv, N, d, dq, dk, dv


def attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, o=None, lse=None, stream=None):
    """O, LSE = attention(q, k, v).  q [B,Hq,N,d], k/v [B,Hkv,N,d] CUDA bf16.

    ``o`` ([B,Hq,N,d] bf16) and ``lse`` ([B,Hq,N] fp32) may be given to reuse buffers."""
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    _dev_bf16("q", q, (B, Hq, N, d))
    _dev_bf16("k", k, (B, Hkv, N, d))
    _dev_bf16("v", v, (B, Hkv, N, d))
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    _dev_bf16("o", o, (B, Hq, N, d))
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, Hq, N):
        raise ValueError("lse: expected a contiguous fp32 tensor [B,Hq,N]")
    _check(_lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d, int(bool(causal)),
                         float(scale), _stream(stream)))
    return o, lse


def attn_fwd_kv_workspace_size(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    n = _lib.attn_fwd_kv_workspace_size(B, Hq, Hkv, Nq, Nk, d)
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(-1, attn_last_error())
    return int(n)


def attn_fwd_kv(q, k, v, causal: bool = False, scale: float | None = None, o=None, lse=None, workspace=None,
                stream=None):
    """O, LSE for Nq queries after a cache of Nk >= Nq keys.  q [B,Hq,Nq,d], k/v [B,Hkv,Nk,d]
    CUDA bf16; query i stands at key position i + Nk - Nq (causal: sees keys up to there).
    ``workspace``: a uint8 CUDA tensor of at least attn_fwd_kv_workspace_size(...) bytes
    (allocated here when None and needed; pass an empty tensor to use the ordinary tiling)."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    _dev_bf16("q", q, (B, Hq, Nq, d))
    _dev_bf16("k", k, (B, Hkv, Nk, d))
    _dev_bf16("v", v, (B, Hkv, Nk, d))
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    _dev_bf16("o", o, (B, Hq, Nq, d))
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse: expected a contiguous fp32 tensor [B,Hq,Nq]")
    if workspace is None:
        n = attn_fwd_kv_workspace_size(B, Hq, Hkv, Nq, Nk, d)
        workspace = torch.empty((n,), dtype=torch.uint8, device=q.device)
    ws_ptr = _ptr(workspace) if workspace.numel() > 0 else ctypes.c_void_p(0)
    _check(_lib.attn_fwd_kv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                            int(bool(causal)), float(scale), ws_ptr, workspace.numel() * workspace.element_size(),
                            _stream(stream)))
    return o, lse


def attn_fwd_varlen_workspace_size(B: int, Hq: int, Hkv: int, total_q: int, d: int) -> int:
    n = _lib.attn_fwd_varlen_workspace_size(B, Hq, Hkv, total_q, d)
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(-1, attn_last_error())
    return int(n)


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, causal: bool = False, scale: float | None = None,
                    o=None, lse=None, workspace=None, stream=None):
    """O, LSE for packed sequences of different lengths.  q [Hq, total_q, d], k/v [Hkv,
    total_k, d] CUDA bf16; ``cu_seqlens_q``/``cu_seqlens_k``: CUDA int32 offsets (B + 1
    each) of the sequences along the row axis.  Within a sequence, query i stands at key
    position i + nk - nq (causal: sees keys up to there).  ``workspace``: a uint8 CUDA
    tensor of at least attn_fwd_varlen_workspace_size(...) bytes (allocated when None).
    The offsets are checked on the device; a failed check shows in attn_device_status()."""
    Hq, Tq, d = q.shape
    Hkv, Tk = k.shape[0], k.shape[1]
    _dev_bf16("q", q, (Hq, Tq, d))
    _dev_bf16("k", k, (Hkv, Tk, d))
    _dev_bf16("v", v, (Hkv, Tk, d))
    for name, c in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if c.dtype != torch.int32 or not c.is_cuda or not c.is_contiguous() or c.dim() != 1:
            raise ValueError(f"{name}: expected a contiguous 1-D CUDA int32 tensor")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k need B + 1 entries each")
    B = cu_seqlens_q.numel() - 1
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    _dev_bf16("o", o, (Hq, Tq, d))
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (Hq, Tq):
        raise ValueError("lse: expected a contiguous fp32 tensor [Hq, total_q]")
    if workspace is None:
        n = attn_fwd_varlen_workspace_size(B, Hq, Hkv, Tq, d)
        workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=q.device)
    _check(_lib.attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q),
                                _ptr(cu_seqlens_k), B, Hq, Hkv, Tq, Tk, d, int(bool(causal)), float(scale),
                                _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def attn_bwd_varlen_workspace_size(B: int, Hq: int, Hkv: int, total_q: int, total_k: int, d: int,
                                   deterministic: bool = False) -> int:
    n = _lib.attn_bwd_varlen_workspace_size(B, Hq, Hkv, total_q, total_k, d, int(bool(deterministic)))
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(-1, attn_last_error())
    return int(n)


def attn_bwd_varlen(q, k, v, o, lse, do, cu_seqlens_q, cu_seqlens_k, causal: bool = False,
                    scale: float | None = None, deterministic: bool = False, dq=None, dk=None, dv=None,
                    workspace=None, stream=None):
    """dQ, dK, dV over packed sequences (layouts and offsets as ``attn_fwd_varlen``; ``o``
    and ``lse`` as it returned them, ``do`` like ``q``)."""
    Hq, Tq, d = q.shape
    Hkv, Tk = k.shape[0], k.shape[1]
    for name, t, shp in (("q", q, (Hq, Tq, d)), ("o", o, (Hq, Tq, d)), ("do", do, (Hq, Tq, d)),
                         ("k", k, (Hkv, Tk, d)), ("v", v, (Hkv, Tk, d))):
        _dev_bf16(name, t, shp)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (Hq, Tq):
        raise ValueError("lse: expected a contiguous fp32 tensor [Hq, total_q]")
    for name, c in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if c.dtype != torch.int32 or not c.is_cuda or not c.is_contiguous() or c.dim() != 1:
            raise ValueError(f"{name}: expected a contiguous 1-D CUDA int32 tensor")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k need B + 1 entries each")
    B = cu_seqlens_q.numel() - 1
    if scale is None:
        scale = d ** -0.5
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _dev_bf16("dq", dq, (Hq, Tq, d))
    _dev_bf16("dk", dk, (Hkv, Tk, d))
    _dev_bf16("dv", dv, (Hkv, Tk, d))
    if workspace is None:
        n = attn_bwd_varlen_workspace_size(B, Hq, Hkv, Tq, Tk, d, deterministic)
        workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=q.device)
    _check(_lib.attn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                                _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, Hq, Hkv, Tq, Tk, d,
                                int(bool(causal)), float(scale), int(bool(deterministic)), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)))
    return dq, dk, dv


def attn_set_fwd_persistent(enable: bool):
    """d = 64/128 forward: one CTA per SM walking the work list (True) or one per unit."""
    _check(_lib.attn_set_fwd_persistent(int(bool(enable))))


def attn_set_fwd_one_tile(enable: bool):
    """d = 128 forward kernel: one query tile per CTA (True) or two (False)."""
    _check(_lib.attn_set_fwd_one_tile(int(bool(enable))))


def attn_set_decode_one_tile(enable: bool):
    """attn_fwd_kv grouped decode at d = 128: the one-tile kernel (True, default) or the
    two-tile kernel (False)."""
    _check(_lib.attn_set_decode_one_tile(int(bool(enable))))


def attn_set_bwd_query_tile(rows: int):
    """d = 64/128 backward: 128-row query tiles (dQ^T in dP^T's columns) or 64-row tiles
    (dQ^T in columns of its own, next tile's products issued ahead)."""
    _check(_lib.attn_set_bwd_query_tile(int(rows)))


def attn_set_varlen_order(longest_first: bool = True):
    _check(_lib.attn_set_varlen_order(int(bool(longest_first))))


def attn_bwd_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int, deterministic: bool = False) -> int:
    n = _lib.attn_bwd_workspace_size(B, Hq, Hkv, N, d, int(bool(deterministic)))
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(-1, attn_last_error())
    return int(n)


def attn_bwd(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None, deterministic: bool = False,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of attention given the forward's o, lse and the upstream gradient do."""
    B, Hq, Hkv, N, d, dq, dk, dv = _bwd_tensors(q, k, v, o, lse, do, dq, dk, dv)
    if scale is None:
        scale = d ** -0.5
    ws_bytes = attn_bwd_workspace_size(B, Hq, Hkv, N, d, deterministic)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 16),), dtype=torch.uint8, device=q.device)
    _check(_lib.attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                         B, Hq, Hkv, N, d, int(bool(causal)), float(scale), int(bool(deterministic)),
                         _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return dq, dk, dv


def attn_bwd_noalloc(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None,
                     deterministic: bool = False, dq=None, dk=None, dv=None, stream=None):
    """attn_bwd without a workspace, for callers that cannot allocate device memory on
    the call path; the library's own fixed 64 MiB array serves as the workspace (sizes
    needing more are rejected).  Overlapping calls on different streams race on it."""
    B, Hq, Hkv, N, d, dq, dk, dv = _bwd_tensors(q, k, v, o, lse, do, dq, dk, dv)
    if scale is None:
        scale = d ** -0.5
    _check(_lib.attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                                 _ptr(dv), B, Hq, Hkv, N, d, int(bool(causal)), float(scale),
                                 int(bool(deterministic)), _stream(stream)))
    return dq, dk, dv


def attn_quantize_fp8(x, x8=None, scales=None, stream=None):
    """e4m3 codes and per-128-row-block fp32 scales of x [B,H,N,128] bf16 (CUDA).  Returns
    (x8 uint8 [B,H,N,128], scales fp32 [B,H,ceil(N/128)])."""
    B, H, N, d = x.shape
    _dev_bf16("x", x, (B, H, N, d))
    nb = (N + 127) // 128
    x8 = torch.empty((B, H, N, d), dtype=torch.uint8, device=x.device) if x8 is None else x8
    scales = torch.empty((B, H, nb), dtype=torch.float32, device=x.device) if scales is None else scales
    if x8.dtype != torch.uint8 or not x8.is_contiguous() or tuple(x8.shape) != (B, H, N, d) or x8.device != x.device:
        raise ValueError("x8: expected a contiguous uint8 tensor shaped like x on its device")
    _dev_f32("scales", scales, (B, H, nb))
    _check(_lib.attn_quantize_fp8(_ptr(x), _ptr(x8), _ptr(scales), B, H, N, d, _stream(stream)))
    return x8, scales


def attn_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, causal: bool = False, scale: float | None = None, o=None,
                 lse=None, stream=None):
    """O, LSE of the FP8 inputs (e4m3 codes as uint8 tensors q8 [B,Hq,N,128], k8/v8
    [B,Hkv,N,128], fp32 block scales [.., ceil(N/128)] as attn_quantize_fp8 returns them).
    O is bf16, LSE fp32."""
    B, Hq, N, d = q8.shape
    Hkv = k8.shape[1]
    nb = (N + 127) // 128
    for name, t, shp in (("q8", q8, (B, Hq, N, d)), ("k8", k8, (B, Hkv, N, d)), ("v8", v8, (B, Hkv, N, d))):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != shp:
            raise ValueError(f"{name}: expected a contiguous CUDA uint8 tensor of shape {shp}")
    _dev_f32("q_scale", q_scale, (B, Hq, nb))
    _dev_f32("k_scale", k_scale, (B, Hkv, nb))
    _dev_f32("v_scale", v_scale, (B, Hkv, nb))
    if scale is None:
        scale = d ** -0.5
    o = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=q8.device) if o is None else o
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q8.device) if lse is None else lse
    _dev_bf16("o", o, (B, Hq, N, d))
    _dev_f32("lse", lse, (B, Hq, N))
    _check(_lib.attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), _ptr(o),
                             _ptr(lse), B, Hq, Hkv, N, d, int(bool(causal)), float(scale), _stream(stream)))
    return o, lse


# The current device's index, and the raw current stream of a device: what torch.cuda.current_device()
# and current_stream() return, without making a Stream object (3 us of a call's host time).
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


@contextlib.contextmanager
def _there(device, stream):
    """``device`` and ``stream`` (a torch stream, a raw one or None) made current, so that what a
    call allocates belongs to the stream it runs on and is not handed out again before it has run."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            # 0 is the legacy default stream; ExternalStream(0) would be some stream of torch's pool.
            raw = int(stream)
            stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            yield


def _bad(name, t, dtype, shape, device):
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")


def _plain(name, t, dtype, shape, device):
    """A contiguous tensor of this type and shape on this device, or ValueError."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _bad(name, t, dtype, shape, device)


def attn_rope_freqs(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                    trained_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda",
                    ramp: str = "pairs"):
    """(inv_freq, mscale) for ``attn_rope``: fp64 [rot/2] radians per position, base^(-2j/rot),
    and the factor on the rotated columns.  ``scaling`` for contexts ``factor`` times longer:

    * ``"none"``;
    * ``"linear"``: positions compressed, every frequency divided by ``factor``;
    * ``"ntk"``: the base raised to base * factor^(rot / (rot - 2)), so that the slowest pair is
      compressed by ``factor`` and the fastest left alone;
    * ``"yarn"``: by the turns a pair makes over ``trained_length`` positions: from ``beta_fast``
      turns on left alone, up to ``beta_slow`` turns compressed, blended in between; mscale =
      0.1 ln(factor) + 1.  ``ramp`` says how: ``"pairs"``, linearly in the pair's index j from the
      last pair with ``beta_fast`` turns or more to the first with ``beta_slow`` or fewer, which is
      what released checkpoints were trained with; ``"turns"``, linearly in the number of turns,
      which is the method's published formula.  (128 columns, base 10^4, factor 4 over 8192 positions:
      24 of 64 frequencies differ, by up to 41 %.)
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot={rot} must be even and at least 2")
    if not (base > 1.0 and math.isfinite(base)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("base must be finite and > 1, factor finite and >= 1")
    j = torch.arange(0, rot, 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "ntk":
        if rot == 2:
            raise ValueError("scaling='ntk' needs rot > 2")
        base *= factor ** (rot / (rot - 2))
    f = float(base) ** (-j / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if trained_length < 1 or not beta_fast > beta_slow:
            raise ValueError("scaling='yarn' needs trained_length >= 1 and beta_fast > beta_slow")
        if ramp == "turns":
            turns = trained_length * f / (2 * math.pi)
            keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        elif ramp == "pairs":
            if not beta_slow > 0:
                raise ValueError("ramp='pairs' needs beta_slow > 0")
            # Pair j makes trained_length base^(-2j/rot) / 2 pi turns: the (real) j that makes n of them.
            pair = lambda n: rot * math.log(trained_length / (2 * math.pi * n)) / (2 * math.log(base))
            first, last = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
            keep = 1 - ((j / 2 - first) / max(last - first, 1e-3)).clamp(0, 1)
        else:
            raise ValueError(f"ramp={ramp!r} (pairs or turns)")
        f = f * keep + f / factor * (1 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling={scaling!r} (none, linear, ntk or yarn)")
    return f.to(device), mscale


_Strides12, _Strides4 = _ll * 12, _ll * 4


def _bad_rows(dev, *rows):
    """ValueError for the first (name, tensor, shape) that is not a bf16 tensor of that shape with
    contiguous columns on the device."""
    for name, t, shape in rows:
        if t is not None and (t.dtype is not torch.bfloat16 or t.shape != shape or t.device != dev or t.stride()[-1] != 1):
            raise ValueError(f"{name}: expected a bf16 tensor of shape {tuple(shape)} with contiguous columns on {dev}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _rope(call, q, k, inv_freq, positions, interleaved, mscale, q_out, k_out, stream):
    shape, dev, bf16 = q.shape, q.device, torch.bfloat16
    dims = len(shape)
    if dims not in (3, 4) or not q.is_cuda:
        raise ValueError(f"q: expected a CUDA tensor [B,H,N,d] or [H,T,d], got {tuple(shape)} on {dev}")
    if stream is not None or dev.index != _current_device():
        with _there(dev, stream):
            return _rope(call, q, k, inv_freq, positions, interleaved, mscale, q_out, k_out, None)
    if dims == 4:
        B, Hq, N, d = shape
    else:
        B, (Hq, N, d) = 1, shape
    if q_out is None:
        q_out = torch.empty(shape, dtype=bf16, device=dev)
    sq, oq = q.stride(), q_out.stride()
    ok = (q.dtype is bf16 and q_out.dtype is bf16 and q_out.shape == shape and q_out.device == dev and sq[-1] == 1
          and oq[-1] == 1)
    kshape, Hk, sk, pk, pok = None, 0, sq, None, None
    so = sk
    if k is not None:
        kshape = (B, k.shape[1], N, d) if dims == 4 and k.dim() == 4 else (k.shape[0], N, d)
        Hk = kshape[-3]
        if k_out is None:
            k_out = torch.empty(kshape, dtype=bf16, device=dev)
        sk, so = k.stride(), k_out.stride()
        ok = (ok and k.dtype is bf16 and k_out.dtype is bf16 and k.shape == kshape and k_out.shape == kshape
              and len(kshape) == dims and k.device == dev and k_out.device == dev and sk[-1] == 1 and so[-1] == 1)
        pk, pok = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    if not ok:
        if kshape is not None and len(kshape) != dims:
            raise ValueError(f"k: expected as many dimensions as q, got {tuple(k.shape)}")
        _bad_rows(dev, ("q", q, shape), ("q_out", q_out, shape), ("k", k, kshape), ("k_out", k_out, kshape))
    half = inv_freq.numel()
    _plain("inv_freq", inv_freq, torch.float64, (half,), dev)
    pos = None
    if positions is not None:
        _plain("positions", positions, torch.int32, (N,) if dims == 3 and positions.dim() == 1 else (B, N), dev)
        pos = positions.data_ptr()
    if dims == 4:
        strides = _Strides12(sq[0], sq[1], sq[2], sk[0], sk[1], sk[2], oq[0], oq[1], oq[2], so[0], so[1], so[2])
    else:
        strides = _Strides12(0, sq[0], sq[1], 0, sk[0], sk[1], 0, oq[0], oq[1], 0, so[0], so[1])
    _check(call(q.data_ptr(), pk, q_out.data_ptr(), pok, inv_freq.data_ptr(), pos, B, Hq, Hk, N, d, 2 * half,
                1 if interleaved else 0, mscale, strides, _current_stream(dev.index)))
    return q_out, k_out


def attn_rope(q, k, inv_freq, positions=None, interleaved: bool = False, mscale: float = 1.0, q_out=None, k_out=None,
              stream=None):
    """q and k (or None) with rotary positions: bf16 [B,H,N,d] (or packed [H,T,d]) CUDA tensors of
    any strides with contiguous columns, such as views of a fused projection.  ``inv_freq``: fp64
    [rot/2] (``attn_rope_freqs``); ``positions``: int32 [B,N] ([T] when packed), default 0 .. N-1.
    Pairs are columns (j, j + rot/2), or (2j, 2j+1) with ``interleaved``.  Returns (q_out, k_out),
    new contiguous tensors unless given; an output may be its own input (in place)."""
    return _rope(_lib.attn_rope, q, k, inv_freq, positions, interleaved, mscale, q_out, k_out, stream)


def attn_rope_bwd(dq, dk, inv_freq, positions=None, interleaved: bool = False, mscale: float = 1.0, q_out=None,
                  k_out=None, stream=None):
    """Gradients of ``attn_rope``'s inputs from those of its outputs (the transposed rotation;
    arguments as there)."""
    return _rope(_lib.attn_rope_bwd, dq, dk, inv_freq, positions, interleaved, mscale, q_out, k_out, stream)


def _cache_tensors(k_cache, v_cache, k_scale, v_scale, page_table, cu, cu_name, kv_lens, dev):
    """Checks a paged cache and its index tensors; (num_pages, Hkv, page_size, d, B, max_pages)."""
    shape = k_cache.shape
    if len(shape) != 4 or page_table.dim() != 2:
        raise ValueError(f"expected k_cache [num_pages, Hkv, page_size, d] and page_table [B, max_pages], got {tuple(shape)} "
                         f"and {tuple(page_table.shape)}")
    B, width = page_table.shape
    pairs, u8, f32, i32 = shape[:2], torch.uint8, torch.float32, torch.int32
    # One condition for all, since the checks are most of a call's host time; then the one that failed.
    if not (k_cache.dtype is u8 and v_cache.dtype is u8 and k_scale.dtype is f32 and v_scale.dtype is f32
            and page_table.dtype is i32 and cu.dtype is i32 and kv_lens.dtype is i32
            and v_cache.shape == shape and k_scale.shape == pairs and v_scale.shape == pairs and cu.shape == (B + 1,)
            and kv_lens.shape == (B,)
            and k_cache.device == dev and v_cache.device == dev and k_scale.device == dev and v_scale.device == dev
            and page_table.device == dev and cu.device == dev and kv_lens.device == dev
            and k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous()
            and v_scale.is_contiguous() and page_table.is_contiguous() and cu.is_contiguous()
            and kv_lens.is_contiguous()):
        for name, t, dtype, want in (("k_cache", k_cache, u8, shape), ("v_cache", v_cache, u8, shape),
                                     ("k_scale", k_scale, f32, pairs), ("v_scale", v_scale, f32, pairs),
                                     ("page_table", page_table, i32, (B, width)), (cu_name, cu, i32, (B + 1,)),
                                     ("kv_lens", kv_lens, i32, (B,))):
            _plain(name, t, dtype, want, dev)
    return (*shape, B, width)


def attn_kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, kv_lens, stream=None):
    """Appends packed rows k, v ([Hkv, total, d] CUDA bf16, contiguous columns, strides multiples
    of 8) to the paged cache in place: k_cache, v_cache uint8 [num_pages, Hkv, page_size, d] e4m3
    codes, k_scale, v_scale fp32 [num_pages, Hkv].  ``page_table`` int32 [B, max_pages];
    ``cu_seqlens`` int32 [B + 1], the new rows of each sequence; ``kv_lens`` int32 [B], its rows
    after the call.  Each page's scale is a power of two that keeps its rows within +-448 codes;
    the offsets, lengths and pages are checked on the device (attn_device_status())."""
    if not k.is_cuda or k.dim() != 3:
        raise ValueError(f"k: expected a CUDA tensor [Hkv, total, d], got {tuple(k.shape)} on {k.device}")
    dev = k.device
    if stream is not None or dev.index != _current_device():
        with _there(dev, stream):
            return attn_kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, kv_lens)
    pages, Hkv, P, d, B, width = _cache_tensors(k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, "cu_seqlens",
                                                kv_lens, dev)
    T = k.shape[1]
    shape, bf16 = (Hkv, T, d), torch.bfloat16
    sk, sv = k.stride(), v.stride()
    if not (k.dtype is bf16 and v.dtype is bf16 and k.shape == shape and v.shape == shape and v.device == dev
            and sk[2] == 1 and sv[2] == 1):
        _bad_rows(dev, ("k", k, shape), ("v", v, shape))
    _check(_lib.attn_kv_append_fp8(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                   k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(), cu_seqlens.data_ptr(),
                                   kv_lens.data_ptr(), B, Hkv, T, d, pages, P, width,
                                   _Strides4(sk[0], sk[1], sv[0], sv[1]), _current_stream(dev.index)))


def attn_fwd_kv_fp8_workspace_size(B: int, Hq: int, Hkv: int, total_q: int, max_q: int, d: int) -> int:
    n = _lib.attn_fwd_kv_fp8_workspace_size(B, Hq, Hkv, total_q, max_q, d)
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(-1, attn_last_error())
    return int(n)


def attn_fwd_kv_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, kv_lens, max_q: int,
                    causal: bool = True, scale: float | None = None, o=None, lse=None, workspace=None, stream=None):
    """O, LSE of packed queries q [Hq, total_q, d] (CUDA bf16) over a paged e4m3 cache (tensors as
    ``attn_kv_append_fp8``): sequence b's n = cu_seqlens_q[b+1] - cu_seqlens_q[b] <= ``max_q`` <=
    total_q queries stand at its last n of kv_lens[b] keys (causal: query i sees keys up to
    i + kv_lens[b] - n).  ``workspace``: a uint8 CUDA tensor of at least
    attn_fwd_kv_fp8_workspace_size(...) bytes (allocated when None).  The offsets, lengths and
    pages are checked on the device (attn_device_status())."""
    if not q.is_cuda or q.dim() != 3:
        raise ValueError(f"q: expected a CUDA tensor [Hq, total_q, d], got {tuple(q.shape)} on {q.device}")
    dev = q.device
    if stream is not None or dev.index != _current_device():
        with _there(dev, stream):
            return attn_fwd_kv_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, kv_lens, max_q, causal,
                                   scale, o, lse, workspace)
    pages, Hkv, P, d, B, width = _cache_tensors(k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q,
                                                "cu_seqlens_q", kv_lens, dev)
    Hq, T, _ = q.shape
    shape = (Hq, T, d)
    if o is None:
        o = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    if not (q.dtype is torch.bfloat16 and o.dtype is torch.bfloat16 and lse.dtype is torch.float32 and q.shape == shape
            and o.shape == shape and lse.shape == (Hq, T) and o.device == dev and lse.device == dev
            and q.is_contiguous() and o.is_contiguous() and lse.is_contiguous()):
        _plain("q", q, torch.bfloat16, shape, dev)
        _plain("o", o, torch.bfloat16, shape, dev)
        _plain("lse", lse, torch.float32, (Hq, T), dev)
    if workspace is None:
        n = attn_fwd_kv_fp8_workspace_size(B, Hq, Hkv, T, max_q, d)
        workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {dev}")
    _check(_lib.attn_fwd_kv_fp8(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), page_table.data_ptr(), cu_seqlens_q.data_ptr(), kv_lens.data_ptr(),
                                o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, T, max_q, d, pages, P, width,
                                1 if causal else 0, d ** -0.5 if scale is None else scale, workspace.data_ptr(),
                                workspace.nbytes, _current_stream(dev.index)))
    return o, lse


def attn_set_debug_knobs(tau: float = 8.0, poly_per_16: int = 0, wait_limit_ns: int = 2_000_000_000,
                         sync_check: bool = False):
    _check(_lib.attn_set_debug_knobs(float(tau), int(poly_per_16), int(wait_limit_ns), int(bool(sync_check))))


def attn_get_debug_knobs():
    tau, poly, wl, sc = _f(), _i(), _ll(), _i()
    _check(_lib.attn_get_debug_knobs(ctypes.byref(tau), ctypes.byref(poly), ctypes.byref(wl), ctypes.byref(sc)))
    return {"tau": tau.value, "poly_per_16": poly.value, "wait_limit_ns": wl.value, "sync_check": bool(sc.value)}


def attn_set_test_hooks(skip_first_kv_load: bool = False):
    _check(_lib.attn_set_test_hooks(int(bool(skip_first_kv_load))))


def attn_device_status(clear: bool = True) -> int:
    """Synchronise and return the raw status (0 = fine, ATTN_ERR_TIMEOUT = a kernel gave up)."""
    return int(_lib.attn_device_status(int(bool(clear))))


def attn_rescale_counter(enable: bool) -> int:
    v = ctypes.c_ulonglong(0)
    _check(_lib.attn_rescale_counter(int(bool(enable)), ctypes.byref(v)))
    return int(v.value)


def attn_exp2_sw(x, variant: int = 0, stream=None):
    """y = 2^x on the GPU: variant 0 = polynomial as used in the forward, 1 = polynomial
    with correct subnormals, 2 = MUFU ex2.approx."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x: contiguous CUDA fp32 tensor expected")
    y = torch.empty_like(x)
    _check(_lib.attn_exp2_sw(_ptr(x), _ptr(y), x.numel(), int(variant), _stream(stream)))
    return y


__all__ = ["attn_fwd", "attn_fwd_fp8", "attn_quantize_fp8", "attn_bwd", "attn_bwd_noalloc", "attn_bwd_workspace_size", "attn_last_error", "attn_version",
           "attn_set_debug_knobs", "attn_get_debug_knobs", "attn_device_status", "attn_rescale_counter",
           "attn_exp2_sw", "attn_set_test_hooks", "attn_rope", "attn_rope_bwd", "attn_rope_freqs", "attn_kv_append_fp8",
           "attn_fwd_kv_fp8", "attn_fwd_kv_fp8_workspace_size", "AttnError", "LIB_PATH"]
