"""Exact attention forward on GB300 (sm_103a): Python binding of libfa_gb300.

The functions here only marshal arguments (tensor pointers, sizes, the
current CUDA stream) into the C ABI declared in ``include/fa_gb300.h``; every
step of the computation runs in the library's CUDA kernels.  There is no CPU
or eager-PyTorch fallback: if the library is missing or the device is not an
sm_103 GPU the call raises.

    o, lse = fa_fwd(q, k, v, causal=True)          # q [B,Hq,Lq,D], k/v [B,Hkv,Lk,D]
    o, lse = fa_fwd_varlen(q, k, v, cu_q, cu_k, max_q, max_k, causal=True)
    o, lse = fa_fwd_splitkv(q, k, v, causal=True)    # decode: (Hq/Hkv)*Lq <= 16, long Lk
    dq, dk, dv = fa_bwd(q, k, v, o, lse, do, causal=True)
    o, lse = fa_fwd_variant(q, k, v, window=(4095, 0), softcap=0.0, alibi_slopes=None)

A paged KV cache held in 4 bits (pool uint8 [pages, Hkv, page_size / 16, 18 D], table int32 [slots, W], seq_lens
int32 [slots], refs int32 [pages]; layout in include/fa_gb300.h):

    pool = kv4_pool(pages, Hkv, page_size, D)
    info = fa_kv4_reserve(new_tokens, table, seq_lens, refs, page_size)         # pages for new positions
    fa_kv4_append(k, v, cu_seqlens, pool, table, seq_lens)                      # quantise them into the cache
    o, lse = fa_fwd_kv4(q, pool, table, seq_lens, causal=True)                  # decode attention over it
    k, v = fa_kv4_read(cu_seqlens, total, pool, table, seq_lens)                # back to bf16 rows
    info = fa_kv4_fork(parents, children, pool, table, seq_lens, refs)          # share and copy pages
    fa_kv4_release(seq_ids, table, seq_lens, refs, page_size)
    info = fa_kv4_compact(pool, table, seq_lens, refs)

Rotary positions, and a paged KV cache in bf16 (pool bf16 [pages, 2, Hkv, page_size, D]; table, lengths, fa_kv4_reserve
and fa_kv4_release as above) for decoding, drafted trees and chunks of prompts:

    rope = rope_plan(D, base=500000.0)                                          # frequencies, on the device
    q, k = fa_rope(q, k, rope, positions)                                       # packed or dense rows
    dq, dk = fa_rope_bwd(dq, dk, rope, positions, dtype=torch.bfloat16)
    pool = kv16_pool(pages, Hkv, page_size, D)
    mask, depth = draft_mask(parents, cu_seqlens)                               # of drafted trees
    q = fa_kv16_append(k, v, cu_seqlens, pool, table, seq_lens, rope=rope, positions=positions, q=q)
    o, lse = fa_fwd_kv16(q, cu_seqlens, pool, table, seq_lens, mask=mask)       # or causal=True
    back = fa_kv16_keep(keep, counts, cu_seqlens, pool, table, seq_lens)        # accepted nodes to the front
    info = fa_kv4_reserve(back, table, seq_lens, refs, page_size)               # the others' positions given back
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading
from fractions import Fraction

import torch

__all__ = ["fa_fwd", "fa_fwd_varlen", "fa_fwd_hdim", "fa_fwd_varlen_hdim", "fa_fwd_varlen_noalloc", "fa_fwd_variant", "fa_fwd_varlen_variant",
           "fa_fwd_splitkv", "fp8_prepare", "fa_fwd_fp8", "fp8_sections", "splitkv_workspace", "fa_bwd",
           "bwd_workspace", "fa_bwd_varlen", "bwd_varlen_workspace", "fa_bwd_variant", "fa_bwd_varlen_variant",
           "kv4_pool", "fa_kv4_append", "fa_kv4_read", "fa_fwd_kv4", "kv4_workspace", "fa_kv4_reserve", "fa_kv4_fork",
           "fa_kv4_release", "fa_kv4_compact", "kv4_pages_workspace", "RopePlan", "rope_plan", "fa_rope", "fa_rope_bwd",
           "kv16_pool", "fa_kv16_append", "fa_fwd_kv16", "kv16_workspace", "fa_kv16_keep", "draft_mask", "fa_check", "fa_status_string", "fa_last_launch_count",
           "FAError", "library_path", "load_library", "EXPORTED_SYMBOLS"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libfa_gb300.so")
_lock = threading.Lock()
_lib = None

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
EXPORTED_SYMBOLS = ("fa_fwd", "fa_fwd_varlen", "fa_fwd_hdim", "fa_fwd_varlen_hdim", "fa_fwd_varlen_noalloc", "fa_fwd_variant", "fa_fwd_varlen_variant",
                    "fa_fwd_splitkv", "fa_fwd_splitkv_workspace", "fa_bwd", "fa_bwd_workspace", "fa_bwd_varlen",
                    "fa_bwd_varlen_workspace", "fa_bwd_variant", "fa_bwd_varlen_variant", "fa_fp8_workspace",
                    "fa_fp8_prepare", "fa_fwd_fp8", "fa_kv4_append", "fa_kv4_read", "fa_fwd_kv4",
                    "fa_fwd_kv4_workspace", "fa_kv4_reserve", "fa_kv4_fork", "fa_kv4_release", "fa_kv4_compact",
                    "fa_kv4_pages_workspace", "fa_rope", "fa_rope_bwd", "fa_kv16_append", "fa_fwd_kv16",
                    "fa_fwd_kv16_workspace", "fa_kv16_keep", "fa_check", "fa_status_string", "fa_last_launch_count",
                    "fa_test_inject_fault")
SPLITKV_MAX_ROWS = 16  # (Hq / Hkv) * Lq limit of fa_fwd_splitkv
NOALLOC_MAX_SEQS = 16384  # FA_NOALLOC_MAX_SEQS in include/fa_gb300.h
KV4_MAX_ROWS = 64  # FA_KV4_MAX_ROWS: (Hq / Hkv) * Lq limit of fa_fwd_kv4
KV4_SEQS_WITHOUT_WORKSPACE = 2048  # FA_KV4_SEQS_WITHOUT_WORKSPACE: reserve and fork up to here
KV4_MAX_SLOTS = 65536  # FA_KV4_MAX_SLOTS
VARLEN_SEQS_PER_LAUNCH = 1536  # FA_VARLEN_SEQS_PER_LAUNCH (64 for head dimensions (192, 128))


class _Variant(ctypes.Structure):
    # struct fa_variant in include/fa_gb300.h
    _fields_ = [("window_left", ctypes.c_int), ("window_right", ctypes.c_int), ("softcap", ctypes.c_float),
                ("alibi_slopes", ctypes.c_void_p)]


class _KV4(ctypes.Structure):
    # struct fa_kv4 in include/fa_gb300.h
    _fields_ = [(n, ctypes.c_void_p) for n in ("pool", "table", "seq_lens", "seq_ids", "k_scale", "v_scale")] + [
        (n, ctypes.c_int) for n in ("num_pages", "num_slots", "table_width", "page_size", "Hkv", "D")]


class _KV4Pages(ctypes.Structure):
    # struct fa_kv4_pages in include/fa_gb300.h
    _fields_ = [(n, ctypes.c_void_p) for n in ("pool", "table", "seq_lens", "refs")] + [
        (n, ctypes.c_int) for n in ("num_pages", "num_slots", "table_width", "page_size", "Hkv", "D", "num_layers")]


class _Rope(ctypes.Structure):
    # struct fa_rope in include/fa_gb300.h
    _fields_ = [("freqs", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("start", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("mscale", ctypes.c_float)]


class _RotaryRows(ctypes.Structure):
    # struct fa_rotary_rows in include/fa_gb300.h
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [
        (n, ctypes.c_longlong) for n in ("x_batch", "x_token", "x_head", "y_batch", "y_token", "y_head")] + [
        ("heads", ctypes.c_int)]


class _KV16(ctypes.Structure):
    # struct fa_kv16 in include/fa_gb300.h
    _fields_ = [(n, ctypes.c_void_p) for n in ("pool", "table", "seq_lens", "seq_ids")] + [
        (n, ctypes.c_int) for n in ("num_pages", "num_slots", "table_width", "page_size", "Hkv", "D")]


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} (status {status})")


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libfa_gb300.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.fa_fwd.restype = i
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
        lib.fa_fwd_varlen.restype = i
        lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp]
        lib.fa_fwd_hdim.restype = i
        lib.fa_fwd_hdim.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp]
        lib.fa_fwd_varlen_hdim.restype = i
        lib.fa_fwd_varlen_hdim.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, i, f, vp]
        lib.fa_fwd_varlen_noalloc.restype = i
        lib.fa_fwd_varlen_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp]
        lib.fa_fwd_splitkv.restype = i
        lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp, ctypes.c_size_t, vp]
        lib.fa_fwd_splitkv_workspace.restype = i
        lib.fa_fwd_splitkv_workspace.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t),
                                                 ctypes.POINTER(ctypes.c_int)]
        vr = ctypes.POINTER(_Variant)
        lib.fa_fwd_variant.restype = i
        lib.fa_fwd_variant.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vr, f, vp]
        lib.fa_fwd_varlen_variant.restype = i
        lib.fa_fwd_varlen_variant.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vr, f, vp]
        lib.fa_fp8_workspace.restype = i
        lib.fa_fp8_workspace.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_fp8_prepare.restype = i
        lib.fa_fp8_prepare.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, ctypes.c_size_t, vp]
        lib.fa_fwd_fp8.restype = i
        lib.fa_fwd_fp8.argtypes = [vp, vp, vp, i, i, i, i, i, i, i, f, vp]
        lib.fa_bwd.restype = i
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, ctypes.c_size_t, vp]
        lib.fa_bwd_workspace.restype = i
        lib.fa_bwd_workspace.argtypes = [i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_bwd_varlen.restype = i
        lib.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp,
                                      ctypes.c_size_t, vp]
        lib.fa_bwd_variant.restype = i
        lib.fa_bwd_variant.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vr, f, vp, ctypes.c_size_t,
                                       vp]
        lib.fa_bwd_varlen_variant.restype = i
        lib.fa_bwd_varlen_variant.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vr,
                                              f, vp, ctypes.c_size_t, vp]
        lib.fa_bwd_varlen_workspace.restype = i
        lib.fa_bwd_varlen_workspace.argtypes = [i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        c4 = pg = ctypes.c_void_p  # a packed struct (bytes) or byref of a _KV4 or _KV4Pages
        sz, ll = ctypes.c_size_t, ctypes.c_longlong
        for name, args in (("fa_kv4_append", [vp, vp, vp, i, i, c4, vp]), ("fa_kv4_read", [vp, vp, vp, i, i, c4, vp]),
                           ("fa_fwd_kv4", [vp, vp, vp, i, i, i, i, f, c4, vp, sz, vp]),
                           ("fa_fwd_kv4_workspace", [i, i, i, i, i, ctypes.POINTER(sz)]),
                           ("fa_kv4_reserve", [vp, vp, i, pg, vp, vp, sz, vp]),
                           ("fa_kv4_fork", [vp, vp, i, pg, vp, vp, sz, vp]), ("fa_kv4_release", [vp, i, pg, vp]),
                           ("fa_kv4_compact", [pg, vp, vp, sz, vp]),
                           ("fa_kv4_pages_workspace", [i, i, ctypes.POINTER(sz)]),
                           ("fa_rope", [vp, vp, i, i, i, i, i, vp, vp, ll, vp]),
                           ("fa_rope_bwd", [vp, vp, i, i, i, i, i, vp, vp, ll, vp]),
                           ("fa_kv16_append", [vp, vp, vp, vp, i, i, vp, vp, vp, vp]),
                           ("fa_fwd_kv16", [vp, ll, ll, vp, vp, vp, i, i, i, vp, i, i, f, vp, vp, sz, vp]),
                           ("fa_fwd_kv16_workspace", [i, i, i, i, ctypes.POINTER(sz)]),
                           ("fa_kv16_keep", [vp, vp, vp, i, i, i, vp, vp, vp])):
            getattr(lib, name).restype = i
            getattr(lib, name).argtypes = args
        lib.fa_check.restype = i
        lib.fa_check.argtypes = [vp]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_status_string.argtypes = [i]
        lib.fa_last_launch_count.restype = i
        lib.fa_last_launch_count.argtypes = []
        lib.fa_test_inject_fault.restype = None
        lib.fa_test_inject_fault.argtypes = [i]
        _lib = lib
        return lib


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def fa_last_launch_count() -> int:
    return int(load_library().fa_last_launch_count())


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check_tensor(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int, on_device: bool = True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if on_device and t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fa_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
           softmax_scale: float | None = None, out: torch.Tensor | None = None,
           lse: torch.Tensor | None = None, stream=None):
    """Dense attention forward.  q [B,Hq,Lq,D], k/v [B,Hkv,Lk,D] bf16 CUDA.

    Returns (o [B,Hq,Lq,D] fp32, lse [B,Hq,Lq] fp32).  Asynchronous on the
    current (or given) stream.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, torch.bfloat16, 4)
    B, Hq, Lq, D = q.shape
    Bk, Hkv, Lk, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    _check_tensor(out, "out", torch.float32, 4)
    if tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, Lq):
        raise ValueError("out/lse shape mismatch")
    _check_tensor(lse, "lse", torch.float32, 3)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                        B, Hq, Hkv, Lq, Lk, D, int(bool(causal)), float(softmax_scale), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd")
    return out, lse


def _check_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse):
    """Dtypes, ranks, layouts and shapes of a packed call (q [Tq,Hq,D], k and
    v [Tk,Hkv,D], offsets of equal length, out [Tq,Hq,D], lse [Hq,Tq]) first,
    then that every tensor lives on a CUDA device.  Returns (Tq, Hq, D, Tk, Hkv)."""
    named = [(q, "q", torch.bfloat16, 3), (k, "k", torch.bfloat16, 3), (v, "v", torch.bfloat16, 3),
             (cu_seqlens_q, "cu_seqlens_q", torch.int32, 1), (cu_seqlens_k, "cu_seqlens_k", torch.int32, 1),
             (out, "out", torch.float32, 3), (lse, "lse", torch.float32, 2)]
    for t, n, dt, nd in named:
        _check_tensor(t, n, dt, nd, on_device=False)
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both hold num_seqs + 1 >= 2 offsets")
    if tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (Hq, Tq):
        raise ValueError(f"out must be {tuple(q.shape)} and lse {(Hq, Tq)}, got {tuple(out.shape)} and "
                         f"{tuple(lse.shape)}")
    for t, n, _, _ in named:
        if t.device.type != "cuda":
            raise ValueError(f"{n} must be a CUDA tensor")
    return Tq, Hq, D, Tk, Hkv


def fa_fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                  cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, causal: bool = False,
                  softmax_scale: float | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, stream=None):
    """Packed variable-length forward.  q [Tq,Hq,D], k/v [Tk,Hkv,D] bf16 CUDA,
    cu_seqlens_* int32 CUDA [num_seqs+1].  Returns (o [Tq,Hq,D] fp32, lse [Hq,Tq] fp32).
    Allocates nothing on the device beyond ``out``/``lse`` when they are not given."""
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    Tq, Hq, D, Tk, Hkv = _check_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                               cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cu_seqlens_q.numel() - 1,
                               Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D, int(bool(causal)),
                               float(softmax_scale), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_varlen")
    return out, lse


def fa_fwd_hdim(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                softmax_scale: float | None = None, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, stream=None):
    """Dense forward whose value head dimension Dv may differ from the
    query/key one D.  q [B,Hq,Lq,D], k [B,Hkv,Lk,D], v [B,Hkv,Lk,Dv] bf16 CUDA;
    (D, Dv) in {(64, 64), (128, 128), (192, 128)}.

    Returns (o [B,Hq,Lq,Dv] fp32, lse [B,Hq,Lq] fp32).  The default scale is
    1/sqrt(D).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, torch.bfloat16, 4)
    B, Hq, Lq, D = q.shape
    Bk, Hkv, Lk, Dk = k.shape
    Dv = v.shape[3]
    if tuple(v.shape[:3]) != tuple(k.shape[:3]) or Bk != B or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if out is None:
        out = torch.empty((B, Hq, Lq, Dv), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    _check_tensor(out, "out", torch.float32, 4)
    _check_tensor(lse, "lse", torch.float32, 3)
    if tuple(out.shape) != (B, Hq, Lq, Dv) or tuple(lse.shape) != (B, Hq, Lq):
        raise ValueError("out/lse shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_hdim(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                             B, Hq, Hkv, Lq, Lk, D, Dv, int(bool(causal)), float(softmax_scale),
                             _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_hdim")
    return out, lse


def fa_fwd_varlen_hdim(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                       cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, causal: bool = False,
                       softmax_scale: float | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, stream=None):
    """Packed forward with value head dimension Dv: q [Tq,Hq,D], k [Tk,Hkv,D],
    v [Tk,Hkv,Dv] bf16 CUDA.  Returns (o [Tq,Hq,Dv] fp32, lse [Hq,Tq] fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, torch.bfloat16, 3)
    _check_tensor(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check_tensor(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    Dv = v.shape[2]
    if tuple(v.shape[:2]) != (Tk, Hkv) or Dk != D or cu_seqlens_q.numel() != cu_seqlens_k.numel():
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((Tq, Hq, Dv), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    _check_tensor(out, "out", torch.float32, 3)
    _check_tensor(lse, "lse", torch.float32, 2)
    if tuple(out.shape) != (Tq, Hq, Dv) or tuple(lse.shape) != (Hq, Tq):
        raise ValueError("out/lse shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_varlen_hdim(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                    cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cu_seqlens_q.numel() - 1,
                                    Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D, Dv,
                                    int(bool(causal)), float(softmax_scale), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_varlen_hdim")
    return out, lse


def fa_fwd_varlen_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                          cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, out: torch.Tensor,
                          lse: torch.Tensor, causal: bool = False, softmax_scale: float | None = None,
                          stream=None):
    """Packed forward for callers that cannot call cudaMalloc on the hot path
    (a process whose device memory all belongs to its own allocator, a server
    that must not allocate while serving): the caller provides ``out`` and
    ``lse``, and the whole batch's schedule (at most NOALLOC_MAX_SEQS
    sequences) goes into a fixed array inside the library, so one attention
    launch covers it.  Calls that can overlap on the GPU share that array and
    must be ordered.  Every shape is checked before the library is touched."""
    Tq, Hq, D, Tk, Hkv = _check_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse)
    if cu_seqlens_q.numel() - 1 > NOALLOC_MAX_SEQS:
        raise ValueError(f"at most {NOALLOC_MAX_SEQS} sequences")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_varlen_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cu_seqlens_q.numel() - 1,
                                       Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D, int(bool(causal)),
                                       float(softmax_scale), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_varlen_noalloc")
    return out, lse


def _variant(window, softcap, alibi_slopes, Hq: int, device):
    if alibi_slopes is not None:
        _check_tensor(alibi_slopes, "alibi_slopes", torch.float32, 1)
        if alibi_slopes.numel() != Hq or alibi_slopes.device != device:
            raise ValueError("alibi_slopes must be a float32 tensor of Hq elements on the inputs' device")
    wl, wr = window
    return _Variant(int(wl), int(wr), float(softcap), alibi_slopes.data_ptr() if alibi_slopes is not None else None)


def fa_fwd_variant(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window=(-1, -1), softcap: float = 0.0,
                   alibi_slopes: torch.Tensor | None = None, softmax_scale: float | None = None,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Dense forward with a key window (left, right) around each query's
    bottom-right-aligned position (-1 = unlimited), soft-capping of the
    scaled scores, or ALiBi slopes per query head.  D = 64 or 128."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, torch.bfloat16, 4)
    B, Hq, Lq, D = q.shape
    Bk, Hkv, Lk, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D:
        raise ValueError("shape mismatch")
    out = torch.empty(q.shape, dtype=torch.float32, device=q.device) if out is None else out
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check_tensor(out, "out", torch.float32, 4)
    _check_tensor(lse, "lse", torch.float32, 3)
    if tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, Lq):
        raise ValueError("out/lse shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    var = _variant(window, softcap, alibi_slopes, Hq, q.device)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_variant(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq,
                                Hkv, Lq, Lk, D, ctypes.byref(var), float(softmax_scale), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_variant")
    return out, lse


def fa_fwd_varlen_variant(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                          cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, window=(-1, -1),
                          softcap: float = 0.0, alibi_slopes: torch.Tensor | None = None,
                          softmax_scale: float | None = None, out: torch.Tensor | None = None,
                          lse: torch.Tensor | None = None, stream=None):
    """Packed forward with a variant; windows and distances are per sequence."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, torch.bfloat16, 3)
    _check_tensor(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check_tensor(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    out = torch.empty(q.shape, dtype=torch.float32, device=q.device) if out is None else out
    lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check_tensor(out, "out", torch.float32, 3)
    _check_tensor(lse, "lse", torch.float32, 2)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    var = _variant(window, softcap, alibi_slopes, Hq, q.device)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_varlen_variant(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cu_seqlens_q.numel() - 1,
                                       Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D, ctypes.byref(var),
                                       float(softmax_scale), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_varlen_variant")
    return out, lse


def fp8_sections(B: int, Hq: int, Hkv: int, Lq: int, Lk: int) -> dict:
    """Byte offsets and shapes of the sections of a prepared FP8 buffer (the
    layout documented with fa_fp8_prepare in include/fa_gb300.h)."""
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    nq, nk = (Lq + 127) // 128, (Lk + 127) // 128
    lk_pad = nk * 128
    sec, off = {}, 0
    for name, nbytes, shape in (("qc", B * Hq * Lq * 128, (B, Hq, Lq, 128)), ("kc", B * Hkv * Lk * 128, (B, Hkv, Lk, 128)),
                                ("vt", B * Hkv * 128 * lk_pad, (B, Hkv, 128, lk_pad)), ("sq", B * Hq * nq * 4, (B, Hq, nq)),
                                ("sk", B * Hkv * nk * 4, (B, Hkv, nk)), ("sv", B * Hkv * 4, (B, Hkv)),
                                ("vmax", B * Hkv * 4, (B, Hkv))):
        sec[name] = (off, nbytes, shape)
        off = up(off + nbytes)
    sec["total"] = off
    return sec


def fp8_prepare(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, signs: torch.Tensor,
                prepared: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotate and quantise bf16 q [B,Hq,Lq,128], k/v [B,Hkv,Lk,128] for
    fa_fwd_fp8; signs: fp32 CUDA [128] of +-1.  Returns the prepared buffer
    (a CUDA uint8 tensor)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, torch.bfloat16, 4)
    _check_tensor(signs, "signs", torch.float32, 1)
    B, Hq, Lq, D = q.shape
    _, Hkv, Lk, _ = k.shape
    lib = load_library()
    n = ctypes.c_size_t(0)
    st = lib.fa_fp8_workspace(B, Hq, Hkv, Lq, Lk, D, ctypes.byref(n))
    if st != FA_OK:
        raise FAError(st, "fa_fp8_workspace")
    if prepared is None or prepared.numel() < n.value:
        prepared = torch.empty(n.value, dtype=torch.uint8, device=q.device)
    with torch.cuda.device(q.device):
        st = lib.fa_fp8_prepare(q.data_ptr(), k.data_ptr(), v.data_ptr(), signs.data_ptr(), B, Hq, Hkv, Lq, Lk, D,
                                prepared.data_ptr(), prepared.numel(), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fp8_prepare")
    return prepared


def fa_fwd_fp8(prepared: torch.Tensor, B: int, Hq: int, Hkv: int, Lq: int, Lk: int, causal: bool = False,
               softmax_scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               D: int = 128, stream=None):
    """Attention of a buffer made by fp8_prepare.  Returns (o fp32 [B,Hq,Lq,D], lse fp32 [B,Hq,Lq])."""
    out = torch.empty((B, Hq, Lq, D), dtype=torch.float32, device=prepared.device) if out is None else out
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=prepared.device) if lse is None else lse
    _check_tensor(out, "out", torch.float32, 4)
    _check_tensor(lse, "lse", torch.float32, 3)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(prepared.device):
        st = lib.fa_fwd_fp8(prepared.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Lq, Lk, D,
                            int(bool(causal)), float(softmax_scale), _stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_fp8")
    return out, lse


def splitkv_workspace(B: int, Hq: int, Hkv: int, Lq: int, Lk: int, D: int, num_splits: int = 0) -> tuple[int, int]:
    """(workspace bytes, partitions) fa_fwd_splitkv uses for this shape on the current device."""
    nbytes, used = ctypes.c_size_t(0), ctypes.c_int(0)
    st = load_library().fa_fwd_splitkv_workspace(B, Hq, Hkv, Lq, Lk, D, int(num_splits), ctypes.byref(nbytes),
                                                 ctypes.byref(used))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_splitkv_workspace")
    return int(nbytes.value), int(used.value)


def fa_fwd_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                   softmax_scale: float | None = None, num_splits: int = 0, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Split-KV (decode) forward.  q [B,Hq,Lq,D], k/v [B,Hkv,Lk,D] bf16 CUDA with
    (Hq/Hkv)*Lq <= 16.  ``num_splits`` <= 0 lets the library choose.  The
    partial-result workspace is taken from ``workspace`` (a CUDA uint8 tensor)
    or allocated here through PyTorch.  Returns (o fp32, lse fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, torch.bfloat16, 4)
    B, Hq, Lq, D = q.shape
    Bk, Hkv, Lk, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    _check_tensor(out, "out", torch.float32, 4)
    _check_tensor(lse, "lse", torch.float32, 3)
    if tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, Lq):
        raise ValueError("out/lse shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(q.device):
        nbytes, _ = splitkv_workspace(B, Hq, Hkv, Lq, Lk, D, num_splits)
        if nbytes and (workspace is None or workspace.numel() * workspace.element_size() < nbytes):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        ws_ptr = workspace.data_ptr() if (nbytes and workspace is not None) else None
        ws_len = workspace.numel() * workspace.element_size() if ws_ptr else 0
        st = lib.fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                B, Hq, Hkv, Lq, Lk, D, int(bool(causal)), float(softmax_scale), int(num_splits),
                                ws_ptr, ws_len, _stream_handle(stream))
        if ws_ptr and isinstance(stream, torch.cuda.Stream):
            workspace.record_stream(stream)  # keep the block out of reuse until that stream is done
    if st != FA_OK:
        raise FAError(st, "fa_fwd_splitkv")
    return out, lse


def bwd_workspace(B: int, Hq: int, Lq: int) -> int:
    """Workspace bytes fa_bwd needs."""
    nbytes = ctypes.c_size_t(0)
    st = load_library().fa_bwd_workspace(B, Hq, Lq, ctypes.byref(nbytes))
    if st != FA_OK:
        raise FAError(st, "fa_bwd_workspace")
    return int(nbytes.value)


def fa_bwd_variant(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                   dout: torch.Tensor, window=(-1, -1), softcap: float = 0.0,
                   alibi_slopes: torch.Tensor | None = None, softmax_scale: float | None = None,
                   dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """Backward of fa_fwd_variant for key windows, soft-capping and ALiBi
    (D = 64 or 128); o and lse from fa_fwd_variant with the same variant."""
    var = _variant(window, softcap, alibi_slopes, q.shape[1], q.device)
    return fa_bwd(q, k, v, o, lse, dout, False, softmax_scale, dq, dk, dv, workspace, stream, variant=var)


def fa_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
           dout: torch.Tensor, causal: bool = False, softmax_scale: float | None = None,
           dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None, stream=None, variant=None):
    """Backward of fa_fwd.  q/dout [B,Hq,Lq,D], k/v [B,Hkv,Lk,D] bf16; o fp32
    [B,Hq,Lq,D] and lse fp32 [B,Hq,Lq] from fa_fwd.  Returns (dq, dk, dv) fp32."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _check_tensor(t, n, torch.bfloat16, 4)
    _check_tensor(o, "o", torch.float32, 4)
    _check_tensor(lse, "lse", torch.float32, 3)
    B, Hq, Lq, D = q.shape
    Bk, Hkv, Lk, Dk = k.shape
    if (tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D or tuple(dout.shape) != tuple(q.shape)
            or tuple(o.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, Lq)):
        raise ValueError("shape mismatch")
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.float32, device=q.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=torch.float32, device=q.device) if dv is None else dv
    for t, n, shp in ((dq, "dq", q.shape), (dk, "dk", k.shape), (dv, "dv", k.shape)):
        _check_tensor(t, n, torch.float32, 4)
        if tuple(t.shape) != tuple(shp):
            raise ValueError(f"{n} shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with torch.cuda.device(q.device):
        nbytes = bwd_workspace(B, Hq, Lq)
        if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Lq, Lk, D)
        tail = (float(softmax_scale), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                _stream_handle(stream))
        if variant is None:
            st, name = lib.fa_bwd(*args, int(bool(causal)), *tail), "fa_bwd"
        else:
            st, name = lib.fa_bwd_variant(*args, ctypes.byref(variant), *tail), "fa_bwd_variant"
        if isinstance(stream, torch.cuda.Stream):
            workspace.record_stream(stream)
    if st != FA_OK:
        raise FAError(st, name)
    return dq, dk, dv


def bwd_varlen_workspace(num_seqs: int, total_q: int, Hq: int) -> int:
    """Workspace bytes fa_bwd_varlen needs."""
    nbytes = ctypes.c_size_t(0)
    st = load_library().fa_bwd_varlen_workspace(num_seqs, total_q, Hq, ctypes.byref(nbytes))
    if st != FA_OK:
        raise FAError(st, "fa_bwd_varlen_workspace")
    return int(nbytes.value)


def fa_bwd_varlen_variant(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                          dout: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                          max_seqlen_q: int, max_seqlen_k: int, window=(-1, -1), softcap: float = 0.0,
                          alibi_slopes: torch.Tensor | None = None, softmax_scale: float | None = None,
                          dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                          dv: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Backward of fa_fwd_varlen_variant for key windows, soft-capping and
    ALiBi (D = 64 or 128)."""
    var = _variant(window, softcap, alibi_slopes, q.shape[1], q.device)
    return fa_bwd_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, False,
                         softmax_scale, dq, dk, dv, workspace, stream, variant=var)


def fa_bwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                  dout: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_seqlen_q: int,
                  max_seqlen_k: int, causal: bool = False, softmax_scale: float | None = None,
                  dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None, variant=None):
    """Backward of fa_fwd_varlen.  q/dout [Tq,Hq,D], k/v [Tk,Hkv,D] bf16; o fp32
    [Tq,Hq,D] and lse fp32 [Hq,Tq] from fa_fwd_varlen; cu_seqlens_* int32 CUDA.
    Returns (dq, dk, dv) fp32 in the layouts of q, k and v."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _check_tensor(t, n, torch.bfloat16, 3)
    _check_tensor(o, "o", torch.float32, 3)
    _check_tensor(lse, "lse", torch.float32, 2)
    _check_tensor(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check_tensor(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if (tuple(v.shape) != tuple(k.shape) or Dk != D or tuple(dout.shape) != tuple(q.shape)
            or tuple(o.shape) != tuple(q.shape) or tuple(lse.shape) != (Hq, Tq)
            or cu_seqlens_q.numel() != cu_seqlens_k.numel()):
        raise ValueError("shape mismatch")
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.float32, device=q.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=torch.float32, device=q.device) if dv is None else dv
    for t, n, shp in ((dq, "dq", q.shape), (dk, "dk", k.shape), (dv, "dv", k.shape)):
        _check_tensor(t, n, torch.float32, 3)
        if tuple(t.shape) != tuple(shp):
            raise ValueError(f"{n} shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    n_seqs = cu_seqlens_q.numel() - 1
    lib = load_library()
    with torch.cuda.device(q.device):
        nbytes = bwd_varlen_workspace(n_seqs, Tq, Hq)
        if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                n_seqs, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D)
        tail = (float(softmax_scale), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                _stream_handle(stream))
        if variant is None:
            st, name = lib.fa_bwd_varlen(*args, int(bool(causal)), *tail), "fa_bwd_varlen"
        else:
            st, name = lib.fa_bwd_varlen_variant(*args, ctypes.byref(variant), *tail), "fa_bwd_varlen_variant"
        if isinstance(stream, torch.cuda.Stream):
            workspace.record_stream(stream)
    if st != FA_OK:
        raise FAError(st, name)
    return dq, dk, dv


# ------------------------------------------------------------- 4-bit cache

def kv4_pool(num_pages: int, Hkv: int, page_size: int, D: int, layers: int | None = None,
             device="cuda") -> torch.Tensor:
    """An empty (all zero) pool of a 4-bit paged KV cache: uint8 [num_pages, Hkv,
    page_size / 16, 18 D], with ``layers`` in front when given."""
    if page_size not in (16, 32, 64, 128, 256) or D not in (64, 128):
        raise ValueError("page_size must be 16, 32, 64, 128 or 256 and D 64 or 128")
    shape = (num_pages, Hkv, page_size // 16, 18 * D)
    return torch.zeros(shape if layers is None else (layers, *shape), dtype=torch.uint8, device=device)


# A decode step makes one such call per layer, a few microseconds of kernel
# each, so the checks below take their time only on the way to an error.

_pack_kv4 = struct.Struct("6P6i").pack    # struct fa_kv4
_KV4_UNITS, _KV4_PAGES = (18 * 64, 18 * 128), (1, 2, 4, 8, 16)  # bytes of a unit, units of a page
_pack_pages = struct.Struct("4P7i").pack  # struct fa_kv4_pages


def _want(t, name, dtype, ndim, device):
    """_check_tensor, and that t is on `device` (a device index)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_cuda and t.is_contiguous()):
        _check_tensor(t, name, dtype, ndim)
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")


def _on_device(index, fn, *args):
    """fn(*args) with the device current."""
    if torch._C._cuda_getDevice() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _on_stream(stream, like, fn, *args, **scratch):
    """fn(*args, **scratch) with `stream` current: a torch stream, or a raw handle, of the device that `like`, a tensor
    of the call, is on.  What the call allocates belongs to that stream; the results may then be used on the caller's
    stream once that waits for it.  A caller's workspace (`scratch`) is kept out of reuse until a torch stream is done
    with it."""
    device = like.get_device() if isinstance(like, torch.Tensor) else -1
    if device < 0:
        return fn(*args, **scratch)  # which refuses it
    named = isinstance(stream, torch.cuda.Stream)
    if not named:
        handle = _stream_handle(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    if stream.device.index != device:
        raise ValueError(f"stream must be of cuda:{device}, got one of {stream.device}")
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        got = fn(*args, **scratch)
    for t in scratch.values():
        if named and t is not None and t.get_device() == device:
            t.record_stream(stream)
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            t.record_stream(here)
    return got


def _check_slots(table, seq_lens, device):
    _want(table, "table", torch.int32, 2, device)
    _want(seq_lens, "seq_lens", torch.int32, 1, device)
    if seq_lens.shape[0] != table.shape[0]:
        raise ValueError(f"table has {table.shape[0]} slots and seq_lens {seq_lens.shape[0]}")


def _check_pool(pool, ndim):
    _check_tensor(pool, "pool", torch.uint8, ndim)
    U, unit = pool.shape[-2:]
    if unit not in _KV4_UNITS or U not in _KV4_PAGES:
        raise ValueError(f"pool must be uint8 [..., pages, Hkv, page_size / 16, 18 D], got {tuple(pool.shape)}")


def _kv4(pool, table, seq_lens, seq_ids, k_scale, v_scale, num_seqs):
    """Checks the cache of a call with num_seqs sequences.  Returns (fa_kv4_t as bytes, device index, Hkv, D)."""
    device = pool.get_device() if isinstance(pool, torch.Tensor) else -1
    if not (device >= 0 and isinstance(table, torch.Tensor) and isinstance(seq_lens, torch.Tensor)
            and pool.dtype is torch.uint8 and pool.dim() == 4 and pool.is_contiguous()
            and table.dtype is torch.int32 and table.dim() == 2 and table.is_contiguous()
            and table.get_device() == device and seq_lens.dtype is torch.int32 and seq_lens.dim() == 1
            and seq_lens.is_contiguous() and seq_lens.get_device() == device):
        _check_pool(pool, 4)
        _check_slots(table, seq_lens, device)
    N, H, U, unit = pool.shape
    slots, width = table.shape
    if unit not in _KV4_UNITS or U not in _KV4_PAGES:
        _check_pool(pool, 4)
    if seq_lens.shape[0] != slots:
        _check_slots(table, seq_lens, device)
    ids = ks = vs = 0
    if seq_ids is not None:
        _want(seq_ids, "seq_ids", torch.int32, 1, device)
        if seq_ids.shape[0] != num_seqs:
            raise ValueError(f"seq_ids must name {num_seqs} slots")
        ids = seq_ids.data_ptr()
    elif num_seqs > slots:
        raise ValueError(f"{num_seqs} sequences but {slots} slots")
    if k_scale is not None:
        _want(k_scale, "k_scale", torch.float32, 1, device)
        ks = k_scale.data_ptr()
    if v_scale is not None:
        _want(v_scale, "v_scale", torch.float32, 1, device)
        vs = v_scale.data_ptr()
    if ks and k_scale.shape[0] != H or vs and v_scale.shape[0] != H:
        raise ValueError(f"k_scale and v_scale must hold one scale for each of the {H} KV heads")
    c = _pack_kv4(pool.data_ptr(), table.data_ptr(), seq_lens.data_ptr(), ids, ks, vs, N, slots, width, 16 * U, H,
                  unit // 18)
    return c, device, H, unit // 18


def _num_seqs(cu_seqlens):
    if not isinstance(cu_seqlens, torch.Tensor):
        raise TypeError("cu_seqlens must be a torch.Tensor")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must hold num_seqs + 1 >= 2 offsets")
    return cu_seqlens.shape[0] - 1


def fa_kv4_append(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, pool: torch.Tensor,
                  table: torch.Tensor, seq_lens: torch.Tensor, seq_ids: torch.Tensor | None = None,
                  k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None, stream=None) -> None:
    """Quantise packed rows k, v [T,Hkv,D] bf16 into the cache: the rows
    [cu_seqlens[s], cu_seqlens[s+1]) become the last positions of sequence s
    (slot seq_ids[s], default s), which seq_lens already counts."""
    if stream is not None:
        return _on_stream(stream, pool, fa_kv4_append, k, v, cu_seqlens, pool, table, seq_lens, seq_ids, k_scale,
                          v_scale)
    n = _num_seqs(cu_seqlens)
    c, device, H, D = _kv4(pool, table, seq_lens, seq_ids, k_scale, v_scale, n)
    _want(k, "k", torch.bfloat16, 3, device)
    _want(v, "v", torch.bfloat16, 3, device)
    _want(cu_seqlens, "cu_seqlens", torch.int32, 1, device)
    if k.shape != v.shape or k.shape[1:] != (H, D):
        raise ValueError(f"shape mismatch: k {tuple(k.shape)} v {tuple(v.shape)}, cache of {H} heads of {D}")
    lib = _lib or load_library()
    st = _on_device(device, lib.fa_kv4_append, k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), n, k.shape[0], c,
                    _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, "fa_kv4_append")


def fa_kv4_read(cu_seqlens: torch.Tensor, total: int, pool: torch.Tensor, table: torch.Tensor,
                seq_lens: torch.Tensor, seq_ids: torch.Tensor | None = None, k_scale: torch.Tensor | None = None,
                v_scale: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                v_out: torch.Tensor | None = None, stream=None):
    """The last cu_seqlens[s+1] - cu_seqlens[s] positions of each sequence as
    packed bf16 rows (k, v), each [total,Hkv,D]: a cached prefix as the keys
    of fa_fwd_varlen.  Rows behind the last sequence are left as they were."""
    if stream is not None:
        return _on_stream(stream, pool, fa_kv4_read, cu_seqlens, total, pool, table, seq_lens, seq_ids, k_scale,
                          v_scale, k_out, v_out)
    n = _num_seqs(cu_seqlens)
    c, device, H, D = _kv4(pool, table, seq_lens, seq_ids, k_scale, v_scale, n)
    _want(cu_seqlens, "cu_seqlens", torch.int32, 1, device)
    shape = (int(total), H, D)
    if shape[0] < 0:
        raise ValueError("total must not be negative")
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=pool.device)
    else:
        _want(k_out, "k_out", torch.bfloat16, 3, device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=pool.device)
    else:
        _want(v_out, "v_out", torch.bfloat16, 3, device)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"k_out and v_out must be {shape}, got {tuple(k_out.shape)} and {tuple(v_out.shape)}")
    lib = _lib or load_library()
    st = _on_device(device, lib.fa_kv4_read, k_out.data_ptr(), v_out.data_ptr(), cu_seqlens.data_ptr(), n, shape[0], c,
                    _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, "fa_kv4_read")
    return k_out, v_out


def kv4_workspace(B: int, Hq: int, Hkv: int, Lq: int, D: int) -> int:
    """Workspace bytes fa_fwd_kv4 needs on the current device."""
    nbytes = ctypes.c_size_t(0)
    st = load_library().fa_fwd_kv4_workspace(B, Hq, Hkv, Lq, D, ctypes.byref(nbytes))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_kv4_workspace")
    return nbytes.value


def fa_fwd_kv4(q: torch.Tensor, pool: torch.Tensor, table: torch.Tensor, seq_lens: torch.Tensor,
               causal: bool = False, softmax_scale: float | None = None, seq_ids: torch.Tensor | None = None,
               k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None):
    """Decode attention over a 4-bit paged cache.  q [B,Hq,Lq,D] bf16 CUDA with
    (Hq/Hkv)*Lq <= 64; sequence b is slot seq_ids[b] (default b) and attends its
    first seq_lens positions; with ``causal`` the queries are the last Lq of
    them.  Returns (o [B,Hq,Lq,D] fp32, lse [B,Hq,Lq] fp32)."""
    if stream is not None:
        return _on_stream(stream, pool, fa_fwd_kv4, q, pool, table, seq_lens, causal, softmax_scale, seq_ids,
                          k_scale, v_scale, out, lse, workspace=workspace)
    if not (isinstance(q, torch.Tensor) and q.dtype is torch.bfloat16 and q.dim() == 4 and q.is_contiguous() and q.is_cuda):
        _check_tensor(q, "q", torch.bfloat16, 4)
    B, Hq, Lq, D = q.shape
    c, device, H, cache_d = _kv4(pool, table, seq_lens, seq_ids, k_scale, v_scale, B)
    if D != cache_d:
        raise ValueError(f"q has head dimension {D} and the cache {cache_d}")
    if q.get_device() != device:
        raise ValueError(f"q must be on {pool.device}, got {q.device}")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    else:
        _want(out, "out", torch.float32, 4, device)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    else:
        _want(lse, "lse", torch.float32, 3, device)
    if out.shape != q.shape or lse.shape != (B, Hq, Lq):
        raise ValueError("out/lse shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = _lib or load_library()
    nbytes = _attn_workspace(device, Hq, H, Lq, D)
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {q.device}, got {workspace.device}")
    st = _on_device(device, lib.fa_fwd_kv4, q.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Lq,
                    1 if causal else 0, softmax_scale, c, workspace.data_ptr(), nbytes, _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_kv4")
    return out, lse


@functools.lru_cache(maxsize=256)
def _attn_workspace(device, Hq, Hkv, Lq, D):
    """kv4_workspace on device `device`."""
    return _on_device(device, kv4_workspace, 1, Hq, Hkv, Lq, D)


@functools.lru_cache(maxsize=256)
def kv4_pages_workspace(num_pages: int, n: int = 0) -> int:
    """Workspace bytes fa_kv4_reserve, fa_kv4_fork (both above 2048 sequences) and fa_kv4_compact (n = 0) need."""
    nbytes = ctypes.c_size_t(0)
    st = load_library().fa_kv4_pages_workspace(num_pages, n, ctypes.byref(nbytes))
    if st != FA_OK:
        raise FAError(st, "fa_kv4_pages_workspace")
    return nbytes.value


def _slots_of(table, seq_lens, device):
    """Shape of a call's table, after the checks of _check_slots."""
    if not (isinstance(table, torch.Tensor) and isinstance(seq_lens, torch.Tensor)
            and table.dtype is torch.int32 and table.dim() == 2 and table.is_contiguous() and table.get_device() == device
            and seq_lens.dtype is torch.int32 and seq_lens.dim() == 1 and seq_lens.is_contiguous()
            and seq_lens.get_device() == device and seq_lens.shape[0] == table.shape[0]):
        _check_slots(table, seq_lens, device)
    return table.shape


def _refs_device(refs):
    if not (isinstance(refs, torch.Tensor) and refs.dtype is torch.int32 and refs.dim() == 1 and refs.is_cuda and refs.is_contiguous()):
        _check_tensor(refs, "refs", torch.int32, 1)
    return refs.get_device()


def _page_call(name, pool, page_size, table, seq_lens, refs, first, second, n, info, workspace, device):
    """Runs one page operation.  first, second: device addresses of its lists
    of n entries (None: the operation has no such list)."""
    slots, width = _slots_of(table, seq_lens, device)
    N = refs.shape[0]
    if page_size is not None:  # a call on the tables alone
        pages = _pack_pages(0, table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(), N, slots, width,
                            int(page_size), 1, 64, 1)
    else:
        if not (isinstance(pool, torch.Tensor) and pool.dtype is torch.uint8 and pool.dim() in (4, 5) and pool.is_contiguous()
                and pool.shape[-1] in _KV4_UNITS and pool.shape[-2] in _KV4_PAGES):
            _check_pool(pool, 5 if isinstance(pool, torch.Tensor) and pool.dim() == 5 else 4)
        P, H, U, unit = pool.shape[-4:]
        if P != N:
            raise ValueError(f"pool has {P} pages and refs {N}")
        if pool.get_device() != device:
            raise ValueError(f"pool must be on cuda:{device}, got {pool.device}")
        pages = _pack_pages(pool.data_ptr(), table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(), N, slots, width,
                            16 * U, H, unit // 18, pool.shape[0] if pool.dim() == 5 else 1)
    lib = _lib or load_library()
    if name == "fa_kv4_release":
        st = _on_device(device, lib.fa_kv4_release, first, n, pages, _raw_stream(device))
    else:
        nbytes = 0 if 0 < n <= KV4_SEQS_WITHOUT_WORKSPACE else kv4_pages_workspace(N, n)
        if info is None:
            info = torch.empty(2, dtype=torch.int32, device=refs.device)
        else:
            _want(info, "info", torch.int32, 1, device)
            if info.shape[0] != 2:
                raise ValueError("info must hold 2 numbers")
        if workspace is not None and (workspace.get_device() != device or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous and on {refs.device}, got {workspace.device}")
        if nbytes and (workspace is None or workspace.numel() * workspace.element_size() < nbytes):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=refs.device)
        tail = (pages, info.data_ptr(), workspace.data_ptr() if nbytes else None, nbytes, _raw_stream(device))
        if name == "fa_kv4_compact":
            st = _on_device(device, lib.fa_kv4_compact, *tail)
        else:
            st = _on_device(device, getattr(lib, name), first, second, n, *tail)
    if st != FA_OK:
        raise FAError(st, name)
    return info


def fa_kv4_reserve(new_tokens: torch.Tensor, table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor,
                   page_size: int, seq_ids: torch.Tensor | None = None, info: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Give slot seq_ids[i] (default i) pages for new_tokens[i] more positions and
    count them in seq_lens, or take its last -new_tokens[i] positions back where
    that is negative (rejected drafts).  Returns info, int32 [2] on the device: free pages
    left, and 0, or the pages that were missing (then nothing was changed), or
    -1 for bad arguments on the device."""
    if stream is not None:
        return _on_stream(stream, refs, fa_kv4_reserve, new_tokens, table, seq_lens, refs, page_size, seq_ids, info,
                          workspace=workspace)
    device = _refs_device(refs)
    _want(new_tokens, "new_tokens", torch.int32, 1, device)
    n = new_tokens.shape[0]
    if seq_ids is not None:
        _want(seq_ids, "seq_ids", torch.int32, 1, device)
        if seq_ids.shape[0] != n:
            raise ValueError(f"seq_ids must name {n} slots")
    return _page_call("fa_kv4_reserve", None, page_size, table, seq_lens, refs,
                      None if seq_ids is None else seq_ids.data_ptr(), new_tokens.data_ptr(), n, info, workspace, device)


def fa_kv4_fork(parents: torch.Tensor, children: torch.Tensor, pool: torch.Tensor, table: torch.Tensor,
                seq_lens: torch.Tensor, refs: torch.Tensor, info: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Make the empty slots children[i] copies of the slots parents[i]: full pages
    are shared, a partly filled last page is copied.  pool as for
    fa_kv4_append, or with the layers in front.  Returns info as fa_kv4_reserve."""
    if stream is not None:
        return _on_stream(stream, refs, fa_kv4_fork, parents, children, pool, table, seq_lens, refs, info,
                          workspace=workspace)
    device = _refs_device(refs)
    _want(parents, "parents", torch.int32, 1, device)
    _want(children, "children", torch.int32, 1, device)
    n = parents.shape[0]
    if children.shape[0] != n:
        raise ValueError(f"{n} parents but {children.shape[0]} children")
    return _page_call("fa_kv4_fork", pool, None, table, seq_lens, refs, parents.data_ptr(), children.data_ptr(), n,
                      info, workspace, device)


def fa_kv4_release(seq_ids: torch.Tensor, table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor,
                   page_size: int, stream=None) -> None:
    """Free the slots seq_ids: their pages lose a reference each, their lengths become 0."""
    if stream is not None:
        return _on_stream(stream, refs, fa_kv4_release, seq_ids, table, seq_lens, refs, page_size)
    device = _refs_device(refs)
    _want(seq_ids, "seq_ids", torch.int32, 1, device)
    _page_call("fa_kv4_release", None, page_size, table, seq_lens, refs, seq_ids.data_ptr(), None, seq_ids.shape[0],
               None, None, device)


def fa_kv4_compact(pool: torch.Tensor, table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor,
                   info: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Move the pages in use to the front of the pool (of every layer).  Returns info as fa_kv4_reserve."""
    if stream is not None:
        return _on_stream(stream, refs, fa_kv4_compact, pool, table, seq_lens, refs, info, workspace=workspace)
    return _page_call("fa_kv4_compact", pool, None, table, seq_lens, refs, None, None, 0, info, workspace,
                      _refs_device(refs))


# ------------------------------------------------------------- rotary positions and the 16-bit cache

_pack_rope = struct.Struct("Piiif").pack       # struct fa_rope
_pack_rows = struct.Struct("2P6qi4x").pack     # struct fa_rotary_rows
_pack_kv16 = struct.Struct("4P6i").pack        # struct fa_kv16
_PER_TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667344")  # 1 / (2 pi)


class RopePlan:
    """Frequencies of rotary positions on a device and how they are applied (see rope_plan)."""

    __slots__ = ("freqs", "rot_dim", "start", "end", "interleaved", "mscale", "device", "packed")

    def __init__(self, freqs, start, interleaved, mscale):
        """freqs: int64 [rot_dim / 2], turns per position times 2^64 modulo 2^64."""
        _check_tensor(freqs, "freqs", torch.int64, 1, on_device=False)
        if freqs.numel() == 0 or freqs.numel() % 8:
            raise ValueError(f"freqs must hold rot_dim / 2 frequencies, a multiple of 8, got {freqs.numel()}")
        if start < 0 or start % 16:
            raise ValueError(f"start must be a multiple of 16, got {start}")
        if not mscale > 0 or math.isinf(mscale):
            raise ValueError(f"mscale must be positive and finite, got {mscale}")
        rot_dim, start, interleaved, mscale = 2 * freqs.numel(), int(start), bool(interleaved), float(mscale)
        packed = _pack_rope(freqs.data_ptr(), rot_dim, start, interleaved, mscale)
        for name, value in (("freqs", freqs), ("rot_dim", rot_dim), ("start", start), ("end", start + rot_dim),
                            ("interleaved", interleaved), ("mscale", mscale), ("packed", packed),
                            ("device", freqs.get_device())):  # -1: not on a GPU
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):  # calls take what is packed
        raise AttributeError(f"a RopePlan stays as it was made: make another for another {name}")

    def __delattr__(self, name):
        raise AttributeError("a RopePlan stays as it was made")

    def __reduce__(self):  # a copy packs the address of its own frequencies
        return RopePlan, (self.freqs, self.start, self.interleaved, self.mscale)


def rope_plan(rot_dim: int | None = None, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
              original_length: int | None = None, inv_freq=None, mscale: float | None = None, start: int = 0,
              interleaved: bool = False, device="cuda") -> RopePlan:
    """The frequencies that fa_rope and fa_kv16_append take.  Pair c < rot_dim / 2 turns by w_c a position, w_c =
    base ** (-2 c / rot_dim); it is made of dimensions start + c and start + c + rot_dim / 2, or with ``interleaved``
    of start + 2 c and the next.  For a context stretched by ``factor``, ``scaling`` is

    "linear"  w_c / factor,
    "base"    the base times factor ** (rot_dim / (rot_dim - 2)),
    "parts"   w_c / factor where a pair turns less than once in ``original_length`` positions, w_c where it turns more
              than 32 times, linear in the turns between; and mscale 0.1 ln(factor) + 1 where none is given.

    ``inv_freq`` (rot_dim / 2 numbers or a tensor, radians a position) replaces all that.  ``mscale`` multiplies the
    turned dimensions (default 1).  Frequencies are kept to 2^-64 of a turn, so angles are exact at any position."""
    if inv_freq is None:
        if rot_dim is None or rot_dim <= 0 or rot_dim % 16:
            raise ValueError(f"rot_dim must be a positive multiple of 16, got {rot_dim}")
        if not base > 0 or not factor > 0 or math.isinf(base) or math.isinf(factor):
            raise ValueError(f"base and factor must be positive and finite, got {base} and {factor}")
        if scaling == "base":
            base = base * factor ** (rot_dim / (rot_dim - 2))
        w = [base ** (-2.0 * c / rot_dim) for c in range(rot_dim // 2)]
        if scaling == "linear":
            w = [x / factor for x in w]
        elif scaling == "parts":
            if not original_length or original_length <= 0:
                raise ValueError("scaling 'parts' needs original_length")
            own = [min(1.0, max(0.0, (original_length * x / (2 * math.pi) - 1) / 31)) for x in w]
            w = [x * a + x / factor * (1 - a) for x, a in zip(w, own)]
            mscale = 0.1 * math.log(factor) + 1.0 if mscale is None else mscale
        elif scaling not in (None, "base"):
            raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
    else:
        if scaling is not None or factor != 1.0 or original_length is not None:
            raise ValueError("inv_freq replaces scaling, factor and original_length")
        w = [float(x) for x in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq)]
        if not w or len(w) % 8 or (rot_dim is not None and rot_dim != 2 * len(w)):
            raise ValueError(f"inv_freq must hold rot_dim / 2 frequencies, a multiple of 8, got {len(w)}")
    if not all(math.isfinite(x) for x in w):
        raise ValueError("frequencies must be finite")
    mscale = 1.0 if mscale is None else float(mscale)
    turns = [round(Fraction(x) * _PER_TURN * 2 ** 64) % 2 ** 64 for x in w]
    freqs = torch.tensor([x - 2 ** 64 if x >> 63 else x for x in turns], dtype=torch.int64).to(device)
    return RopePlan(freqs, start, interleaved, mscale)


_ROPE_TYPES = (torch.bfloat16, torch.float32)


def _check_rows(t, name, ndim, dtype, device):
    """Rows [..., D] of `dtype` on `device` whose D elements are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{max(device, 0)}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows, got strides {t.stride()}")


def _check_out(out, x, name, dtype):
    """`out` for the turned rows of x: a contiguous tensor, or x itself."""
    _check_rows(out, name, x.dim(), dtype, x.get_device())
    if out.shape != x.shape:
        raise ValueError(f"{name} must be {tuple(x.shape)}, got {tuple(out.shape)}")
    if out.data_ptr() == x.data_ptr() and out.dtype is x.dtype:
        if out.stride() != x.stride():
            raise ValueError(f"{name} in place must have its input's strides {x.stride()}, got {out.stride()}")
    elif not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous, or the input itself")


def _rows_of(x, y, heads):
    """struct fa_rotary_rows of packed rows x [T, heads, D] (and y, or None)."""
    a0, a1, _ = x.stride()
    if y is None:
        return _pack_rows(x.data_ptr(), 0, 0, a0, a1, 0, 0, 0, heads)
    b0, b1, _ = y.stride()
    return _pack_rows(x.data_ptr(), y.data_ptr(), 0, a0, a1, 0, b0, b1, heads)


def _dense_rows_of(x, y, heads):
    """struct fa_rotary_rows of rows x and y [B, heads, L, D]."""
    (a0, a1, a2, _), (b0, b1, b2, _) = x.stride(), y.stride()
    return _pack_rows(x.data_ptr(), y.data_ptr(), a0, a2, a1, b0, b2, b1, heads)


def _refuse_rows(q, rope):
    """Says what is wrong with the q or the rope of a rotary call, if anything is."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() not in (3, 4):
        raise ValueError(f"q must be [T, H, D] or [B, H, L, D], got shape {tuple(q.shape)}")
    if q.dtype not in _ROPE_TYPES:
        raise TypeError(f"q must be bfloat16 or float32, got {q.dtype}")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    _check_rows(q, "q", q.dim(), q.dtype, q.get_device())
    if not isinstance(rope, RopePlan):
        raise TypeError("rope must be a RopePlan (rope_plan)")
    if rope.device != q.get_device():
        raise ValueError(f"rope must be on {q.device}, got cuda:{rope.device}")
    if rope.end > q.shape[-1]:
        raise ValueError(f"rope turns dimensions {rope.start} to {rope.end} of {q.shape[-1]}")


def _rope_call(backward, q, k, rope, positions, dtype, q_out, k_out):
    if not (isinstance(q, torch.Tensor) and isinstance(rope, RopePlan)):
        _refuse_rows(q, rope)
    device, kind, shape = q.get_device(), q.dtype, q.shape
    if len(shape) == 3:
        B, (T, Hq, D), dense, pack = 1, shape, False, _rows_of
    elif len(shape) == 4:
        (B, Hq, T, D), dense, pack = shape, True, _dense_rows_of
    else:
        return _refuse_rows(q, rope)
    if kind not in _ROPE_TYPES or device < 0 or q.stride(-1) != 1 or rope.device != device or rope.end > D:
        _refuse_rows(q, rope)
    to = dtype or kind
    if to is not kind and (to not in _ROPE_TYPES or kind is torch.bfloat16):
        raise TypeError(f"rows of {kind} can not become {to}")
    rows_k = None
    if k is not None:
        if not (isinstance(k, torch.Tensor) and k.dtype is kind and k.get_device() == device and k.dim() == len(shape)
                and k.stride(-1) == 1):
            _check_rows(k, "k", len(shape), kind, device)
        Hk = k.shape[1]
        if k.shape != ((B, Hk, T, D) if dense else (T, Hk, D)):
            raise ValueError(f"shape mismatch: q {tuple(shape)} k {tuple(k.shape)}")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=to, device=k.device)
        else:
            _check_out(k_out, k, "k_out", to)
        if Hk:
            rows_k = pack(k, k_out, Hk)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_out is None:
        q_out = torch.empty(shape, dtype=to, device=q.device)
    else:
        _check_out(q_out, q, "q_out", to)
    at, step = None, 0
    if positions is not None:
        if not (isinstance(positions, torch.Tensor) and positions.dtype is torch.int32 and positions.get_device() == device
                and positions.is_contiguous()):
            _want(positions, "positions", torch.int32, positions.dim() if isinstance(positions, torch.Tensor) else 1, device)
        if positions.shape != (T,):
            if positions.shape != (B, T) or not dense:
                raise ValueError(f"positions must be {(T,)}{f' or {(B, T)}' if dense else ''}, got {tuple(positions.shape)}")
            step = T
        at = positions.data_ptr() or None
    lib = _lib or load_library()
    fp32 = kind is torch.float32
    st = _on_device(device, lib.fa_rope_bwd if backward else lib.fa_rope, pack(q, q_out, Hq), rows_k, B, T, D, fp32,
                    fp32 and to is kind, rope.packed, at, step, _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, "fa_rope_bwd" if backward else "fa_rope")
    return q_out, k_out


def fa_rope(q: torch.Tensor, k: torch.Tensor | None, rope: RopePlan, positions: torch.Tensor | None = None,
            dtype: torch.dtype | None = None, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
            stream=None):
    """Turn the rows of q and k (which may be None) by their positions' angles.  q, k: packed [T,H,D] or dense
    [B,H,L,D], bf16 or fp32, of any strides with contiguous rows (views of a fused projection, or of [B,L,H,D]);
    positions int32 [T], [L] or [B,L] (default: the index along the tokens; packed rows of several sequences need
    theirs, as the call does not know where one begins).  Returns (q_out, k_out), contiguous, of ``dtype`` (default: the
    input's; fp32 rows may become bf16).  q_out may be q itself, and k_out k, but neither the other's."""
    if stream is not None:
        return _on_stream(stream, q, fa_rope, q, k, rope, positions, dtype, q_out, k_out)
    return _rope_call(False, q, k, rope, positions, dtype, q_out, k_out)


def fa_rope_bwd(dq: torch.Tensor, dk: torch.Tensor | None, rope: RopePlan, positions: torch.Tensor | None = None,
                dtype: torch.dtype | None = None, dq_out: torch.Tensor | None = None,
                dk_out: torch.Tensor | None = None, stream=None):
    """Backward of fa_rope: from the gradients of its outputs (fa_bwd's fp32 dq and dk, or bf16) those of its inputs.
    Arguments as fa_rope.  Returns (dq_out, dk_out)."""
    if stream is not None:
        return _on_stream(stream, dq, fa_rope_bwd, dq, dk, rope, positions, dtype, dq_out, dk_out)
    return _rope_call(True, dq, dk, rope, positions, dtype, dq_out, dk_out)


def kv16_pool(num_pages: int, Hkv: int, page_size: int, D: int, layers: int | None = None,
              device="cuda") -> torch.Tensor:
    """An empty (all zero) pool of a paged bf16 KV cache: [num_pages, 2, Hkv, page_size, D], K then V, with ``layers`` in
    front when given."""
    if page_size not in (16, 32, 64, 128, 256) or D not in (64, 128):
        raise ValueError("page_size must be 16, 32, 64, 128 or 256 and D 64 or 128")
    shape = (num_pages, 2, Hkv, page_size, D)
    return torch.zeros(shape if layers is None else (layers, *shape), dtype=torch.bfloat16, device=device)


def draft_mask(parents, cu_seqlens) -> tuple[torch.Tensor, torch.Tensor]:
    """The mask of fa_fwd_kv16, int32 [T, words], and the depths, int32 [T], of drafted trees, on the host: parents[i]
    is the parent of packed node i, an index in its own sequence in front of i's, or -1 for a child of the prefix's
    last position.  A node sees its ancestors and itself; its position is the prefix length plus its depth."""
    parents = parents.tolist() if isinstance(parents, torch.Tensor) else list(parents)
    cu = cu_seqlens.tolist() if isinstance(cu_seqlens, torch.Tensor) else list(cu_seqlens)
    if len(cu) < 2 or cu[0] != 0 or any(b < a for a, b in zip(cu, cu[1:])) or cu[-1] > len(parents):
        raise ValueError("cu_seqlens must hold num_seqs + 1 >= 2 offsets of the nodes, from 0, not decreasing")
    words = max(1, -(-max(b - a for a, b in zip(cu, cu[1:])) // 32))
    seen, depth = [0] * len(parents), [0] * len(parents)
    for a, b in zip(cu, cu[1:]):
        for i in range(a, b):
            p = parents[i]
            if not -1 <= p < i - a:
                raise ValueError(f"node {i - a} of a sequence has parent {p}")
            seen[i] = (seen[a + p] if p >= 0 else 0) | 1 << (i - a)
            depth[i] = depth[a + p] + 1 if p >= 0 else 0
    bits = b"".join(x.to_bytes(4 * words, "little") for x in seen)
    mask = torch.frombuffer(bytearray(bits or b"0000"), dtype=torch.int32)[:words * len(parents)]
    return mask.reshape(len(parents), words).clone(), torch.tensor(depth, dtype=torch.int32)


def _kv16(pool, table, seq_lens, seq_ids, cu_seqlens, layers=False):
    """Checks the cache of a call and its packed sequences.  Returns (fa_kv16_t as bytes, device index, sequences, Hkv,
    D)."""
    if not (isinstance(pool, torch.Tensor) and isinstance(table, torch.Tensor) and isinstance(seq_lens, torch.Tensor)
            and isinstance(cu_seqlens, torch.Tensor)):
        for t, name in ((pool, "pool"), (table, "table"), (seq_lens, "seq_lens"), (cu_seqlens, "cu_seqlens")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
    device, shape, i32 = pool.get_device(), pool.shape, torch.int32
    if not (device >= 0 and pool.dtype is torch.bfloat16 and (len(shape) == 5 or len(shape) == 6 and layers)
            and pool.is_contiguous() and table.dtype is i32 and table.dim() == 2 and table.get_device() == device
            and table.is_contiguous() and seq_lens.dtype is i32 and seq_lens.dim() == 1 and seq_lens.get_device() == device
            and seq_lens.is_contiguous() and cu_seqlens.dtype is i32 and cu_seqlens.dim() == 1
            and cu_seqlens.get_device() == device and cu_seqlens.is_contiguous()):
        _check_tensor(pool, "pool", torch.bfloat16, 6 if layers and len(shape) == 6 else 5)
        _check_slots(table, seq_lens, device)
        _want(cu_seqlens, "cu_seqlens", i32, 1, device)
    n = cu_seqlens.shape[0] - 1
    slots, width = table.shape
    N, two, H, P, D = shape[-5:] if layers else shape
    if two != 2 or P not in (16, 32, 64, 128, 256) or D not in (64, 128):
        raise ValueError(f"pool must be bfloat16 [..., pages, 2, Hkv, page_size, D], got {tuple(shape)}")
    if n < 1:
        raise ValueError("cu_seqlens must hold num_seqs + 1 >= 2 offsets")
    if seq_lens.shape[0] != slots:
        raise ValueError(f"table has {slots} slots and seq_lens {seq_lens.shape[0]}")
    ids = 0
    if seq_ids is not None:
        _want(seq_ids, "seq_ids", i32, 1, device)
        if seq_ids.shape[0] != n:
            raise ValueError(f"seq_ids must name {n} slots")
        ids = seq_ids.data_ptr()
    elif n > slots:
        raise ValueError(f"{n} sequences but {slots} slots")
    return (_pack_kv16(pool.data_ptr(), table.data_ptr(), seq_lens.data_ptr(), ids, N, slots, width, P, H, D), device, n, H,
            D)


def fa_kv16_append(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, pool: torch.Tensor,
                   table: torch.Tensor, seq_lens: torch.Tensor, seq_ids: torch.Tensor | None = None,
                   rope: RopePlan | None = None, positions: torch.Tensor | None = None,
                   q: torch.Tensor | None = None, q_out: torch.Tensor | None = None, stream=None):
    """Write packed rows k, v [T,Hkv,D] bf16 (of any strides with contiguous rows) into the cache, k turned by
    ``rope``: the rows [cu_seqlens[s], cu_seqlens[s+1]) become the last positions of sequence s (slot seq_ids[s],
    default s), which seq_lens already counts.  positions int32 [T] (default: the index in the cache).  q [T,Hq,D] is
    turned alike; returns q_out (a new tensor, or q itself where given so), or None without q.  Rows of q behind the
    last sequence are not written."""
    if stream is not None:
        return _on_stream(stream, pool, fa_kv16_append, k, v, cu_seqlens, pool, table, seq_lens, seq_ids, rope,
                          positions, q, q_out)
    c, device, n, H, D = _kv16(pool, table, seq_lens, seq_ids, cu_seqlens)
    bf16 = torch.bfloat16
    for t, name in ((k, "k"), (v, "v")):
        if not (isinstance(t, torch.Tensor) and t.dtype is bf16 and t.dim() == 3 and t.get_device() == device and t.stride(2) == 1):
            _check_rows(t, name, 3, bf16, device)
    T = k.shape[0]
    if k.shape != (T, H, D) or v.shape != (T, H, D):
        raise ValueError(f"shape mismatch: k {tuple(k.shape)} v {tuple(v.shape)}, cache of {H} heads of {D}")
    packed = None
    if rope is not None:
        if not isinstance(rope, RopePlan):
            raise TypeError("rope must be a RopePlan (rope_plan)")
        if rope.device != device or rope.end > D:
            raise ValueError(f"rope must be on {pool.device} and turn at most {D} dimensions")
        packed = rope.packed
    elif q is not None or positions is not None:
        raise ValueError("q and positions need rope")
    rows_q = None
    if q is not None:
        if not (isinstance(q, torch.Tensor) and q.dtype is bf16 and q.dim() == 3 and q.get_device() == device and q.stride(2) == 1):
            _check_rows(q, "q", 3, bf16, device)
        Tq, Hq, Dq = q.shape
        if Tq != T or Dq != D:
            raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)}")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=bf16, device=q.device)
        else:
            _check_out(q_out, q, "q_out", bf16)
        if Hq:
            rows_q = _rows_of(q, q_out, Hq)
    elif q_out is not None:
        raise ValueError("q_out without q")
    at = None
    if positions is not None:
        _want(positions, "positions", torch.int32, 1, device)
        if positions.shape[0] != T:
            raise ValueError(f"positions must hold {T} numbers, got {positions.shape[0]}")
        at = positions.data_ptr() or None
    lib = _lib or load_library()
    st = _on_device(device, lib.fa_kv16_append, rows_q, _rows_of(k, None, H), _rows_of(v, None, H),
                    cu_seqlens.data_ptr(), n, T, c, packed, at, _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, "fa_kv16_append")
    return q_out


def kv16_workspace(total: int, Hq: int, Hkv: int, D: int) -> int:
    """Workspace bytes fa_fwd_kv16 needs on the current device."""
    nbytes = ctypes.c_size_t(0)
    st = load_library().fa_fwd_kv16_workspace(total, Hq, Hkv, D, ctypes.byref(nbytes))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_kv16_workspace")
    return nbytes.value


@functools.lru_cache(maxsize=1024)
def _kv16_workspace(device, total, Hq, Hkv, D):
    """kv16_workspace on device `device`."""
    return _on_device(device, kv16_workspace, total, Hq, Hkv, D)


def fa_fwd_kv16(q: torch.Tensor, cu_seqlens: torch.Tensor, pool: torch.Tensor, table: torch.Tensor,
                seq_lens: torch.Tensor, mask: torch.Tensor | None = None, causal: bool = False,
                softmax_scale: float | None = None, seq_ids: torch.Tensor | None = None,
                out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """Attention of packed queries q [T,Hq,D] bf16 (contiguous rows) over a paged bf16 cache: the rows
    [cu_seqlens[s], cu_seqlens[s+1]) are the last positions of sequence s (slot seq_ids[s], default s), whose keys the
    cache already holds.  They see every position in front of the call's and, of the call's own, with ``mask`` (int32
    [T,words], bit j % 32 of word j / 32 for position j of the sequence's rows; draft_mask) the marked ones, with
    ``causal`` those up to their own, else all.  Returns (o [T,Hq,D] bf16, lse [Hq,T] fp32); rows behind the last
    sequence are left as they were."""
    if stream is not None:
        return _on_stream(stream, pool, fa_fwd_kv16, q, cu_seqlens, pool, table, seq_lens, mask, causal, softmax_scale,
                          seq_ids, out, lse, workspace=workspace)
    c, device, n, H, D = _kv16(pool, table, seq_lens, seq_ids, cu_seqlens)
    if not (isinstance(q, torch.Tensor) and q.dtype is torch.bfloat16 and q.dim() == 3 and q.get_device() == device
            and q.stride(2) == 1):
        _check_rows(q, "q", 3, torch.bfloat16, device)
    T, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError(f"q has head dimension {Dq} and the cache {D}")
    if Hq % H or not Hq:
        raise ValueError(f"{Hq} query heads over {H} KV heads")
    words, bits = 0, None
    if mask is not None:
        _want(mask, "mask", torch.int32, 2, device)
        rows, words = mask.shape
        if rows != T or words < 1:
            raise ValueError(f"mask must be [{T}, words], got {tuple(mask.shape)}")
        if causal:
            raise ValueError("mask and causal exclude each other")
        bits = mask.data_ptr()
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    else:
        _want(out, "out", torch.bfloat16, 3, device)
        if out.shape != q.shape:
            raise ValueError("out shape mismatch")
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    else:
        _want(lse, "lse", torch.float32, 2, device)
        if lse.shape != (Hq, T):
            raise ValueError("lse shape mismatch")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    lib = _lib or load_library()
    nbytes = _kv16_workspace(device, min(T, 129), Hq, H, D)  # more tokens need no more
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {q.device}, got {workspace.device}")
    step, head, _ = q.stride()
    st = _on_device(device, lib.fa_fwd_kv16, q.data_ptr(), step, head, out.data_ptr(), lse.data_ptr(),
                    cu_seqlens.data_ptr(), n, T, Hq, bits, words, 1 if causal else 0, softmax_scale, c, workspace.data_ptr(), nbytes, _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_kv16")
    return out, lse


def fa_kv16_keep(keep: torch.Tensor, counts: torch.Tensor, cu_seqlens: torch.Tensor, pool: torch.Tensor,
                 table: torch.Tensor, seq_lens: torch.Tensor, seq_ids: torch.Tensor | None = None,
                 new_tokens: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Keep the accepted nodes of drafted trees: of the last cu_seqlens[s+1] - cu_seqlens[s] positions of sequence s,
    those named by keep[cu_seqlens[s] + j], j < counts[s] (int32, ascending, from 0), become the first, in order, in
    every layer of pool (as for fa_kv16_append, or with the layers in front).  Returns new_tokens, int32 [num_seqs] (a
    tensor of its own, not counts): counts[s] less the drafted ones, for fa_kv4_reserve, which takes the other positions
    back."""
    if stream is not None:
        return _on_stream(stream, pool, fa_kv16_keep, keep, counts, cu_seqlens, pool, table, seq_lens, seq_ids,
                          new_tokens)
    c, device, n, H, D = _kv16(pool, table, seq_lens, seq_ids, cu_seqlens, layers=True)
    _want(keep, "keep", torch.int32, 1, device)
    _want(counts, "counts", torch.int32, 1, device)
    if counts.shape[0] != n:
        raise ValueError(f"counts must hold {n} numbers, got {counts.shape[0]}")
    if new_tokens is None:
        new_tokens = torch.empty(n, dtype=torch.int32, device=pool.device)
    else:
        _want(new_tokens, "new_tokens", torch.int32, 1, device)
        if new_tokens.shape[0] != n:
            raise ValueError(f"new_tokens must hold {n} numbers, got {new_tokens.shape[0]}")
    lib = _lib or load_library()
    st = _on_device(device, lib.fa_kv16_keep, keep.data_ptr() or counts.data_ptr(), counts.data_ptr(),
                    cu_seqlens.data_ptr(), n, keep.shape[0], pool.shape[0] if pool.dim() == 6 else 1,
                    new_tokens.data_ptr(), c, _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, "fa_kv16_keep")
    return new_tokens


def fa_check(stream=None) -> int:
    """Synchronise the stream and raise if a kernel latched an error."""
    st = load_library().fa_check(_stream_handle(stream))
    if st != FA_OK:
        raise FAError(st, "fa_check")
    return st
