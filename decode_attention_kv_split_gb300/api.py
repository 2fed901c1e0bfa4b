"""Python binding over libdecode_attn.so (ctypes; argument marshalling only).

Every step of the computation runs in the library's CUDA kernels.  This
module checks tensor shapes/dtypes/devices, takes raw device pointers and the
current CUDA stream from PyTorch, allocates the split workspace with PyTorch,
and calls the C entry points of the same names.  There is no CPU fallback:
if the shared library is missing the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdecode_attn.so")

DA_FP32 = 0
DA_BF16 = 1
DA_INT8 = 2          # 8-bit caches: one-byte codes + a float32 scale per cached row
DA_FP8_E4M3 = 3
DA_OUT_BF16 = 0x100  # dtype flag: out is bfloat16
DA_BF16_WEIGHTS = 0x400  # dtype flag of chunk_attn and decode_attn_shared: weights as one bfloat16
DEVERR_SEQ_LEN = 1
DEVERR_POS = 2
DEVERR_TIMEOUT = 4
DEVERR_BOUNDS = 8    # set only by the bounds-checked test build
DEVERR_VALUE = 16    # a NaN or infinity among rows to quantise

_DTYPES = {torch.float32: DA_FP32, torch.bfloat16: DA_BF16}
# 8-bit caches are passed as torch.int8 / torch.float8_e4m3fn tensors of codes
_Q8_DTYPES = {torch.int8: DA_INT8, torch.float8_e4m3fn: DA_FP8_E4M3}
_ALL_DTYPES = {**_DTYPES, **_Q8_DTYPES}

_lock = threading.Lock()
_lib = None

# Every entry point of include/decode_attn.h with its ctypes signature.
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
SIGNATURES = {
    "decode_attn_resolve_splits": (_I, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "decode_attn_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    "decode_attn_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P, _P]),
    "decode_attn": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "decode_attn_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I,
                                _P, _SZ, _P, _P]),
    "decode_attn_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _P]),
    "kv_append": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "decode_attn_status_string": (ctypes.c_char_p, [_I]),
    "decode_attn_last_cuda_error": (ctypes.c_char_p, []),
    "decode_attn_launch_count": (ctypes.c_uint64, []),
    "decode_attn_q8_ex": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P,
                               _SZ, _P, _P]),
    "decode_attn_q8_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                   _I, _I, _F, _I, _I, _P, _SZ, _P, _P]),
    "kv_append_q8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "kv_quantize": (_I, [_P, _I, _P, _P, ctypes.c_longlong, _I, _I, _P]),
    "decode_attn_partial": (_I, [_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I,
                                 _I, _P, _SZ, _P, _P]),
    "decode_attn_combine": (_I, [_P, _P, _I, _P, _P, _I, _I, _I, _I, _P]),
    "decode_attn_mod_workspace_bytes": (_SZ, [_P, _I, _I, _I, _I, _I, _I, _I, _I,
                                              ctypes.POINTER(_I)]),
    "decode_attn_mod": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ,
                             _P, _P]),
    "decode_attn_mod_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F,
                                    _I, _I, _P, _SZ, _P, _P]),
    "decode_attn_q8b_workspace_bytes": (_SZ, [_P, _I, _I, _I, _I, _I, _I, _I, _I,
                                              ctypes.POINTER(_I)]),
    "decode_attn_q8b": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I,
                             _P, _SZ, _P, _P]),
    "kv_append_q8b": (_I, [_P, _P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I,
                           _P, _P]),
    "kv_append_rope": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I,
                            _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
    "chunk_attn_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    "chunk_attn": (_I, [_P, _P, _I, _P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P,
                        _SZ, _P, _P]),
    "decode_attn_shared_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    "decode_attn_shared": (_I, [_P, _P, _P, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P,
                                _SZ, _P, _P]),
    "kv_read_q8b": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
}


class DecodeAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.decode_attn_status_string(status).decode()
        if status == -6:
            msg += ": " + lib.decode_attn_last_cuda_error().decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the shared library once; raise if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with __graft_entry__.build() "
                    "(there is no fallback implementation)")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
        return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise DecodeAttnError(status, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor, stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(s.cuda_stream)


class _on_device:
    """Make t's device current for the call (a no-op when it already is)."""

    def __init__(self, t: torch.Tensor):
        self.idx = t.device.index
        self.prev = None

    def __enter__(self):
        cur = torch.cuda.current_device()
        if self.idx is not None and cur != self.idx:
            self.prev = cur
            torch.cuda.set_device(self.idx)

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)


def _cache_dims(q, K, V, seq_lens):
    if q.dim() != 3 or K.dim() != 4 or V.dim() != 4:
        raise ValueError("expected q [B, h_q, d_k], K [B, h_kv, n_max, d_k], V [B, h_kv, n_max, d_v]")
    B, h_q, d_k = q.shape
    Bk, h_kv, n_max, d_k2 = K.shape
    Bv, h_kv2, n_max2, d_v = V.shape
    if (Bk, Bv) != (B, B) or h_kv2 != h_kv or n_max2 != n_max or d_k2 != d_k:
        raise ValueError("q, K and V shapes disagree")
    if seq_lens.shape != (B,) or seq_lens.dtype != torch.int32:
        raise ValueError("seq_lens must be an int32 tensor of shape [B]")
    for name, t in (("q", q), ("K", K), ("V", V), ("seq_lens", seq_lens)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if not (q.dtype == K.dtype == V.dtype) or q.dtype not in _DTYPES:
        raise ValueError("q, K, V must share dtype float32 or bfloat16")
    return B, h_q, h_kv, d_k, d_v, n_max


def resolve_splits(B, h_q, h_kv, d_k, d_v, n_max, dtype: torch.dtype, num_splits: int = 0) -> int:
    """Splits per (b, kv head) the library uses for this request (on the current device).
    ``dtype`` is the cache's element type (torch.int8 / torch.float8_e4m3fn: 8-bit caches)."""
    r = load().decode_attn_resolve_splits(B, h_q, h_kv, d_k, d_v, n_max, _ALL_DTYPES[dtype],
                                          num_splits)
    if r < 0:
        raise DecodeAttnError(r, "decode_attn_resolve_splits")
    return r


_ws_bytes_cache: dict = {}


def workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, dtype: torch.dtype, num_splits: int = 0) -> int:
    key = (torch.cuda.current_device(), B, h_q, h_kv, d_k, d_v, n_max, dtype, num_splits)
    hit = _ws_bytes_cache.get(key)
    if hit is not None:
        return hit
    st = ctypes.c_int(0)
    n = load().decode_attn_workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, _ALL_DTYPES[dtype],
                                           num_splits, ctypes.byref(st))
    _check(st.value, "decode_attn_workspace_bytes")
    _ws_bytes_cache[key] = int(n)
    return int(n)


_no_stream = contextlib.nullcontext()


def _on_stream(stream):
    """Allocations in the order of ``stream`` (None: the current one)."""
    return _no_stream if stream is None else torch.cuda.stream(stream)


_ws_cache: dict = {}
_ws_locks: dict = {}


def _ws_lock(key):
    """The lock of a kept workspace.  A call with splits is two launches that pass partials
    through it, and the library call drops the GIL: without the lock a call that another host
    thread makes on the same stream could come between them."""
    return _ws_locks.get(key) or _ws_locks.setdefault(key, threading.Lock())


def _out(out: torch.Tensor | None, out_dtype: torch.dtype | None, B: int, h_q: int, d_v: int,
         device: torch.device, stream) -> tuple[torch.Tensor, int]:
    """The output tensor (allocated when None, in the call's stream) and its dtype flag."""
    if out is None:
        with _on_stream(stream):
            out = torch.empty((B, h_q, d_v), dtype=out_dtype or torch.float32, device=device)
    if (out.shape != (B, h_q, d_v) or out.dtype not in (torch.float32, torch.bfloat16)
            or not out.is_contiguous() or out.device != device
            or (out_dtype is not None and out.dtype != out_dtype)):
        raise ValueError("out must be a contiguous float32 or bfloat16 tensor [B, h_q, d_v] "
                         "on the query's device")
    return out, (DA_OUT_BF16 if out.dtype == torch.bfloat16 else 0)


def _workspace(device: torch.device, nbytes: int, given: torch.Tensor | None, stream):
    """A call's workspace (the given one, or one of its stream), its bytes, and the lock to
    hold while the library is called."""
    if given is not None or nbytes == 0:
        return given, 0 if given is None else given.numel() * given.element_size(), _unlocked
    return _kept_workspace((device.index, _raw(stream, device.index)), nbytes, stream)


def _kept_workspace(key, need: int, stream):
    """A workspace of ``need`` bytes, its bytes and its lock: a tensor of the stream the call
    runs on, kept under ``key`` (the device first) for its next call; while that stream is
    captured, a tensor of the graph's own pool, since two graphs that share scratch may be
    replayed at the same time."""
    with _on_stream(stream):
        if torch._C._cuda_isCurrentStreamCapturing():
            return torch.empty(need, dtype=torch.uint8, device=key[0]), need, _unlocked
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < need:
            ws = _ws_cache[key] = torch.empty(need, dtype=torch.uint8, device=key[0])
    return ws, ws.numel(), _ws_lock(key)


_unlocked = contextlib.nullcontext()


def decode_attn(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor,
                out: torch.Tensor | None = None, scale: float | None = None, num_splits: int = 0,
                workspace: torch.Tensor | None = None, dev_error: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None,
                out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Decode attention (calls ``decode_attn_ex``); returns ``out`` [B, h_q, d_v], float32
    or bfloat16 (``out_dtype``, or the dtype of a given ``out``).

    ``scale`` defaults to 1/sqrt(d_k).  ``workspace`` (uint8 CUDA tensor) is
    allocated and cached per stream when not given.  ``dev_error`` is an
    optional int32 CUDA scalar the kernels OR error bits into.
    """
    B, h_q, h_kv, d_k, d_v, n_max = _cache_dims(q, K, V, seq_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    out, oflag = _out(out, out_dtype, B, h_q, d_v, q.device, stream)
    dt = _DTYPES[q.dtype] | oflag
    lib = load()
    with _on_device(q):
        need = workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, q.dtype, num_splits)
        workspace, nbytes, lock = _workspace(q.device, need, workspace, stream)
        with lock:
            st = lib.decode_attn_ex(_ptr(q), _ptr(K), _ptr(V), _ptr(seq_lens), _ptr(out), B, h_q,
                                    h_kv, d_k, d_v, n_max, float(scale), dt, int(num_splits),
                                    _ptr(workspace), nbytes, _ptr(dev_error), _stream(q, stream))
    _check(st, "decode_attn_ex")
    return out


def decode_attn_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, K: torch.Tensor,
                       V: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor | None = None,
                       seq_lens_out: torch.Tensor | None = None, scale: float | None = None,
                       num_splits: int = 0, workspace: torch.Tensor | None = None,
                       dev_error: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None,
                       out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Append row seq_lens[b] of every kv head and decode over seq_lens[b] + 1 rows,
    in one launch (calls ``decode_attn_append``); returns ``out``."""
    B, h_q, h_kv, d_k, d_v, n_max = _cache_dims(q, K, V, seq_lens)
    if k_new.shape != (B, h_kv, d_k) or v_new.shape != (B, h_kv, d_v):
        raise ValueError("k_new/v_new must be [B, h_kv, d]")
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != K.dtype:
            raise ValueError(f"{name} must be a contiguous CUDA tensor of the cache dtype")
    if seq_lens_out is not None and (seq_lens_out.shape != (B,) or seq_lens_out.dtype != torch.int32):
        raise ValueError("seq_lens_out must be an int32 tensor of shape [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    out, oflag = _out(out, out_dtype, B, h_q, d_v, q.device, stream)
    lib = load()
    with _on_device(q):
        need = workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, q.dtype, num_splits)
        workspace, nbytes, lock = _workspace(q.device, need, workspace, stream)
        with lock:
            st = lib.decode_attn_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(K), _ptr(V),
                                        _ptr(seq_lens), _ptr(seq_lens_out), _ptr(out), B, h_q, h_kv,
                                        d_k, d_v, n_max, float(scale), _DTYPES[q.dtype] | oflag,
                                        int(num_splits), _ptr(workspace), nbytes, _ptr(dev_error),
                                        _stream(q, stream))
    _check(st, "decode_attn_append")
    return out


def decode_attn_owned(q, K, V, seq_lens, out=None, scale=None, stream=None,
                      out_dtype=None) -> torch.Tensor:
    """Decode attention through ``decode_attn`` (library-owned workspace)."""
    B, h_q, h_kv, d_k, d_v, n_max = _cache_dims(q, K, V, seq_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    out, oflag = _out(out, out_dtype, B, h_q, d_v, q.device, stream)
    with _on_device(q):
        st = load().decode_attn(_ptr(q), _ptr(K), _ptr(V), _ptr(seq_lens), _ptr(out), B, h_q, h_kv,
                                d_k, d_v, n_max, float(scale), _DTYPES[q.dtype] | oflag,
                                _stream(q, stream))
    _check(st, "decode_attn")
    return out


def decode_attn_noalloc(q, K, V, seq_lens, out=None, scale=None, num_splits: int = 0,
                        dev_error=None, stream=None, out_dtype=None) -> torch.Tensor:
    """Decode attention through ``decode_attn_noalloc``: the split scratch is the
    library's own fixed device buffer, so nothing is allocated for it.  Calls
    whose kernels may overlap on the GPU share that buffer and must be
    serialised by the caller."""
    B, h_q, h_kv, d_k, d_v, n_max = _cache_dims(q, K, V, seq_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    out, oflag = _out(out, out_dtype, B, h_q, d_v, q.device, stream)
    with _on_device(q):
        st = load().decode_attn_noalloc(_ptr(q), _ptr(K), _ptr(V), _ptr(seq_lens), _ptr(out), B, h_q,
                                        h_kv, d_k, d_v, n_max, float(scale),
                                        _DTYPES[q.dtype] | oflag,
                                        int(num_splits), _ptr(dev_error), _stream(q, stream))
    _check(st, "decode_attn_noalloc")
    return out


def decode_attn_partial(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor,
                        row_begin: int = 0, row_end: int | None = None,
                        o: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        scale: float | None = None, num_splits: int = 0,
                        workspace: torch.Tensor | None = None,
                        dev_error: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None):
    """One shard of a sequence-sharded decode (calls ``decode_attn_partial``): the
    decode of rows [row_begin, row_end) of every sequence (clipped to its length).
    Returns ``(o, lse)``: the normalised output [B, h_q, d_v] float32 and the
    natural-log log-sum-exp of those rows' scores [B, h_q] float32 (-inf when a
    sequence has no rows in the range)."""
    B, h_q, h_kv, d_k, d_v, n_max = _cache_dims(q, K, V, seq_lens)
    if row_end is None:
        row_end = n_max
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    o, _ = _out(o, torch.float32, B, h_q, d_v, q.device, stream)
    if lse is None:
        with _on_stream(stream):
            lse = torch.empty((B, h_q), dtype=torch.float32, device=q.device)
    if lse.shape != (B, h_q) or lse.dtype != torch.float32 or not lse.is_contiguous() \
            or lse.device != q.device:
        raise ValueError("lse must be a contiguous float32 tensor [B, h_q] on the query's device")
    lib = load()
    with _on_device(q):
        need = workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, q.dtype, num_splits)
        workspace, nbytes, lock = _workspace(q.device, need, workspace, stream)
        with lock:
            st = lib.decode_attn_partial(_ptr(q), _ptr(K), _ptr(V), _ptr(seq_lens), int(row_begin),
                                         int(row_end), _ptr(o), _ptr(lse), B, h_q, h_kv, d_k, d_v,
                                         n_max, float(scale), _DTYPES[q.dtype], int(num_splits),
                                         _ptr(workspace), nbytes, _ptr(dev_error),
                                         _stream(q, stream))
    _check(st, "decode_attn_partial")
    return o, lse


def decode_attn_combine(o_parts: torch.Tensor, lse_parts: torch.Tensor,
                        out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None,
                        out_dtype: torch.dtype | None = None,
                        stream: torch.cuda.Stream | None = None):
    """Merge S partial results over disjoint row sets (calls ``decode_attn_combine``):
    ``o_parts`` [S, B, h_q, d_v] and ``lse_parts`` [S, B, h_q] (float32, natural log,
    on this GPU).  Returns ``(out, lse_out)``."""
    if o_parts.dim() != 4 or lse_parts.dim() != 3 or o_parts.shape[:3] != lse_parts.shape:
        raise ValueError("expected o_parts [S, B, h_q, d_v] and lse_parts [S, B, h_q]")
    for name, t in (("o_parts", o_parts), ("lse_parts", lse_parts)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    S, B, h_q, d_v = o_parts.shape
    out, oflag = _out(out, out_dtype, B, h_q, d_v, o_parts.device, stream)
    if lse_out is None:
        with _on_stream(stream):
            lse_out = torch.empty((B, h_q), dtype=torch.float32, device=o_parts.device)
    if lse_out.shape != (B, h_q) or lse_out.dtype != torch.float32 or not lse_out.is_contiguous():
        raise ValueError("lse_out must be a contiguous float32 tensor [B, h_q]")
    with _on_device(o_parts):
        st = load().decode_attn_combine(_ptr(o_parts), _ptr(lse_parts), S, _ptr(out), _ptr(lse_out),
                                        B, h_q, d_v, DA_FP32 | oflag, _stream(o_parts, stream))
    _check(st, "decode_attn_combine")
    return out, lse_out


def kv_append(k_new: torch.Tensor, v_new: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
              pos: torch.Tensor, dev_error: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None) -> None:
    """Write row pos[b] of every (b, kv head) of K and V in place (exact copy)."""
    if K.dim() != 4 or V.dim() != 4:
        raise ValueError("K, V must be [B, h_kv, n_max, d]")
    B, h_kv, n_max, d_k = K.shape
    d_v = V.shape[3]
    if k_new.shape != (B, h_kv, d_k) or v_new.shape != (B, h_kv, d_v) or V.shape[:3] != K.shape[:3]:
        raise ValueError("k_new/v_new/K/V shapes disagree")
    if pos.shape != (B,) or pos.dtype != torch.int32:
        raise ValueError("pos must be an int32 tensor of shape [B]")
    for name, t in (("k_new", k_new), ("v_new", v_new), ("K", K), ("V", V), ("pos", pos)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if not (k_new.dtype == v_new.dtype == K.dtype == V.dtype) or K.dtype not in _DTYPES:
        raise ValueError("k_new, v_new, K, V must share dtype float32 or bfloat16")
    with _on_device(K):
        st = load().kv_append(_ptr(k_new), _ptr(v_new), _ptr(K), _ptr(V), _ptr(pos), B, h_kv, d_k,
                              d_v, n_max, _DTYPES[K.dtype], _ptr(dev_error), _stream(K, stream))
    _check(st, "kv_append")


# ----------------------------------------------------------------- 8-bit caches
def _q8_dims(q, K, V, k_scale, v_scale, seq_lens):
    if q.dim() != 3 or K.dim() != 4 or V.dim() != 4:
        raise ValueError("expected q [B, h_q, d], K/V codes [B, h_kv, n_max, d]")
    B, h_q, d_k = q.shape
    Bk, h_kv, n_max, d_k2 = K.shape
    if V.shape != K.shape or Bk != B or d_k2 != d_k:
        raise ValueError("q, K and V shapes disagree")
    if K.dtype not in _Q8_DTYPES or V.dtype != K.dtype:
        raise ValueError("K and V must be torch.int8 or torch.float8_e4m3fn code tensors")
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16 with an 8-bit cache")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.shape != (B, h_kv, n_max) or t.dtype != torch.float32:
            raise ValueError(f"{name} must be a float32 tensor [B, h_kv, n_max]")
    if seq_lens.shape != (B,) or seq_lens.dtype != torch.int32:
        raise ValueError("seq_lens must be an int32 tensor of shape [B]")
    for name, t in (("q", q), ("K", K), ("V", V), ("k_scale", k_scale), ("v_scale", v_scale),
                    ("seq_lens", seq_lens)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return B, h_q, h_kv, d_k, d_k, n_max


def kv_quantize(x: torch.Tensor, code_dtype: torch.dtype, stream=None):
    """Rows x [..., d] (float32 or bfloat16, CUDA) -> (codes [..., d] of ``code_dtype``
    (torch.int8 or torch.float8_e4m3fn), scales float32 [...]) by absmax scaling
    (calls ``kv_quantize``)."""
    if x.dtype not in _DTYPES or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 or bfloat16 CUDA tensor")
    d = x.shape[-1]
    with _on_stream(stream):
        codes = torch.empty(x.shape, dtype=code_dtype, device=x.device)
        scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    with _on_device(x):
        st = load().kv_quantize(_ptr(x), _DTYPES[x.dtype], _ptr(codes), _ptr(scales),
                                x.numel() // d if d else 0, d, _Q8_DTYPES[code_dtype],
                                _stream(x, stream))
    _check(st, "kv_quantize")
    return codes, scales


def decode_attn_q8(q, K, V, k_scale, v_scale, seq_lens, out=None, scale=None, num_splits: int = 0,
                   workspace=None, dev_error=None, stream=None, out_dtype=None) -> torch.Tensor:
    """Decode over an 8-bit cache (calls ``decode_attn_q8_ex``): K, V codes
    [B, h_kv, n_max, d] (torch.int8 or torch.float8_e4m3fn) with row scales
    [B, h_kv, n_max]; q bf16 [B, h_q, d].  Returns ``out``."""
    B, h_q, h_kv, d_k, d_v, n_max = _q8_dims(q, K, V, k_scale, v_scale, seq_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    out, oflag = _out(out, out_dtype, B, h_q, d_v, q.device, stream)
    lib = load()
    with _on_device(q):
        need = workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, K.dtype, num_splits)
        workspace, nbytes, lock = _workspace(q.device, need, workspace, stream)
        with lock:
            st = lib.decode_attn_q8_ex(_ptr(q), _ptr(K), _ptr(V), _ptr(k_scale), _ptr(v_scale),
                                       _ptr(seq_lens), _ptr(out), B, h_q, h_kv, d_k, d_v, n_max,
                                       float(scale), _Q8_DTYPES[K.dtype] | oflag, int(num_splits),
                                       _ptr(workspace), nbytes, _ptr(dev_error), _stream(q, stream))
    _check(st, "decode_attn_q8_ex")
    return out


def decode_attn_q8_append(q, k_new, v_new, k_new_scale, v_new_scale, K, V, k_scale, v_scale,
                          seq_lens, out=None, seq_lens_out=None, scale=None, num_splits: int = 0,
                          workspace=None, dev_error=None, stream=None, out_dtype=None):
    """Append the code rows k_new/v_new [B, h_kv, d] (scales [B, h_kv]) at row
    seq_lens[b] of an 8-bit cache and decode over seq_lens[b] + 1 rows in one
    launch (calls ``decode_attn_q8_append``).  Returns ``out``."""
    B, h_q, h_kv, d_k, d_v, n_max = _q8_dims(q, K, V, k_scale, v_scale, seq_lens)
    for name, t, shape, dt in (("k_new", k_new, (B, h_kv, d_k), K.dtype),
                               ("v_new", v_new, (B, h_kv, d_v), K.dtype),
                               ("k_new_scale", k_new_scale, (B, h_kv), torch.float32),
                               ("v_new_scale", v_new_scale, (B, h_kv), torch.float32)):
        if t.shape != shape or t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor {list(shape)} of {dt}")
    if seq_lens_out is not None and (seq_lens_out.shape != (B,) or seq_lens_out.dtype != torch.int32):
        raise ValueError("seq_lens_out must be an int32 tensor of shape [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    out, oflag = _out(out, out_dtype, B, h_q, d_v, q.device, stream)
    lib = load()
    with _on_device(q):
        need = workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, K.dtype, num_splits)
        workspace, nbytes, lock = _workspace(q.device, need, workspace, stream)
        with lock:
            st = lib.decode_attn_q8_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_new_scale),
                                           _ptr(v_new_scale), _ptr(K), _ptr(V), _ptr(k_scale),
                                           _ptr(v_scale), _ptr(seq_lens), _ptr(seq_lens_out),
                                           _ptr(out), B, h_q, h_kv, d_k, d_v, n_max, float(scale),
                                           _Q8_DTYPES[K.dtype] | oflag, int(num_splits),
                                           _ptr(workspace), nbytes, _ptr(dev_error),
                                           _stream(q, stream))
    _check(st, "decode_attn_q8_append")
    return out


def kv_append_q8(k_new, v_new, k_new_scale, v_new_scale, K, V, k_scale, v_scale, pos,
                 dev_error=None, stream=None) -> None:
    """Write code row pos[b] and its scale into every (b, kv head) of an 8-bit cache."""
    if K.dim() != 4 or V.shape != K.shape or K.dtype not in _Q8_DTYPES or V.dtype != K.dtype:
        raise ValueError("K, V must be 8-bit code tensors [B, h_kv, n_max, d] of one dtype")
    B, h_kv, n_max, d = K.shape
    for name, t, shape, dt in (("k_new", k_new, (B, h_kv, d), K.dtype),
                               ("v_new", v_new, (B, h_kv, d), K.dtype),
                               ("k_new_scale", k_new_scale, (B, h_kv), torch.float32),
                               ("v_new_scale", v_new_scale, (B, h_kv), torch.float32),
                               ("k_scale", k_scale, (B, h_kv, n_max), torch.float32),
                               ("v_scale", v_scale, (B, h_kv, n_max), torch.float32),
                               ("pos", pos, (B,), torch.int32)):
        if t.shape != shape or t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor {list(shape)} of {dt}")
    with _on_device(K):
        st = load().kv_append_q8(_ptr(k_new), _ptr(v_new), _ptr(k_new_scale), _ptr(v_new_scale),
                                 _ptr(K), _ptr(V), _ptr(k_scale), _ptr(v_scale), _ptr(pos), B, h_kv,
                                 d, d, n_max, _Q8_DTYPES[K.dtype], _ptr(dev_error),
                                 _stream(K, stream))
    _check(st, "kv_append_q8")


def launch_count() -> int:
    """Kernels launched by the library in this process so far."""
    return int(load().decode_attn_launch_count())


# ----------------------------------------------------------------- score terms
class ScoreMod(NamedTuple):
    """What a model adds to the plain scores before the softmax, and which cached
    rows the query (at row n - 1 of its n rows) sees; see ``da_score_mod``.

    ``softcap`` c > 0: u = c tanh(t / c) of the scaled score t.  ``slopes`` (float32
    CUDA tensor [h_q]): s_l = u_l - slopes[h] * (n - 1 - l).  Row l < n is seen when
    l < ``prefix`` or l >= max(doc_begin[b], n - window): ``window`` last rows (0: all),
    ``doc_begin`` (int32 CUDA tensor [B]) the first row of the query's document."""
    softcap: float = 0.0
    slopes: torch.Tensor | None = None
    window: int = 0
    prefix: int = 0
    doc_begin: torch.Tensor | None = None


class _CMod(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int), ("prefix", ctypes.c_int),
                ("slopes", ctypes.c_void_p), ("doc_begin", ctypes.c_void_p)]


def _c_mod(mod: ScoreMod, B: int, h_q: int, device: int) -> _CMod:
    """The C struct of ``mod`` for tensors on CUDA device ``device``."""
    softcap, slopes, window, prefix, begin = mod
    if slopes is not None and (slopes.shape != (h_q,) or slopes.dtype != torch.float32
                               or slopes.get_device() != device or not slopes.is_contiguous()):
        raise ValueError("slopes must be a contiguous float32 tensor [h_q] on the query's device")
    if begin is not None:
        _row_counts("doc_begin", begin, B, device)
    if not 0 <= window < 1 << 31 or not 0 <= prefix < 1 << 31:
        raise ValueError("window and prefix must be non-negative ints")
    return _CMod(softcap, window, prefix, None if slopes is None else slopes.data_ptr(),
                 None if begin is None else begin.data_ptr())


def _row_counts(name: str, t: torch.Tensor | None, B: int, device: int) -> None:
    if t is not None and (t.shape != (B,) or t.dtype != torch.int32 or t.get_device() != device
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor [B] on the device of the others")


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _error_word(t: torch.Tensor | None, device: int):
    if t is None:
        return None
    if t.get_device() != device or t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError("dev_error must be an int32 tensor on the device of the others")
    return t.data_ptr()


def _bad_seq_lens(t: torch.Tensor, B: int, device: int) -> bool:
    return (t.dtype is not torch.int32 or t.shape != (B,) or t.get_device() != device
            or not t.is_contiguous())


def _out_on(out: torch.Tensor | None, out_dtype: torch.dtype | None, B: int, h_q: int, d_v: int,
            q: torch.Tensor, device: int, stream):
    """The output tensor (allocated when None, in the call's stream) and its dtype flag."""
    if out is None:
        with _on_stream(stream):
            out = torch.empty((B, h_q, d_v), dtype=out_dtype or torch.float32, device=q.device)
    dtype = out.dtype
    if out.shape != (B, h_q, d_v) or out.get_device() != device or not out.is_contiguous() \
            or (dtype is not torch.bfloat16 and dtype is not torch.float32) \
            or (out_dtype is not None and dtype is not out_dtype):
        raise ValueError("out must be a contiguous float32 or bfloat16 tensor [B, h_q, d_v] "
                         "on the query's device")
    return out, (DA_OUT_BF16 if dtype is torch.bfloat16 else 0)


def _cache_args(q, K, V, seq_lens, out, out_dtype, stream):
    """Checks of a decode over an fp32 or bf16 cache: its sizes, the output, the dtype code.
    (A step's host time is mostly these checks and the launches: 2 us of about 11.)"""
    device = q.get_device()
    dtype = q.dtype
    if q.dim() != 3 or K.dim() != 4 or V.dim() != 4:
        raise ValueError("expected q [B, h_q, d_k], K [B, h_kv, n_max, d_k], V [B, h_kv, n_max, d_v]")
    B, h_q, d_k = q.shape
    Bk, h_kv, n_max, d = K.shape
    Bv, h_kv2, n_max2, d_v = V.shape
    if Bk != B or Bv != B or h_kv2 != h_kv or n_max2 != n_max or d != d_k:
        raise ValueError("q, K and V shapes disagree")
    code = _DTYPES.get(dtype)
    if code is None or K.dtype is not dtype or V.dtype is not dtype:
        raise ValueError("q, K, V must share dtype float32 or bfloat16")
    if device < 0 or K.get_device() != device or V.get_device() != device \
            or not (q.is_contiguous() and K.is_contiguous() and V.is_contiguous()):
        raise ValueError("q, K and V must be contiguous CUDA tensors on one device")
    if _bad_seq_lens(seq_lens, B, device):
        raise ValueError("seq_lens must be a contiguous int32 tensor [B] on the device of the others")
    out, oflag = _out_on(out, out_dtype, B, h_q, d_v, q, device, stream)
    return device, out, (B, h_q, h_kv, d_k, d_v, n_max), code | oflag


def _enter(device: int) -> int:
    """Makes ``device`` current; returns the device to go back to, or -1."""
    cur = torch._C._cuda_getDevice()
    if cur == device:
        return -1
    torch.cuda.set_device(device)
    return cur


def _raw(stream, device: int) -> int:
    """The raw stream of a call: that of ``stream``, else the device's current one."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


_mod_bytes_cache: dict = {}


def _terms_workspace(entry: str, cmod, sizes, device: int, stream, raw: int,
                     workspace: torch.Tensor | None):
    """The workspace of a call with score terms or block scales, its bytes and the lock to hold
    while the library is called (``sizes``: the sizes, dtype code and split choice)."""
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the query's device")
        return workspace, workspace.numel() * workspace.element_size(), _unlocked
    key = (entry, device, sizes, 0, 0) if cmod is None else (entry, device, sizes, cmod.window,
                                                             cmod.prefix)
    need = _mod_bytes_cache.get(key)
    if need is None:
        st = ctypes.c_int(0)
        need = int(getattr(load(), entry)(None if cmod is None else ctypes.byref(cmod), *sizes,
                                          ctypes.byref(st)))
        _check(st.value, entry)
        if len(_mod_bytes_cache) > 4096:
            _mod_bytes_cache.clear()
        _mod_bytes_cache[key] = need
    if need == 0:
        return None, 0, _unlocked
    return _kept_workspace((device, raw, "terms"), need, stream)


def decode_attn_mod(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor,
                    mod: ScoreMod, out: torch.Tensor | None = None, scale: float | None = None,
                    num_splits: int = 0, workspace: torch.Tensor | None = None,
                    dev_error: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None,
                    out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """``decode_attn`` with score terms (calls ``decode_attn_mod``): capped scores, a distance
    bias, a window, documents and an always-seen prefix, as ``mod`` says.  Returns ``out``."""
    device, out, dims, dt = _cache_args(q, K, V, seq_lens, out, out_dtype, stream)
    cm = _c_mod(mod, dims[0], dims[1], device)
    err = None if dev_error is None else _error_word(dev_error, device)
    if scale is None:
        scale = 1.0 / math.sqrt(dims[3])
    prev = _enter(device)
    try:
        raw = _raw(stream, device)
        ws, nbytes, lock = _terms_workspace("decode_attn_mod_workspace_bytes", cm,
                                            (*dims, dt, num_splits), device, stream, raw, workspace)
        with lock:
            st = (_lib or load()).decode_attn_mod(
                q.data_ptr(), K.data_ptr(), V.data_ptr(), seq_lens.data_ptr(), ctypes.byref(cm),
                out.data_ptr(), *dims, scale, dt, num_splits, _addr(ws), nbytes, err, raw)
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "decode_attn_mod")
    return out


def decode_attn_mod_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                           K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor, mod: ScoreMod,
                           out: torch.Tensor | None = None,
                           seq_lens_out: torch.Tensor | None = None, scale: float | None = None,
                           num_splits: int = 0, workspace: torch.Tensor | None = None,
                           dev_error: torch.Tensor | None = None,
                           stream: torch.cuda.Stream | None = None,
                           out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """``decode_attn_append`` with score terms (calls ``decode_attn_mod_append``): row
    seq_lens[b] of every kv head is appended, and the query sees what ``mod`` says of the
    seq_lens[b] + 1 rows.  Returns ``out``."""
    device, out, dims, dt = _cache_args(q, K, V, seq_lens, out, out_dtype, stream)
    B, h_q, h_kv, d_k, d_v, _ = dims
    if k_new.shape != (B, h_kv, d_k) or v_new.shape != (B, h_kv, d_v):
        raise ValueError("k_new/v_new must be [B, h_kv, d]")
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.get_device() != device or not t.is_contiguous() or t.dtype != K.dtype:
            raise ValueError(f"{name} must be a contiguous CUDA tensor of the cache dtype")
    _row_counts("seq_lens_out", seq_lens_out, B, device)
    cm = _c_mod(mod, B, h_q, device)
    err = None if dev_error is None else _error_word(dev_error, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    prev = _enter(device)
    try:
        raw = _raw(stream, device)
        ws, nbytes, lock = _terms_workspace("decode_attn_mod_workspace_bytes", cm,
                                            (*dims, dt, num_splits), device, stream, raw, workspace)
        with lock:
            st = (_lib or load()).decode_attn_mod_append(
                q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), K.data_ptr(), V.data_ptr(),
                seq_lens.data_ptr(), _addr(seq_lens_out), ctypes.byref(cm), out.data_ptr(), *dims,
                scale, dt, num_splits, _addr(ws), nbytes, err, raw)
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "decode_attn_mod_append")
    return out


# ------------------------------------------------- 8-bit caches with a scale per block
def _q8b_cache(K, V, k_scale, v_scale, block: int):
    """Checks a block-scaled cache; returns its device, B, h_kv, n_max, d."""
    dtype, device, shape = K.dtype, K.get_device(), K.shape
    if len(shape) != 4 or dtype not in _Q8_DTYPES or V.dtype is not dtype or V.shape != shape:
        raise ValueError("K, V must be 8-bit code tensors [B, h_kv, n_max, d] of one dtype")
    if block not in (16, 32, 64, 128):
        raise ValueError("block must be 16, 32, 64 or 128")
    B, h_kv, n_max, d = shape
    if device < 0 or V.get_device() != device or not (K.is_contiguous() and V.is_contiguous()):
        raise ValueError("K and V must be contiguous CUDA tensors on one device")
    scales = (B, h_kv, -(-n_max // block))
    for t in (k_scale, v_scale):
        if t.dtype is not torch.float32 or t.shape != scales or t.get_device() != device \
                or not t.is_contiguous():
            raise ValueError("k_scale and v_scale must be contiguous float32 tensors "
                             f"{list(scales)} on the cache's device")
    return device, B, h_kv, n_max, d


def decode_attn_q8b(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, seq_lens: torch.Tensor, block: int,
                    mod: ScoreMod | None = None, out: torch.Tensor | None = None,
                    scale: float | None = None, num_splits: int = 0,
                    workspace: torch.Tensor | None = None, dev_error: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None,
                    out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Decode over an 8-bit cache with a scale per block of tokens and head (calls
    ``decode_attn_q8b``): K, V codes [B, h_kv, n_max, d] (torch.int8 or torch.float8_e4m3fn),
    scales float32 [B, h_kv, ceil(n_max / block)], q bf16 [B, h_q, d]; ``mod`` adds score terms.
    Returns ``out``."""
    device, B, h_kv, n_max, d = _q8b_cache(K, V, k_scale, v_scale, block)
    h_q = q.shape[1] if q.dim() == 3 else 0
    if q.shape != (B, h_q, d) or q.dtype is not torch.bfloat16 or q.get_device() != device \
            or not q.is_contiguous():
        raise ValueError("q must be a contiguous bfloat16 tensor [B, h_q, d] on the cache's device")
    if _bad_seq_lens(seq_lens, B, device):
        raise ValueError("seq_lens must be a contiguous int32 tensor [B] on the cache's device")
    out, oflag = _out_on(out, out_dtype, B, h_q, d, q, device, stream)
    dt = _Q8_DTYPES[K.dtype] | oflag
    cm = None if mod is None else _c_mod(mod, B, h_q, device)
    err = None if dev_error is None else _error_word(dev_error, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    prev = _enter(device)
    try:
        raw = _raw(stream, device)
        ws, nbytes, lock = _terms_workspace("decode_attn_q8b_workspace_bytes", cm,
                                            (B, h_q, h_kv, d, d, n_max, dt, num_splits), device,
                                            stream, raw, workspace)
        with lock:
            st = (_lib or load()).decode_attn_q8b(
                q.data_ptr(), K.data_ptr(), V.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                block, seq_lens.data_ptr(), None if cm is None else ctypes.byref(cm),
                out.data_ptr(), B, h_q, h_kv, d, d, n_max, scale, dt, num_splits, _addr(ws), nbytes,
                err, raw)
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "decode_attn_q8b")
    return out


_Strides = ctypes.c_longlong * 3


def kv_append_q8b(k_new: torch.Tensor, v_new: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                  k_scale: torch.Tensor, v_scale: torch.Tensor, pos: torch.Tensor, block: int,
                  n_new: torch.Tensor | None = None, dev_error: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None) -> None:
    """Quantise rows as they are written into a block-scaled cache (calls ``kv_append_q8b``):
    the rows k_new/v_new [B, h_kv, T, d] (float32 or bfloat16, any strides but a contiguous last
    dimension; [B, h_kv, d] for one row) become rows pos[b] .. of sequence b, n_new[b] of them
    where given.  A block's scale grows to what its new rows need, and the codes it holds are
    then rewritten.  Lengths are the caller's to advance."""
    device, B, h_kv, n_max, d = _q8b_cache(K, V, k_scale, v_scale, block)
    if k_new.dim() == 3:
        k_new = k_new.unsqueeze(2)
    if v_new.dim() == 3:
        v_new = v_new.unsqueeze(2)
    T = k_new.shape[2] if k_new.dim() == 4 else -1
    x_dtype = k_new.dtype
    code = _DTYPES.get(x_dtype)
    if code is None or v_new.dtype is not x_dtype or k_new.shape != (B, h_kv, T, d) \
            or v_new.shape != k_new.shape or k_new.get_device() != device \
            or v_new.get_device() != device:
        raise ValueError("k_new and v_new must be float32 or bfloat16 tensors [B, h_kv, T, d] of "
                         "one type on the cache's device")
    strides = []
    for t in (k_new, v_new):
        sb, sh, st, sd = t.stride()
        if sd != 1:
            raise ValueError("k_new and v_new must be contiguous in their last dimension")
        # a dimension of one element has no step: its stride in the tensor may be anything
        strides.append(_Strides(sb if B > 1 else 0, sh if h_kv > 1 else 0, st if T > 1 else 0))
    if _bad_seq_lens(pos, B, device):
        raise ValueError("pos must be a contiguous int32 tensor [B] on the cache's device")
    if n_new is not None:
        _row_counts("n_new", n_new, B, device)
    err = None if dev_error is None else _error_word(dev_error, device)
    prev = _enter(device)
    try:
        st = (_lib or load()).kv_append_q8b(
            k_new.data_ptr(), v_new.data_ptr(), strides[0], strides[1], code, T,
            _addr(n_new), K.data_ptr(), V.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block,
            pos.data_ptr(), B, h_kv, d, n_max, _Q8_DTYPES[K.dtype], err, _raw(stream, device))
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "kv_append_q8b")


def kv_read_q8b(K: torch.Tensor, V: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                seq_lens: torch.Tensor, block: int, rows: int | None = None,
                row_begin: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                v_out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                dev_error: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Read rows of a block-scaled cache back as values (calls ``kv_read_q8b``): row
    row_begin[b] + i (row_begin None: i) of sequence b goes to row i of k_out/v_out
    [B, h_kv, rows, d] (float32 or bfloat16) while it lies below seq_lens[b]; other rows of the
    outputs are left as they are (zero in outputs allocated here, of ``out_dtype``, with ``rows``
    rows, n_max by default).  Returns ``(k_out, v_out)``."""
    device, B, h_kv, n_max, d = _q8b_cache(K, V, k_scale, v_scale, block)
    if k_out is None or v_out is None:
        if k_out is not None or v_out is not None:
            raise ValueError("give both k_out and v_out, or neither")
        with _on_stream(stream):
            k_out, v_out = (torch.zeros((B, h_kv, n_max if rows is None else rows, d),
                                        dtype=out_dtype, device=K.device) for _ in range(2))
    T = k_out.shape[2] if k_out.dim() == 4 else -1
    if rows is not None and rows != T:
        raise ValueError("rows disagrees with the outputs")
    code = _DTYPES.get(k_out.dtype)
    for t in (k_out, v_out):
        if code is None or t.dtype is not k_out.dtype or t.shape != (B, h_kv, T, d) \
                or t.get_device() != device or not t.is_contiguous():
            raise ValueError("k_out and v_out must be contiguous float32 or bfloat16 tensors "
                             "[B, h_kv, rows, d] of one type on the cache's device")
    if _bad_seq_lens(seq_lens, B, device) or row_begin is not None \
            and _bad_seq_lens(row_begin, B, device):
        raise ValueError("seq_lens and row_begin must be contiguous int32 tensors [B] on the "
                         "cache's device")
    err = None if dev_error is None else _error_word(dev_error, device)
    prev = _enter(device)
    try:
        st = (_lib or load()).kv_read_q8b(
            K.data_ptr(), V.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block,
            seq_lens.data_ptr(), _addr(row_begin), k_out.data_ptr(), v_out.data_ptr(),
            code, T, B, h_kv, d, n_max, _Q8_DTYPES[K.dtype], err, _raw(stream, device))
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "kv_read_q8b")
    return k_out, v_out


# ----------------------------------- from projections to the cache, chunks, shared prefixes
_stride_cache: dict = {}


def _row_strides(name: str, t: torch.Tensor, shape, dtype, device: int, write: bool = False):
    """The strides (b, head, token) of rows t, which has to be of ``shape`` [B, h, T, d]."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} on the cache's device")
    key = (shape, t.stride(), write)
    known = _stride_cache.get(key)
    if known is not None:
        return known
    sb, sh, st, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    B, h, T, d = shape
    # a dimension of one element has no step: its stride in the tensor may be anything
    steps = (sb if B > 1 else 0, sh if h > 1 else 0, st if T > 1 else 0)
    if write:
        # rows that are written may not share an element: each step passes what the smaller ones reach
        reach = d
        for step, n in sorted(zip(steps, (B, h, T))):
            if n > 1:
                if step < reach:
                    raise ValueError(f"{name} must not overlap itself")
                reach = step * (n - 1) + reach
    if len(_stride_cache) > 4096:
        _stride_cache.clear()
    strides = _stride_cache[key] = _Strides(*steps)
    return strides


def _new_out(out, dtype, B: int, h: int, T: int, d: int, device, stream):
    """Rows [B, h, T, d] of an output; allocated token after token where not given."""
    if out is None:
        with _on_stream(stream):
            out = torch.empty((B, T, h, d), dtype=dtype, device=device).transpose(1, 2)
    return out


def kv_append_rope(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, K: torch.Tensor,
                   V: torch.Tensor, pos: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                   q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                   eps: float = 1e-6, n_new: torch.Tensor | None = None,
                   angle_pos: torch.Tensor | None = None, interleaved: bool = False,
                   q_out: torch.Tensor | None = None, dev_error: torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Norm each head of q and k, rotate them by position, and write k and v into the cache (calls
    ``kv_append_rope``): tokens q [B, h_q, T, d_k], k_new [B, h_kv, T, d_k], v_new [B, h_kv, T, d_v]
    (any strides but a contiguous last dimension; [B, h, d] for one token) become rows pos[b] ..
    of the caches K [B, h_kv, n_max, d_k], V [B, h_kv, n_max, d_v], n_new[b] of them where given.
    ``cos`` and ``sin`` are float32 [n_angles, rot / 2]; angle row angle_pos[b] + i (pos[b] + i where
    not given) turns token i.  Weights None: no norm.  Returns ``q_out``, shaped as q (allocated as
    [B, T, h_q, d_k] in memory when None; q itself is allowed).  Lengths are the caller's to advance."""
    single = q.dim() == 3
    if single:
        q, k_new, v_new = q.unsqueeze(2), k_new.unsqueeze(2), v_new.unsqueeze(2)
        if q_out is not None:
            q_out = q_out.unsqueeze(2)
    device, dtype = K.get_device(), K.dtype
    code = _DTYPES.get(dtype)
    if q.dim() != 4 or K.dim() != 4 or V.dim() != 4 or code is None or V.dtype is not dtype:
        raise ValueError("expected q [B, h_q, T, d_k] and float32 or bfloat16 caches K [B, h_kv, n_max, d_k], "
                         "V [B, h_kv, n_max, d_v]")
    B, h_kv, n_max, d_k = K.shape
    _, h_q, T, _ = q.shape
    d_v = V.shape[3]
    if device < 0 or V.shape != (B, h_kv, n_max, d_v) or V.get_device() != device \
            or not (K.is_contiguous() and V.is_contiguous()):
        raise ValueError("K and V must be contiguous CUDA tensors of one batch, on one device")
    q_shape = (B, h_q, T, d_k)
    strides = (_row_strides("q", q, q_shape, dtype, device),
               _row_strides("k_new", k_new, (B, h_kv, T, d_k), dtype, device),
               _row_strides("v_new", v_new, (B, h_kv, T, d_v), dtype, device))
    q_out = _new_out(q_out, dtype, B, h_q, T, d_k, K.device, stream)
    out_strides = _row_strides("q_out", q_out, q_shape, dtype, device, write=True)
    angles, f32 = cos.shape, torch.float32
    if len(angles) != 2 or sin.shape != angles or cos.dtype is not f32 or sin.dtype is not f32 \
            or cos.get_device() != device or sin.get_device() != device \
            or not (cos.is_contiguous() and sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous float32 tensors [n_angles, rot / 2] on the "
                         "cache's device")
    if angles[0] >= 1 << 31 or angles[1] >= 1 << 30:   # (the library would take 32 bits of them)
        raise ValueError("cos and sin must have less than 2^31 rows, of at most d_k / 2 angles")
    for t in (q_weight, k_weight):
        if t is not None and (t.dtype is not dtype or t.shape != (d_k,) or t.get_device() != device
                              or not t.is_contiguous()):
            raise ValueError("q_weight and k_weight must be contiguous tensors [d_k] of the cache's "
                             "type and device")
    if _bad_seq_lens(pos, B, device):
        raise ValueError("pos must be a contiguous int32 tensor [B] on the cache's device")
    if n_new is not None:
        _row_counts("n_new", n_new, B, device)
    if angle_pos is not None:
        _row_counts("angle_pos", angle_pos, B, device)
    err = None if dev_error is None else _error_word(dev_error, device)
    prev = _enter(device)
    try:
        st = (_lib or load()).kv_append_rope(
            q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), *strides, T, _addr(n_new),
            q_out.data_ptr(), out_strides, K.data_ptr(), V.data_ptr(), pos.data_ptr(),
            cos.data_ptr(), sin.data_ptr(), angles[0], 2 * angles[1], 1 if interleaved else 0,
            _addr(angle_pos), _addr(q_weight), _addr(k_weight), eps, B, h_q, h_kv, d_k, d_v, n_max,
            code, err, _raw(stream, device))
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "kv_append_rope")
    return q_out.squeeze(2) if single else q_out


def _attend_workspace(entry: str, sizes, device: int, stream, raw: int,
                      workspace: torch.Tensor | None):
    """The workspace of a chunk or shared-prefix call, its bytes and the lock to hold while the
    library is called."""
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the query's device")
        return workspace, workspace.numel() * workspace.element_size(), _unlocked
    key = (entry, device, sizes)
    need = _mod_bytes_cache.get(key)
    if need is None:
        st = ctypes.c_int(0)
        need = int(getattr(load(), entry)(*sizes, ctypes.byref(st)))
        _check(st.value, entry)
        if len(_mod_bytes_cache) > 4096:
            _mod_bytes_cache.clear()
        _mod_bytes_cache[key] = need
    if need == 0:
        return None, 0, _unlocked
    return _kept_workspace((device, raw, "attend"), need, stream)


def _bf16_weights(code: int) -> int:
    if not code & DA_OUT_BF16:
        raise ValueError("bf16_weights goes with a bfloat16 out")
    return code | DA_BF16_WEIGHTS


def chunk_attn(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor,
               n_new: torch.Tensor | None = None, window: int = 0, prefix: int = 0,
               out: torch.Tensor | None = None, scale: float | None = None,
               workspace: torch.Tensor | None = None, dev_error: torch.Tensor | None = None,
               stream: torch.cuda.Stream | None = None,
               out_dtype: torch.dtype | None = None, bf16_weights: bool = False) -> torch.Tensor:
    """Attention of a chunk of tokens over the cache that holds them (calls ``chunk_attn``): q
    [B, h_q, T, d] bf16 (any strides but a contiguous last dimension), K, V [B, h_kv, n_max, d];
    the last n_new[b] of sequence b's seq_lens[b] rows (T where not given) are the chunk's.  Token i
    at row p sees row l <= p when l > p - window (0: all) or l < prefix.  Returns ``out`` [B, h_q,
    T, d], float32 or bfloat16 (any strides; allocated as [B, T, h_q, d] in memory when None);
    tokens at or past n_new[b] are left as they are.  ``bf16_weights`` (with a bfloat16 out): the
    softmax's weights are multiplied as one bfloat16, 2^-8 of each, instead of 2^-16; prompts then
    take three quarters of the time."""
    device = q.get_device()
    if q.dim() != 4 or K.dim() != 4 or V.shape != K.shape:
        raise ValueError("expected q [B, h_q, T, d], K and V [B, h_kv, n_max, d]")
    B, h_kv, n_max, d = K.shape
    _, h_q, T, _ = q.shape
    if K.dtype is not torch.bfloat16 or V.dtype is not torch.bfloat16 or device < 0 \
            or K.get_device() != device or V.get_device() != device \
            or not (K.is_contiguous() and V.is_contiguous()):
        raise ValueError("K and V must be contiguous bfloat16 CUDA tensors on the query's device")
    shape = (B, h_q, T, d)
    q_strides = _row_strides("q", q, shape, torch.bfloat16, device)
    out = _new_out(out, out_dtype or torch.float32, B, h_q, T, d, q.device, stream)
    dtype = out.dtype
    if (dtype is not torch.bfloat16 and dtype is not torch.float32) \
            or (out_dtype is not None and dtype is not out_dtype):
        raise ValueError("out must be float32 or bfloat16 (and of out_dtype where that is given)")
    out_strides = _row_strides("out", out, shape, dtype, device, write=True)
    if _bad_seq_lens(seq_lens, B, device):
        raise ValueError("seq_lens must be a contiguous int32 tensor [B] on the device of the others")
    if n_new is not None:
        _row_counts("n_new", n_new, B, device)
    if not 0 <= window < 1 << 31 or not 0 <= prefix < 1 << 31:
        raise ValueError("window and prefix must be non-negative ints")
    err = None if dev_error is None else _error_word(dev_error, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    code = DA_BF16 | (DA_OUT_BF16 if dtype is torch.bfloat16 else 0)
    if bf16_weights:
        code = _bf16_weights(code)
    prev = _enter(device)
    try:
        raw = _raw(stream, device)
        ws, nbytes, lock = _attend_workspace("chunk_attn_workspace_bytes",
                                             (B, T, h_q, h_kv, d, n_max, code), device, stream, raw,
                                             workspace)
        with lock:
            st = (_lib or load()).chunk_attn(
                q.data_ptr(), q_strides, T, _addr(n_new), K.data_ptr(), V.data_ptr(),
                seq_lens.data_ptr(), window, prefix, out.data_ptr(), out_strides, B, h_q, h_kv, d,
                n_max, scale, code, _addr(ws), nbytes, err, raw)
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "chunk_attn")
    return out


def decode_attn_shared(q: torch.Tensor, K_prefix: torch.Tensor, V_prefix: torch.Tensor,
                       K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor,
                       out: torch.Tensor | None = None, prefix_len: int | None = None,
                       scale: float | None = None, workspace: torch.Tensor | None = None,
                       dev_error: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None,
                       out_dtype: torch.dtype | None = None,
                       bf16_weights: bool = False) -> torch.Tensor:
    """Decode attention of a batch that shares a prefix (calls ``decode_attn_shared``): each query q
    [B, h_q, d] sees the first prefix_len rows (all by default) of K_prefix, V_prefix [h_kv,
    prefix_max, d], then the seq_lens[b] rows of its own K, V [B, h_kv, n_max, d] (bf16).  The
    prefix is read once for every 256 query rows (sequences times a group's heads) of a KV head.
    ``bf16_weights``: as in ``chunk_attn``.  Returns ``out`` [B, h_q, d]."""
    device, out, dims, dt = _cache_args(q, K, V, seq_lens, out, out_dtype, stream)
    if bf16_weights:
        dt = _bf16_weights(dt)
    B, h_q, h_kv, d, d_v, n_max = dims
    shape, dtype = K_prefix.shape, K.dtype
    if len(shape) != 3 or shape[0] != h_kv or shape[2] != d or d_v != d or V_prefix.shape != shape \
            or K_prefix.dtype is not dtype or V_prefix.dtype is not dtype \
            or K_prefix.get_device() != device or V_prefix.get_device() != device \
            or not (K_prefix.is_contiguous() and V_prefix.is_contiguous()):
        raise ValueError("K_prefix and V_prefix must be contiguous tensors [h_kv, prefix_max, d] of "
                         "the cache's type and device")
    prefix_max = shape[1]
    if prefix_len is None:
        prefix_len = prefix_max
    elif not -(1 << 31) <= prefix_len < 1 << 31:   # (the library would take 32 bits of it)
        raise ValueError("prefix_len must be between 0 and prefix_max")
    err = None if dev_error is None else _error_word(dev_error, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    prev = _enter(device)
    try:
        raw = _raw(stream, device)
        ws, nbytes, lock = _attend_workspace("decode_attn_shared_workspace_bytes",
                                             (B, h_q, h_kv, d, n_max, prefix_len, dt), device,
                                             stream, raw, workspace)
        with lock:
            st = (_lib or load()).decode_attn_shared(
                q.data_ptr(), K_prefix.data_ptr(), V_prefix.data_ptr(), prefix_len, prefix_max,
                K.data_ptr(), V.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), B, h_q, h_kv, d,
                n_max, scale, dt, _addr(ws), nbytes, err, raw)
    finally:
        if prev >= 0:
            torch.cuda.set_device(prev)
    _check(st, "decode_attn_shared")
    return out
