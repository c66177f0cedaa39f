"""GB300 (sm_103a) chunk-parallel Kimi Delta Attention: forward and backward.

Thin Python binding of the C ABI in ``include/kda.h`` and, for the single-token
operators of serving, ``include/kda_serve.h`` (``lib/libkda_gb300.so``, built by
:func:`build`). This module only marshals arguments (those of the single-token
operators in C++, ``lib/_kda_serve.so``, where a call costs less): it checks
shapes, allocates outputs and the workspace with PyTorch's caching allocator,
passes raw device pointers and the current CUDA stream, and turns status codes
into exceptions. Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback, and calling without the built
library raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
from typing import Optional

import torch

from .build import LIB, SERVE, build  # noqa: F401

__all__ = ["build", "load", "Dims", "prepare_chunks", "workspace_bytes", "saved_bytes", "chunk_fwd", "chunk_bwd",
           "chunk_fwd_save", "chunk_bwd_from_saved", "step", "new_cache", "cache_append", "cache_attend",
           "cache_attend_workspace_bytes", "cache_resize", "KdaError", "STATUS", "DTYPE_BF16", "DTYPE_F32", "DTYPE_E4M3",
           "PASS_FWD", "PASS_BWD"]

DTYPE_BF16, DTYPE_F32, DTYPE_E4M3 = 0, 1, 2
PASS_FWD, PASS_BWD = 0, 1
CHUNK = 64
STATUS = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED", 3: "KDA_ERR_WORKSPACE", 4: "KDA_ERR_CUDA",
          5: "KDA_ERR_DEVICE_TIMEOUT"}


class KdaError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        msg = f"{where}: {STATUS.get(code, code)} ({load().kda_status_string(code).decode()})"
        if code == 4:
            msg += f" [{load().kda_last_cuda_error().decode()}]"
        super().__init__(msg)


class Dims(ctypes.Structure):
    """Mirror of ``kda_dims``."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("HV", ctypes.c_int32),
                ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("chunk", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("num_chunks", ctypes.c_int64), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class StepDims(ctypes.Structure):
    """Mirror of ``kda_step_dims``."""
    _fields_ = [("N", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("HV", ctypes.c_int32),
                ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("num_slots", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class Cache(ctypes.Structure):
    """Mirror of ``kda_cache``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_page", ctypes.c_int64), ("k_row", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_page", ctypes.c_int64), ("v_row", ctypes.c_int64),
                ("v_head", ctypes.c_int64), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("HKV", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Cache8(ctypes.Structure):
    """Mirror of ``kda_cache8``."""
    _fields_ = [("cache", Cache), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("k_scale_page", ctypes.c_int64),
                ("k_scale_block", ctypes.c_int64), ("k_scale_head", ctypes.c_int64), ("v_scale_page", ctypes.c_int64),
                ("v_scale_block", ctypes.c_int64), ("v_scale_head", ctypes.c_int64), ("block", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()
_P = ctypes.c_void_p


def load():
    """Load the built library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB):
                raise RuntimeError(f"KDA CUDA library not built ({LIB}); call chunked_gated_delta_10_gb300.build()")
            lib = ctypes.CDLL(LIB)
            lib.kda_status_string.restype = ctypes.c_char_p
            lib.kda_status_string.argtypes = [ctypes.c_int]
            lib.kda_prepare_chunks.restype = ctypes.c_int
            lib.kda_prepare_chunks.argtypes = [_P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P]
            lib.kda_workspace_bytes.restype = ctypes.c_size_t
            lib.kda_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32]
            lib.kda_chunk_fwd.restype = ctypes.c_int
            lib.kda_chunk_fwd.argtypes = [ctypes.POINTER(Dims)] + [_P] * 13 + [ctypes.c_size_t, _P]
            lib.kda_chunk_bwd.restype = ctypes.c_int
            lib.kda_chunk_bwd.argtypes = [ctypes.POINTER(Dims)] + [_P] * 19 + [ctypes.c_size_t, _P]
            lib.kda_chunk_bwd_fused.restype = ctypes.c_int
            lib.kda_chunk_bwd_fused.argtypes = [ctypes.POINTER(Dims)] + [_P] * 19 + [ctypes.c_size_t, _P]
            lib.kda_saved_bytes.restype = ctypes.c_size_t
            lib.kda_saved_bytes.argtypes = [ctypes.POINTER(Dims)]
            lib.kda_chunk_fwd_save.restype = ctypes.c_int
            lib.kda_chunk_fwd_save.argtypes = [ctypes.POINTER(Dims)] + [_P] * 12 + [ctypes.c_size_t, _P]
            lib.kda_chunk_bwd_from_saved.restype = ctypes.c_int
            lib.kda_chunk_bwd_from_saved.argtypes = ([ctypes.POINTER(Dims)] + [_P] * 12 + [ctypes.c_size_t] +
                                                     [_P] * 6 + [_P])
            lib.kda_device_status.restype = ctypes.c_int
            lib.kda_device_status.argtypes = [_P, _P]
            lib.kda_set_profile_events.restype = ctypes.c_int
            lib.kda_set_profile_events.argtypes = [_P, ctypes.c_int32]
            lib.kda_last_launch_count.restype = ctypes.c_int32
            lib.kda_last_launch_count.argtypes = []
            lib.kda_last_cuda_error.restype = ctypes.c_char_p
            lib.kda_last_cuda_error.argtypes = []
            lib.kda_launch_name.restype = ctypes.c_char_p
            lib.kda_launch_name.argtypes = [ctypes.c_int32]
            i32, i64 = ctypes.c_int32, ctypes.c_int64
            lib.kda_step.restype = ctypes.c_int
            lib.kda_step.argtypes = [ctypes.POINTER(StepDims)] + [_P] * 10
            lib.kda_cache_append.restype = ctypes.c_int
            lib.kda_cache_append.argtypes = [ctypes.POINTER(Cache), _P, i64, _P, i64, _P, i64, _P, i32, i32, i64, _P, _P,
                                             i32, i32, i32, _P, i64, i32, _P, _P, _P]
            lib.kda_cache_attend.restype = ctypes.c_int
            lib.kda_cache_attend.argtypes = [ctypes.POINTER(Cache), _P, i64, i32, i32, _P, i64, i32, _P, i32,
                                             ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P]
            lib.kda_cache_attend_workspace_bytes.restype = ctypes.c_size_t
            lib.kda_cache_attend_workspace_bytes.argtypes = [ctypes.POINTER(Cache), i32, i32, i32, i32]
            lib.kda_cache_attend_sinks.restype = ctypes.c_int
            lib.kda_cache_attend_sinks.argtypes = [ctypes.POINTER(Cache), _P, i64, i32, i32, _P, i64, i32, _P, i32, i32,
                                                   ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P]
            lib.kda_cache_attend_sinks_workspace_bytes.restype = ctypes.c_size_t
            lib.kda_cache_attend_sinks_workspace_bytes.argtypes = [ctypes.POINTER(Cache), i32, i32, i32, i32, i32]
            lib.kda_cache8_append.restype = ctypes.c_int
            lib.kda_cache8_append.argtypes = [ctypes.POINTER(Cache8)] + lib.kda_cache_append.argtypes[1:]
            lib.kda_cache_append_granted.restype = lib.kda_cache8_append_granted.restype = ctypes.c_int
            lib.kda_cache_append_granted.argtypes = lib.kda_cache_append.argtypes[:-2] + [_P, _P, _P]
            lib.kda_cache8_append_granted.argtypes = lib.kda_cache8_append.argtypes[:-2] + [_P, _P, _P]
            lib.kda_cache8_attend.restype = ctypes.c_int
            lib.kda_cache8_attend.argtypes = [ctypes.POINTER(Cache8)] + lib.kda_cache_attend_sinks.argtypes[1:]
            lib.kda_cache8_attend_workspace_bytes.restype = ctypes.c_size_t
            lib.kda_cache8_attend_workspace_bytes.argtypes = [ctypes.POINTER(Cache8), i32, i32, i32, i32, i32]
            lib.kda_cache_resize.restype = ctypes.c_int
            lib.kda_cache_resize.argtypes = [_P, i64, i32, i32, i32, _P, _P, _P, i32, _P, _P, _P, i64, _P, _P, _P,
                                             ctypes.c_size_t, _P]
            lib.kda_cache_resize_workspace_bytes.restype = ctypes.c_size_t
            lib.kda_cache_resize_workspace_bytes.argtypes = [i32, i32, i64]
            _lib = lib
    return _lib


def _check(code, where):
    if code != 0:
        raise KdaError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def prepare_chunks(cu_seqlens):
    """Host chunk table of packed sequences: (chunk_idx int32 [NT, 2], chunk_off int64 [N+1], NT), CPU tensors."""
    lib = load()
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int64).cpu().contiguous()
    N = cu.numel() - 1
    nt = ctypes.c_int64(0)
    _check(lib.kda_prepare_chunks(_ptr(cu), N, CHUNK, None, None, ctypes.byref(nt)), "kda_prepare_chunks")
    idx = torch.empty(max(nt.value, 1), 2, dtype=torch.int32)
    off = torch.empty(N + 1, dtype=torch.int64)
    _check(lib.kda_prepare_chunks(_ptr(cu), N, CHUNK, _ptr(idx), _ptr(off), ctypes.byref(nt)), "kda_prepare_chunks")
    return idx[:nt.value], off, nt.value


def make_dims(q: torch.Tensor, v: torch.Tensor, scale: Optional[float], cu_seqlens=None) -> Dims:
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    if q.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif q.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if cu_seqlens is None:
        N, NT = B, B * ((T + CHUNK - 1) // CHUNK)
    else:
        cu = torch.as_tensor(cu_seqlens).cpu().tolist()
        N = len(cu) - 1
        NT = sum((cu[i + 1] - cu[i] + CHUNK - 1) // CHUNK for i in range(N))
    return Dims(B, T, H, HV, K, V, CHUNK, N, NT, dt, float(K ** -0.5 if scale is None else scale))


def workspace_bytes(dims: Dims, which: int) -> int:
    return int(load().kda_workspace_bytes(ctypes.byref(dims), which))


class _Varlen:
    """Device copies of cu_seqlens and its chunk table."""

    def __init__(self, cu_seqlens, device):
        if cu_seqlens is None:
            self.cu = self.idx = self.off = None
            return
        idx, off, _ = prepare_chunks(cu_seqlens)
        self.cu = torch.as_tensor(cu_seqlens, dtype=torch.int64).to(device).contiguous()
        self.idx = idx.to(device).contiguous()
        self.off = off.to(device).contiguous()


def _req(t, name, dtype=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _opt(t, name, dtype=None):
    return None if t is None else _req(t, name, dtype)


def _workspace(dims, which, device, ws):
    need = workspace_bytes(dims, which)
    if need == 0:
        raise KdaError(1, "kda_workspace_bytes")
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws


def chunk_fwd(q, k, v, g, beta, scale=None, h0=None, cu_seqlens=None, output_states=False, ws=None):
    """Chunked KDA forward. Returns (o, ht, states); states is [num_chunks, HV, K, V] fp32 when
    ``output_states`` (the state entering every chunk, for a backward that skips the recompute), else None."""
    lib = load()
    dt = q.dtype
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _req(t, n, dt)
    _req(g, "g", torch.float32)
    _opt(h0, "h0", torch.float32)
    dims = make_dims(q, v, scale, cu_seqlens)
    dev = q.device
    vl = _Varlen(cu_seqlens, dev)
    o = torch.empty_like(v)
    ht = torch.empty(dims.num_seqs, dims.HV, dims.K, dims.V, dtype=torch.float32, device=dev)
    states = (torch.empty(dims.num_chunks, dims.HV, dims.K, dims.V, dtype=torch.float32, device=dev)
              if output_states else None)
    ws = _workspace(dims, PASS_FWD, dev, ws)
    _check(lib.kda_chunk_fwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                             _ptr(vl.cu), _ptr(vl.idx), _ptr(vl.off), _ptr(o), _ptr(ht), _ptr(states), _ptr(ws),
                             ws.numel(), _stream()), "kda_chunk_fwd")
    return o, ht, states


def chunk_bwd(q, k, v, g, beta, do, scale=None, h0=None, dht=None, cu_seqlens=None, states=None, ws=None,
              out=None):
    """Chunked KDA backward (recomputes the forward state pass unless ``states`` is given).

    Returns a dict with dq, dk ([B,T,H,K]), dv, dg (fp32), dbeta and dh0
    (fp32, or None without h0). ``out`` may pass preallocated outputs."""
    return _chunk_bwd("kda_chunk_bwd", q, k, v, g, beta, do, scale, h0, dht, cu_seqlens, states, ws, out)


def chunk_bwd_fused(q, k, v, g, beta, do, scale=None, h0=None, dht=None, cu_seqlens=None, states=None, ws=None,
                    out=None):
    """As :func:`chunk_bwd` through ``kda_chunk_bwd_fused`` (the reverse pass and the per-chunk gradients in
    one launch; bf16, K = V = 128, H == HV)."""
    return _chunk_bwd("kda_chunk_bwd_fused", q, k, v, g, beta, do, scale, h0, dht, cu_seqlens, states, ws, out)


def _chunk_bwd(entry, q, k, v, g, beta, do, scale, h0, dht, cu_seqlens, states, ws, out):
    lib = load()
    dt = q.dtype
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (do, "do")):
        _req(t, n, dt)
    _req(g, "g", torch.float32)
    _opt(h0, "h0", torch.float32)
    _opt(dht, "dht", torch.float32)
    _opt(states, "states", torch.float32)
    dims = make_dims(q, v, scale, cu_seqlens)
    dev = q.device
    vl = _Varlen(cu_seqlens, dev)
    if out is None:
        out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                   dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
                   dh0=torch.empty_like(h0) if h0 is not None else None)
    ws = _workspace(dims, PASS_BWD, dev, ws)
    _check(getattr(lib, entry)(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                _ptr(vl.cu), _ptr(vl.idx), _ptr(vl.off), _ptr(do), _ptr(dht), _ptr(states),
                                _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                                _ptr(out["dbeta"]), _ptr(out.get("dh0")), _ptr(ws), ws.numel(), _stream()), entry)
    return out


def saved_bytes(dims: Dims) -> int:
    return int(load().kda_saved_bytes(ctypes.byref(dims)))


def chunk_fwd_save(q, k, v, g, beta, scale=None, h0=None, cu_seqlens=None):
    """Forward that also keeps the saved context for chunk_bwd_from_saved (bf16, K = V = 128).
    Returns (o, ht, saved); saved is a uint8 device tensor of saved_bytes(dims)."""
    lib = load()
    dt = q.dtype
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _req(t, n, dt)
    _req(g, "g", torch.float32)
    _opt(h0, "h0", torch.float32)
    dims = make_dims(q, v, scale, cu_seqlens)
    dev = q.device
    vl = _Varlen(cu_seqlens, dev)
    need = saved_bytes(dims)
    if need == 0:
        raise KdaError(2, "kda_saved_bytes")
    saved = torch.empty(need, dtype=torch.uint8, device=dev)
    o = torch.empty_like(v)
    ht = torch.empty(dims.num_seqs, dims.HV, dims.K, dims.V, dtype=torch.float32, device=dev)
    _check(lib.kda_chunk_fwd_save(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                  _ptr(vl.cu), _ptr(vl.idx), _ptr(vl.off), _ptr(o), _ptr(ht), _ptr(saved),
                                  saved.numel(), _stream()), "kda_chunk_fwd_save")
    return o, ht, saved


def chunk_bwd_from_saved(q, k, v, g, beta, do, saved, scale=None, h0=None, dht=None, cu_seqlens=None, out=None):
    """Backward from chunk_fwd_save's context: only the reverse pass and the per-chunk gradients run.
    Same returns as chunk_bwd, and the same values bit for bit."""
    lib = load()
    dt = q.dtype
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (do, "do")):
        _req(t, n, dt)
    _req(g, "g", torch.float32)
    _opt(h0, "h0", torch.float32)
    _opt(dht, "dht", torch.float32)
    _req(saved, "saved", torch.uint8)
    dims = make_dims(q, v, scale, cu_seqlens)
    vl = _Varlen(cu_seqlens, q.device)
    if out is None:
        out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                   dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
                   dh0=torch.empty_like(h0) if h0 is not None else None)
    _check(lib.kda_chunk_bwd_from_saved(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                        _ptr(vl.cu), _ptr(vl.idx), _ptr(vl.off), _ptr(do), _ptr(dht), _ptr(saved),
                                        saved.numel(), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                        _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out.get("dh0")), _stream()),
           "kda_chunk_bwd_from_saved")
    return out


def device_status(ws: torch.Tensor) -> int:
    """Status word of the last call that used workspace ``ws`` (syncs the current stream)."""
    return int(load().kda_device_status(_ptr(ws), _stream()))


# ------------------------------------------------------------------ single tokens (include/kda_serve.h)


_serve_module = None


def _serve():
    """The compiled binding of these operators (raises if the library has not been built)."""
    global _serve_module
    if _serve_module is None:
        load()
        if not os.path.exists(SERVE):
            raise RuntimeError(f"KDA single-token module not built ({SERVE}); call chunked_gated_delta_10_gb300.build() with "
                               "a PyTorch with CUDA and Python's headers")
        spec = importlib.util.spec_from_file_location("_kda_serve", SERVE)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _serve_module = module
    return _serve_module


def step(q, k, v, g, beta, state, scale=None, slots=None, out=None, status=None):
    """T new tokens (one, or a few) per sequence through the KDA recurrence; ``state`` is updated in place.

    q, k [N,T,H,K], v [N,T,HV,V], g [N,T,HV,K] fp32, beta [N,T,HV] as in :func:`chunk_fwd`; ``state``
    [slots,HV,K,V] fp32 (:func:`chunk_fwd`'s ht is one). ``slots`` (int32 [N]) names each sequence's state, a
    negative one marks an inactive row; without it sequence n has state[n]. Returns o [N,T,HV,V] (``out``, if
    given). ``status`` (int32 [1], zeroed by the caller) is set where a slot does not exist."""
    r = (_serve_module or _serve()).step(q, k, v, g, beta, state, scale, slots, out, status)
    if type(r) is int:
        raise KdaError(r, "kda_step")
    return r


def new_cache(num_pages, page_size, heads, K, V, dtype=torch.bfloat16, device="cuda", scale_block=None):
    """An empty paged cache (k_cache [num_pages, page_size, heads, K], v_cache likewise with V), each head's rows
    of a page contiguous: the layout that :func:`cache_attend` reads in the longest runs.

    With ``dtype`` torch.float8_e4m3fn a cache in 8 bits, and the scales of its blocks of ``scale_block`` rows (which
    divide a page; without it 16, or a page that 16 does not divide): (k_cache, v_cache, k_scale, v_scale), scales fp32
    [num_pages, page_size / scale_block, heads]."""
    pair = tuple(torch.zeros(num_pages, heads, page_size, d, dtype=dtype, device=device).transpose(1, 2) for d in (K, V))
    if dtype != torch.float8_e4m3fn:
        if scale_block is not None:
            raise ValueError("scale_block is for a cache in float8_e4m3fn")
        return pair
    block = (16 if page_size % 16 == 0 else page_size) if scale_block is None else scale_block
    if block < 1 or page_size % block:
        raise ValueError(f"scale_block {block} does not divide the page size {page_size}")
    return pair + tuple(torch.zeros(num_pages, heads, page_size // block, device=device).transpose(1, 2) for _ in range(2))


def cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q=None, rope=None, interleaved=False, cu_seqlens=None,
                 q_out=None, status=None, k_scale=None, v_scale=None, granted=None):
    """Append new keys and values to a paged cache, keys (and queries) rotated by their position on the way.

    k [R,HKV,K], v [R,HKV,V] and q [R,HQ,K] hold the new rows of all sequences: R / N each, or as ``cu_seqlens``
    (int64 [N+1] on the device) says. k_cache, v_cache [pages, page_size, HKV, K or V], any strides with contiguous
    channels; ``page_table`` int32 [N, max_pages]; ``kv_lens`` int32 [N], the rows already there (not changed;
    negative: inactive). ``rope`` fp32 [positions, r]: r/2 cosines, then r/2 sines; channel i turns with i + r/2, or,
    ``interleaved``, 2i with 2i+1. Returns the rotated queries (``q_out``, if given), or None without q.
    ``status`` (int32 [1], zeroed by the caller) is set where a page or position does not exist, or a row lies in
    no sequence of ``cu_seqlens``. ``granted`` (int32 [N], as :func:`cache_resize` returns it) are lengths up to which rows
    are appended: those beyond are dropped, and their queries are 0, as in an inactive sequence.

    A cache in torch.float8_e4m3fn has ``k_scale`` and ``v_scale`` beside it (fp32 [pages, blocks, HKV], any strides; see
    :func:`new_cache`): a row is stored in units of its block's scale, the smallest power of two by which the block's
    values come to 448 at most. A block that has rows already is written again where its scale has to grow. The rows are
    bf16 or fp32 then, whichever k is, and the queries too."""
    r = (_serve_module or _serve()).append(k, v, k_cache, v_cache, page_table, kv_lens, q, rope, interleaved, cu_seqlens,
                                           q_out, status, k_scale, v_scale, granted)
    if type(r) is int:
        raise KdaError(r, "kda_cache_append")
    return r


def cache_attend(q, k_cache, v_cache, page_table, kv_lens, scale=None, window=0, ws=None, out=None, status=None, sinks=0,
                 k_scale=None, v_scale=None):
    """Attention of one new token per sequence over its cached rows: all of them, or, if ``window`` is positive, the last
    ``window`` of them and the first ``sinks``.

    q [N,HQ,K]; the cache, ``page_table`` and ``status`` as in :func:`cache_append`; ``kv_lens`` int32 [N], the
    rows to attend, the new token's own among them (none: o is 0 and lse -inf). Returns (o [N,HQ,V], lse fp32
    [N,HQ]): new tensors, or ``out`` as o. ``ws`` (contiguous uint8) is scratch memory, of
    :func:`cache_attend_workspace_bytes` bytes or more; without it, or with less, the call allocates its own for as
    long as it takes. What it holds does not matter, but two calls that may overlap on the GPU cannot share one.

    ``k_scale`` and ``v_scale`` are those of a cache in 8 bits, as in :func:`cache_append`; q, in bf16 or fp32, says o's
    type then."""
    r = (_serve_module or _serve()).attend(q, k_cache, v_cache, page_table, kv_lens, scale, window, ws, out, status, sinks,
                                           k_scale, v_scale)
    if type(r) is int:
        raise KdaError(r, "kda_cache_attend")
    return r


def cache_attend_workspace_bytes(q, k_cache, v_cache, page_table, window=0, sinks=0) -> int:
    """Bytes of ``ws`` that :func:`cache_attend` wants for these tensors (their sizes count, and the device)."""
    (N, max_pages), HQ = page_table.shape, q.shape[1]
    pages, rows, heads, K = k_cache.shape
    dtypes = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32, torch.float8_e4m3fn: DTYPE_E4M3}
    for t, n in ((k_cache, "k_cache"), (q, "q")):
        if t.dtype not in dtypes and (t is k_cache or k_cache.dtype == torch.float8_e4m3fn):  # (else q's says nothing)
            raise TypeError(f"unsupported dtype {t.dtype} of {n}")
    strides = [s if n > 1 else 0 for t in (k_cache, v_cache) for n, s in zip(t.shape[:3], t.stride())]
    c = Cache(k_cache.data_ptr(), v_cache.data_ptr(), *strides, pages, rows, heads, K, v_cache.shape[3], dtypes[k_cache.dtype])
    with torch.cuda.device(k_cache.device):
        if k_cache.dtype == torch.float8_e4m3fn:  # (where the scales are does not count)
            c8 = Cache8(c, k_cache.data_ptr(), v_cache.data_ptr(), 0, 0, 0, 0, 0, 0, 1, dtypes[q.dtype])
            need = int(load().kda_cache8_attend_workspace_bytes(ctypes.byref(c8), HQ, N, max_pages, window, sinks))
        else:
            need = int(load().kda_cache_attend_sinks_workspace_bytes(ctypes.byref(c), HQ, N, max_pages, window, sinks))
    if need == 0:
        raise KdaError(1, "kda_cache_attend_workspace_bytes")
    return need


def cache_resize(page_table, kv_lens, new_lens, free_pages, free_count, page_size, rows=0, status=None):
    """Pages for new lengths: a paged cache's table brought from ``kv_lens`` to ``new_lens`` rows, on the GPU alone.

    ``page_table`` int32 [N, max_pages], changed in place: entries that ``new_lens`` (int32 [N]) needs beyond those of
    ``kv_lens`` (int32 [N]; negative: none) are filled, entries that it does not need become -1. The pages come from the
    end of ``free_pages`` (int32 [pages of the cache]), of which the first ``free_count`` (int32 [1]) are free, and go to
    it: all that go back first, so that they can be taken in the same call. A sequence whose pages, after those of the
    sequences before it, are not there gets none.

    Returns (cu_seqlens int64 [N+1], slots int64 [``rows``], granted int32 [N]): the new rows' offsets as
    :func:`cache_append` takes them (with ``granted``: the rows of a sequence that was not served have offsets too); where
    each new row goes, its page times ``page_size`` plus its row in the page, or -1 (of a sequence that was not served, and
    behind the last new row), for kernels of one's own; and each sequence's length now, ``new_lens`` or, not served,
    ``kv_lens``. ``status`` (int32 [1], zeroed by the caller) is set where a sequence is not served, an entry is no page,
    or the new rows are more than ``rows``, if that is not 0."""
    r = (_serve_module or _serve()).resize(page_table, kv_lens, new_lens, free_pages, free_count, page_size, rows, status)
    if type(r) is int:
        raise KdaError(r, "kda_cache_resize")
    return r
