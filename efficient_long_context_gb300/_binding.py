"""ctypes binding of include/orthros_attn.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

ORTHROS_BF16 = 0
ORTHROS_F32 = 1
_DTYPES = {torch.bfloat16: ORTHROS_BF16, torch.float32: ORTHROS_F32}

STATUS_NAMES = {0: "ORTHROS_OK", 1: "ORTHROS_EINVAL", 2: "ORTHROS_EUNSUPPORTED", 3: "ORTHROS_ECUDA",
                4: "ORTHROS_EWORKSPACE", 5: "ORTHROS_EDEVICE", 6: "ORTHROS_ETIMEOUT"}

# the public symbols of include/orthros_attn.h
EXPORTS = ("orthros_prefill_workspace_size", "orthros_prefill", "orthros_prefill_from_host_workspace_size",
           "orthros_prefill_from_host", "orthros_prefill_shard_workspace_size",
           "orthros_prefill_shard", "orthros_merge_partials", "orthros_prefill_backward_workspace_size",
           "orthros_prefill_backward", "orthros_extend_workspace_size", "orthros_extend", "orthros_qkv_project",
           "orthros_decode_workspace_size",
           "orthros_decode", "orthros_decode_static", "orthros_rotary_frequencies", "orthros_rotary_steps",
           "orthros_rotate", "orthros_rotate_backward_workspace_size", "orthros_rotate_backward",
           "orthros_rotate_append", "orthros_chunk_attention_workspace_size", "orthros_chunk_attention",
           "orthros_check", "orthros_profile_begin", "orthros_profile_end",
           "orthros_selftest_wait_timeout", "orthros_status_string", "orthros_last_error")


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double)]


class OrthrosError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load_library(path: str | None = None):
    """Load liborthros_attn.so (built by efficient_long_context_gb300.build)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            raise OrthrosError(-1, f"{p} is missing: run efficient_long_context_gb300.build.build() first "
                                   "(there is no fallback path)")
        lib = ctypes.CDLL(p)
        vp, i32, f32p, i32p, sz = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_float), \
            ctypes.POINTER(ctypes.c_int32), ctypes.c_size_t
        lib.orthros_prefill_workspace_size.restype = sz
        lib.orthros_prefill_workspace_size.argtypes = [i32] * 7 + [i32]
        lib.orthros_prefill.restype = i32
        lib.orthros_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32p, vp, i32, vp,
                                        i32, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                        vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]
        lib.orthros_prefill_from_host_workspace_size.restype = sz
        lib.orthros_prefill_from_host_workspace_size.argtypes = [i32] * 8
        lib.orthros_prefill_from_host.restype = i32
        lib.orthros_prefill_from_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32p, i32p, i32, vp,
                                                  i32, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                                  vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]
        lib.orthros_prefill_shard_workspace_size.restype = sz
        lib.orthros_prefill_shard_workspace_size.argtypes = [i32] * 9
        lib.orthros_prefill_shard.restype = i32
        lib.orthros_prefill_shard.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32p, vp, i32, vp,
                                              i32, i32, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                              vp, vp, vp, vp, vp, sz, vp]
        lib.orthros_merge_partials.restype = i32
        lib.orthros_merge_partials.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
        lib.orthros_prefill_backward_workspace_size.restype = sz
        lib.orthros_prefill_backward_workspace_size.argtypes = [i32] * 8
        lib.orthros_prefill_backward.restype = i32
        lib.orthros_prefill_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32p, vp, i32, vp,
                                                 i32, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                                 vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                 vp, sz, vp]
        lib.orthros_extend_workspace_size.restype = sz
        lib.orthros_extend_workspace_size.argtypes = [i32] * 9
        lib.orthros_extend.restype = i32
        lib.orthros_extend.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32p, i32p, vp,
                                       vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                       vp, vp, vp, vp, vp, sz, vp]
        lib.orthros_qkv_project.restype = i32
        lib.orthros_qkv_project.argtypes = [vp, i32, i32, i32, vp, i32, i32, i32, vp, vp, vp, vp,
                                            vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, i32,
                                            vp, sz, vp]
        lib.orthros_decode_workspace_size.restype = sz
        lib.orthros_decode_workspace_size.argtypes = [i32] * 7
        lib.orthros_decode.restype = i32
        lib.orthros_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp,
                                       vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                       vp, vp, vp, vp, vp, sz, vp]
        lib.orthros_decode_static.restype = i32
        lib.orthros_decode_static.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp,
                                              vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                              vp, vp, vp, vp, vp]
        ll, f32, f64, u64 = ctypes.c_longlong, ctypes.c_float, ctypes.c_double, ctypes.c_uint64
        lib.orthros_rotary_frequencies.restype = i32
        lib.orthros_rotary_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, ctypes.POINTER(f64),
                                                   ctypes.POINTER(f32)]
        lib.orthros_rotary_steps.restype = i32
        lib.orthros_rotary_steps.argtypes = [ctypes.POINTER(f64), i32, ctypes.POINTER(u64)]
        lib.orthros_rotate.restype = i32
        lib.orthros_rotate.argtypes = [vp, ll, vp, vp, vp, vp, i32, i32, f32, i32, i32, i32, i32, vp, ll, vp]
        lib.orthros_rotate_backward_workspace_size.restype = sz
        lib.orthros_rotate_backward_workspace_size.argtypes = [i32] * 4
        lib.orthros_rotate_backward.restype = i32
        lib.orthros_rotate_backward.argtypes = [vp, ll, vp, ll, vp, vp, vp, i32, i32, f32, i32, i32, i32, i32, vp, ll,
                                                vp, vp, vp, sz, vp]
        lib.orthros_rotate_append.restype = i32
        lib.orthros_rotate_append.argtypes = [vp, ll, vp, ll, vp, ll, vp, ll, vp, vp, vp, vp, vp, i32, i32, f32, vp, vp,
                                              vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                              vp, sz, vp]
        lib.orthros_chunk_attention_workspace_size.restype = sz
        lib.orthros_chunk_attention_workspace_size.argtypes = [i32] * 9
        lib.orthros_chunk_attention.restype = i32
        lib.orthros_chunk_attention.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32,
                                                i32, i32, i32, vp, vp, vp, sz, vp]
        lib.orthros_selftest_wait_timeout.restype = i32
        lib.orthros_selftest_wait_timeout.argtypes = [ctypes.c_longlong, vp, sz, vp]
        lib.orthros_check.restype = i32
        lib.orthros_check.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.orthros_profile_begin.restype = i32
        lib.orthros_profile_begin.argtypes = []
        lib.orthros_profile_end.restype = i32
        lib.orthros_profile_end.argtypes = [ctypes.POINTER(KernelTime), i32]
        lib.orthros_status_string.restype = ctypes.c_char_p
        lib.orthros_status_string.argtypes = [i32]
        lib.orthros_last_error.restype = ctypes.c_char_p
        lib.orthros_last_error.argtypes = []
        del f32p
        if path is None:
            _lib = lib
        return lib


def orthros_status_string(status: int) -> str:
    return load_library().orthros_status_string(int(status)).decode()


def orthros_last_error() -> str:
    return load_library().orthros_last_error().decode()


def _raise_if(rc: int, lib):
    if rc != 0:
        raise OrthrosError(rc, lib.orthros_last_error().decode())


def _ptr(t):
    """Device address of a tensor argument. Every tensor the library reads or
    writes must live on the current CUDA device: a host tensor's address
    handed to a kernel would make it read host memory. Raised here, while the
    call's arguments are marshalled, so nothing is launched."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.is_cuda or t.device.index != torch.cuda.current_device():
            raise OrthrosError(1, f"tensor on {t.device}: every tensor argument must be on the current CUDA device")
        return ctypes.c_void_p(t.data_ptr()) if t.numel() else ctypes.c_void_p(0)
    return t


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise OrthrosError(1, f"unsupported element type {t.dtype}")
    return _DTYPES[t.dtype]


def _contig(name, t):
    if t is not None and not t.is_contiguous():
        raise OrthrosError(1, f"{name} must be contiguous")
    return t


def orthros_prefill_workspace_size(B, T, Hq, Hkv, d, n_out, window, dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_prefill_workspace_size(B, T, Hq, Hkv, d, n_out, window, _DTYPES[dtype]))


def orthros_decode_workspace_size(B, Hq, Hkv, d, max_pages, page_size, dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_decode_workspace_size(B, Hq, Hkv, d, max_pages, page_size, _DTYPES[dtype]))


def orthros_prefill(q, k, v, alpha_base, beta_base, alpha_out, beta_out, out_indptr, out_positions,
                    window, scale=None, *, q_out=None, out=None, k_cache=None, v_cache=None,
                    block_table=None, page_size=0, workspace=None, stream=None):
    """orthros_prefill of include/orthros_attn.h on torch CUDA tensors.

    out_indptr is a HOST int32 array-like [B+1]; every other tensor lives on
    the GPU. Returns (o_base [B,T,Hq,d], lse_base [B,Hq,T], o_out [n_out,Hq,d],
    lse_out [n_out,Hq]), allocated here unless `out` gives all four.
    """
    lib = load_library()
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    indptr = np.ascontiguousarray(np.asarray(out_indptr.cpu() if isinstance(out_indptr, torch.Tensor)
                                             else out_indptr, dtype=np.int32))
    n_out = int(indptr[-1]) if indptr.size else 0
    if scale is None:
        scale = d ** -0.5
    for name, t in (("q", q), ("k", k), ("v", v), ("q_out", q_out), ("out_positions", out_positions)):
        _contig(name, t)
    if out is None:
        o_base = torch.empty_like(q)
        lse_base = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
        o_out = torch.empty((n_out, Hq, d), dtype=q.dtype, device=q.device)
        lse_out = torch.empty((n_out, Hq), dtype=torch.float32, device=q.device)
    else:
        o_base, lse_base, o_out, lse_out = out
    if workspace is None:
        ws = orthros_prefill_workspace_size(B, T, Hq, Hkv, d, n_out, window, q.dtype)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=q.device)
    max_pages = block_table.shape[1] if block_table is not None else 0
    num_pages = k_cache.shape[0] if k_cache is not None else 0
    rc = lib.orthros_prefill(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out), _ptr(beta_out),
        indptr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), _ptr(out_positions), n_out, _ptr(q_out),
        B, T, Hq, Hkv, d, int(window), float(scale), _dtype(q),
        _ptr(o_base), _ptr(lse_base), _ptr(o_out), _ptr(lse_out),
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), max_pages, int(page_size), num_pages,
        _ptr(workspace), workspace.numel(), _stream(stream))
    _raise_if(rc, lib)
    return o_base, lse_base, o_out, lse_out


def _host_ptr(t):
    """Host address of a CPU tensor argument of orthros_prefill_from_host."""
    if t is None:
        return None
    if t.is_cuda:
        raise OrthrosError(1, "orthros_prefill_from_host takes its inputs and outputs in host memory")
    _contig("host tensor", t)
    return ctypes.c_void_p(t.data_ptr())


def orthros_prefill_from_host_workspace_size(B, T, Hq, Hkv, d, n_out, window, dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_prefill_from_host_workspace_size(B, T, Hq, Hkv, d, n_out, window,
                                                                       _DTYPES[dtype]))


def orthros_prefill_from_host(q, k, v, alpha_base, beta_base, alpha_out, beta_out, out_indptr, out_positions,
                              window, scale=None, *, q_out=None, out=None, k_cache=None, v_cache=None,
                              block_table=None, page_size=0, workspace=None, stream=None):
    """orthros_prefill_from_host of include/orthros_attn.h.

    q, k, v, out_positions, q_out and the outputs are CPU tensors (pinned, for
    copies that overlap the compute); the affines, the optional cache and the
    workspace are CUDA tensors. Returns (o_base, lse_base, o_out, lse_out) as
    CPU tensors, allocated here (pinned) unless `out` gives all four. The
    outputs are complete once `stream` has passed this call.
    """
    lib = load_library()
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    indptr = np.ascontiguousarray(np.asarray(out_indptr.cpu() if isinstance(out_indptr, torch.Tensor)
                                             else out_indptr, dtype=np.int32))
    n_out = int(indptr[-1]) if indptr.size else 0
    pos = np.ascontiguousarray(np.asarray(out_positions.cpu() if isinstance(out_positions, torch.Tensor)
                                          else out_positions, dtype=np.int32))
    if scale is None:
        scale = d ** -0.5
    if out is None:
        pin = torch.cuda.is_available()
        o_base = torch.empty(q.shape, dtype=q.dtype, pin_memory=pin)
        lse_base = torch.empty((B, Hq, T), dtype=torch.float32, pin_memory=pin)
        o_out = torch.empty((n_out, Hq, d), dtype=q.dtype, pin_memory=pin)
        lse_out = torch.empty((n_out, Hq), dtype=torch.float32, pin_memory=pin)
    else:
        o_base, lse_base, o_out, lse_out = out
    dev = alpha_base.device
    if workspace is None:
        ws = orthros_prefill_from_host_workspace_size(B, T, Hq, Hkv, d, n_out, window, q.dtype)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
    max_pages = block_table.shape[1] if block_table is not None else 0
    num_pages = k_cache.shape[0] if k_cache is not None else 0
    rc = lib.orthros_prefill_from_host(
        _host_ptr(q), _host_ptr(k), _host_ptr(v), _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out),
        _ptr(beta_out), indptr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
        pos.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) if n_out else None, n_out, _host_ptr(q_out),
        B, T, Hq, Hkv, d, int(window), float(scale), _dtype(q),
        _host_ptr(o_base), _host_ptr(lse_base), _host_ptr(o_out) if n_out else None,
        _host_ptr(lse_out) if n_out else None,
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), max_pages, int(page_size), num_pages,
        _ptr(workspace), workspace.numel(), _stream(stream))
    _raise_if(rc, lib)
    return o_base, lse_base, o_out, lse_out


def orthros_prefill_shard_workspace_size(B, Tq, Tkv, Hq, Hkv, d, n_rows, window, dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_prefill_shard_workspace_size(B, Tq, Tkv, Hq, Hkv, d, n_rows, window,
                                                                   _DTYPES[dtype]))


def orthros_prefill_shard(q, k, v, alpha_base, beta_base, alpha_out, beta_out, row_indptr, row_positions,
                          window, scale=None, *, q_rows=None, out=None, workspace=None, stream=None):
    """orthros_prefill_shard of include/orthros_attn.h on torch CUDA tensors.

    q [B, Tq, Hq, d] (the chunk's queries), k, v [B, Tkv, Hkv, d] (halo then
    chunk); row_indptr is a HOST int32 array-like [B+1], row_positions [n_rows]
    int32 in the K/V buffer's coordinates, q_rows [n_rows, Hq, d]. Returns
    (o_base [B,Tq,Hq,d], lse_base [B,Hq,Tq], o_part [n_rows,Hq,d] float,
    lse_part [n_rows,Hq] float), allocated here unless `out` gives all four.
    """
    lib = load_library()
    B, Tq, Hq, d = q.shape
    Tkv, Hkv = k.shape[1], k.shape[2]
    indptr = np.ascontiguousarray(np.asarray(row_indptr.cpu() if isinstance(row_indptr, torch.Tensor)
                                             else row_indptr, dtype=np.int32))
    n_rows = int(indptr[-1]) if indptr.size else 0
    if scale is None:
        scale = d ** -0.5
    for name, t in (("q", q), ("k", k), ("v", v), ("q_rows", q_rows), ("row_positions", row_positions)):
        _contig(name, t)
    if out is None:
        out = (torch.empty_like(q), torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device),
               torch.empty((n_rows, Hq, d), dtype=torch.float32, device=q.device),
               torch.empty((n_rows, Hq), dtype=torch.float32, device=q.device))
    o_base, lse_base, o_part, lse_part = out
    if workspace is None:
        ws = orthros_prefill_shard_workspace_size(B, Tq, Tkv, Hq, Hkv, d, n_rows, window, q.dtype)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=q.device)
    rc = lib.orthros_prefill_shard(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out), _ptr(beta_out),
        indptr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), _ptr(row_positions), n_rows, _ptr(q_rows),
        B, Tq, Tkv, Hq, Hkv, d, int(window), float(scale), _dtype(q),
        _ptr(o_base), _ptr(lse_base), _ptr(o_part), _ptr(lse_part), _ptr(workspace), workspace.numel(),
        _stream(stream))
    _raise_if(rc, lib)
    return o_base, lse_base, o_part, lse_part


def orthros_merge_partials(o_parts, lse_parts, dtype=torch.bfloat16, *, out=None, stream=None):
    """orthros_merge_partials of include/orthros_attn.h: o_parts [P, n, Hq, d]
    float, lse_parts [P, n, Hq] float -> (o [n, Hq, d] of `dtype`, lse [n, Hq])."""
    lib = load_library()
    P, n, Hq, d = o_parts.shape
    for name, t in (("o_parts", o_parts), ("lse_parts", lse_parts)):
        _contig(name, t)
    if out is None:
        out = (torch.empty((n, Hq, d), dtype=dtype, device=o_parts.device),
               torch.empty((n, Hq), dtype=torch.float32, device=o_parts.device))
    o, lse = out
    rc = lib.orthros_merge_partials(_ptr(o_parts), _ptr(lse_parts), P, n, Hq, d, _DTYPES[o.dtype], _ptr(o), _ptr(lse),
                                    _stream(stream))
    _raise_if(rc, lib)
    return o, lse


def orthros_prefill_backward_workspace_size(B, T, Hq, Hkv, d, n_out, window, dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_prefill_backward_workspace_size(B, T, Hq, Hkv, d, n_out, window,
                                                                      _DTYPES[dtype]))


def orthros_prefill_backward(q, k, v, alpha_base, beta_base, alpha_out, beta_out, out_indptr, out_positions,
                             window, scale, o_base, lse_base, o_out, lse_out, do_base, do_out, *, q_out=None,
                             out=None, workspace=None, stream=None):
    """orthros_prefill_backward of include/orthros_attn.h on torch CUDA tensors.

    Returns a dict with dq, dk, dv, dq_out (None without q_out), d_alpha_base,
    d_beta_base, d_alpha_out, d_beta_out; allocated here unless `out` (a dict
    with the same keys) gives them.
    """
    lib = load_library()
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    indptr = np.ascontiguousarray(np.asarray(out_indptr.cpu() if isinstance(out_indptr, torch.Tensor)
                                             else out_indptr, dtype=np.int32))
    n_out = int(indptr[-1]) if indptr.size else 0
    if scale is None:
        scale = d ** -0.5
    for name, t in (("q", q), ("k", k), ("v", v), ("q_out", q_out), ("out_positions", out_positions),
                    ("o_base", o_base), ("o_out", o_out), ("do_base", do_base), ("do_out", do_out)):
        _contig(name, t)
    if out is None:
        dev = q.device
        out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
               "dq_out": torch.empty_like(q_out) if q_out is not None else None}
        for n in ("d_alpha_base", "d_beta_base", "d_alpha_out", "d_beta_out"):
            out[n] = torch.empty((Hq, d), dtype=torch.float32, device=dev)
    if workspace is None:
        ws = orthros_prefill_backward_workspace_size(B, T, Hq, Hkv, d, n_out, window, q.dtype)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=q.device)
    rc = lib.orthros_prefill_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out), _ptr(beta_out),
        indptr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), _ptr(out_positions), n_out, _ptr(q_out),
        B, T, Hq, Hkv, d, int(window), float(scale), _dtype(q),
        _ptr(o_base), _ptr(lse_base), _ptr(o_out), _ptr(lse_out), _ptr(do_base), _ptr(do_out),
        _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dq_out"]),
        _ptr(out["d_alpha_base"]), _ptr(out["d_beta_base"]), _ptr(out["d_alpha_out"]), _ptr(out["d_beta_out"]),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _raise_if(rc, lib)
    return out


def orthros_extend_workspace_size(B, n_new, n_out, Hq, Hkv, d, max_pages, page_size, dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_extend_workspace_size(B, n_new, n_out, Hq, Hkv, d, max_pages, page_size,
                                                            _DTYPES[dtype]))


def orthros_extend(q, k_new, v_new, k_cache, v_cache, block_table, cache_lens, new_indptr, out_indptr,
                   out_positions, alpha_base, beta_base, alpha_out, beta_out, window, scale=None, *, q_out=None,
                   out=None, workspace=None, stream=None):
    """orthros_extend of include/orthros_attn.h on torch CUDA tensors.

    new_indptr / out_indptr are HOST int32 array-likes [B+1]; k_cache /
    v_cache are updated in place. Returns (o_base [n_new,Hq,d], lse_base
    [n_new,Hq], o_out [n_out,Hq,d], lse_out [n_out,Hq]).
    """
    lib = load_library()
    n_new, Hq, d = q.shape
    Hkv = k_new.shape[1]
    num_pages, page_size = k_cache.shape[0], k_cache.shape[1]
    max_pages = block_table.shape[1]
    ni = np.ascontiguousarray(np.asarray(new_indptr, dtype=np.int32))
    oi = np.ascontiguousarray(np.asarray(out_indptr, dtype=np.int32))
    B = ni.shape[0] - 1
    n_out = int(oi[-1]) if oi.size else 0
    if scale is None:
        scale = d ** -0.5
    for name, t in (("q", q), ("q_out", q_out), ("k_new", k_new), ("v_new", v_new), ("out_positions", out_positions)):
        _contig(name, t)
    if out is None:
        out = (torch.empty_like(q), torch.empty((n_new, Hq), dtype=torch.float32, device=q.device),
               torch.empty((n_out, Hq, d), dtype=q.dtype, device=q.device),
               torch.empty((n_out, Hq), dtype=torch.float32, device=q.device))
    o_base, lse_base, o_out, lse_out = out
    if workspace is None:
        ws = orthros_extend_workspace_size(B, n_new, n_out, Hq, Hkv, d, max_pages, page_size, q.dtype)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=q.device)
    i32p = ctypes.POINTER(ctypes.c_int32)
    rc = lib.orthros_extend(
        _ptr(q), _ptr(q_out), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        max_pages, page_size, num_pages, _ptr(cache_lens), ni.ctypes.data_as(i32p), oi.ctypes.data_as(i32p),
        _ptr(out_positions), _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out), _ptr(beta_out),
        B, Hq, Hkv, d, int(window), float(scale), _dtype(q),
        _ptr(o_base), _ptr(lse_base), _ptr(o_out), _ptr(lse_out), _ptr(workspace), workspace.numel(), _stream(stream))
    _raise_if(rc, lib)
    return o_base, lse_base, o_out, lse_out


def orthros_qkv_project(x, n_base, w_qkv, Hq, Hkv, d, alpha_base, beta_base, alpha_out, beta_out, *,
                        kv_out=False, k_cache=None, v_cache=None, block_table=None, token_seq=None,
                        token_pos=None, out=None, workspace=None, stream=None):
    """orthros_qkv_project of include/orthros_attn.h on torch CUDA tensors.

    x [n_base + n_out, d_model] (base rows first), w_qkv [(Hq+2Hkv) d, d_model].
    Returns (q_base [n_base,Hq,d], q_out [n_out,Hq,d], k [n_base,Hkv,d] or None,
    v or None); the caches are written in place when given.
    """
    lib = load_library()
    rows, d_model = x.shape
    n_out = rows - int(n_base)
    for name, t in (("x", x), ("w_qkv", w_qkv)):
        _contig(name, t)
    if out is None:
        dev = x.device
        out = (torch.empty((n_base, Hq, d), dtype=x.dtype, device=dev),
               torch.empty((n_out, Hq, d), dtype=x.dtype, device=dev),
               torch.empty((n_base, Hkv, d), dtype=x.dtype, device=dev) if kv_out else None,
               torch.empty((n_base, Hkv, d), dtype=x.dtype, device=dev) if kv_out else None)
    q_b, q_o, k_o, v_o = out
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=x.device)
    max_pages = block_table.shape[1] if block_table is not None else 0
    B = block_table.shape[0] if block_table is not None else 0
    page_size = k_cache.shape[1] if k_cache is not None else 0
    num_pages = k_cache.shape[0] if k_cache is not None else 0
    rc = lib.orthros_qkv_project(
        _ptr(x), int(n_base), n_out, d_model, _ptr(w_qkv), Hq, Hkv, d,
        _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out), _ptr(beta_out),
        _ptr(q_b), _ptr(q_o), _ptr(k_o), _ptr(v_o), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), B,
        max_pages, page_size, num_pages, _ptr(token_seq), _ptr(token_pos), _dtype(x),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _raise_if(rc, lib)
    return out


def orthros_decode(q, k_new, v_new, k_cache, v_cache, block_table, cache_lens, alpha_base, beta_base,
                   alpha_out, beta_out, window, scale=None, *, q_out=None, out=None, workspace=None,
                   stream=None):
    """orthros_decode of include/orthros_attn.h on torch CUDA tensors.

    k_cache / v_cache [num_pages, page_size, Hkv, d] are updated in place.
    Returns (o_base [B,Hq,d], lse_base [B,Hq], o_out [B,Hq,d], lse_out [B,Hq]).
    """
    lib = load_library()
    B, Hq, d = q.shape
    Hkv = k_new.shape[1]
    num_pages, page_size = k_cache.shape[0], k_cache.shape[1]
    max_pages = block_table.shape[1]
    if scale is None:
        scale = d ** -0.5
    if out is None:
        o_base = torch.empty_like(q)
        o_out = torch.empty_like(q)
        lse_base = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        lse_out = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    else:
        o_base, lse_base, o_out, lse_out = out
    if workspace is None:
        ws = orthros_decode_workspace_size(B, Hq, Hkv, d, max_pages, page_size, q.dtype)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=q.device)
    rc = lib.orthros_decode(
        _ptr(q), _ptr(q_out), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        max_pages, page_size, num_pages, _ptr(cache_lens),
        _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out), _ptr(beta_out),
        B, Hq, Hkv, d, int(window), float(scale), _dtype(q),
        _ptr(o_base), _ptr(lse_base), _ptr(o_out), _ptr(lse_out),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _raise_if(rc, lib)
    return o_base, lse_base, o_out, lse_out


def orthros_decode_static(q, k_new, v_new, k_cache, v_cache, block_table, cache_lens, alpha_base, beta_base,
                          alpha_out, beta_out, window, scale=None, *, q_out=None, out=None, stream=None):
    """orthros_decode_static of include/orthros_attn.h: orthros_decode with the
    library's built-in scratch array instead of a caller workspace."""
    lib = load_library()
    B, Hq, d = q.shape
    Hkv = k_new.shape[1]
    num_pages, page_size = k_cache.shape[0], k_cache.shape[1]
    max_pages = block_table.shape[1]
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = (torch.empty_like(q), torch.empty((B, Hq), dtype=torch.float32, device=q.device),
               torch.empty_like(q), torch.empty((B, Hq), dtype=torch.float32, device=q.device))
    o_base, lse_base, o_out, lse_out = out
    rc = lib.orthros_decode_static(
        _ptr(q), _ptr(q_out), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        max_pages, page_size, num_pages, _ptr(cache_lens),
        _ptr(alpha_base), _ptr(beta_base), _ptr(alpha_out), _ptr(beta_out),
        B, Hq, Hkv, d, int(window), float(scale), _dtype(q),
        _ptr(o_base), _ptr(lse_base), _ptr(o_out), _ptr(lse_out), _stream(stream))
    _raise_if(rc, lib)
    return o_base, lse_base, o_out, lse_out


# The calls below are also made once per layer and decoding step on tensors of a
# few hundred KB, where the marshalling is what takes the time: one look-up of
# the current device and stream per call, plain integers for addresses.
def _here(t):
    """(device that every tensor of the call has to be on, its current stream's handle):
    the current CUDA device, for a call whose main tensor is t. For a t elsewhere a
    device that no tensor is on, so that the call is refused while it is marshalled."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        return -2, None
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _on(stream):
    """Context in which the caller's stream is the current one: what a call allocates
    then belongs to the stream that writes it, and is not handed on before that is done."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _new(t, shape):
    """An uninitialised contiguous tensor of t's type on its device."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(shape, dtype=t.dtype, device=t.device)


def _elsewhere(t):
    return OrthrosError(1, f"tensor on {t.device}: every tensor argument must be on the current CUDA device")


def _addr(t, dev):
    """_ptr for a known current device: the address as an integer (None for no or no elements)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise _elsewhere(t)
    return t.data_ptr()


_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_SCALINGS = {"plain": 0, "linear": 1, "stretch": 2, "bands": 3, "bands_tempered": 4}


def _rope_layout(layout) -> int:
    if layout not in _ROPE_LAYOUTS:
        raise OrthrosError(1, f"rotary layout {layout!r}: one of {sorted(_ROPE_LAYOUTS)}")
    return _ROPE_LAYOUTS[layout]


def _rows(name, t, dev, dtype, shape):
    """(address, elements between tokens) of t [n, heads, d], whose tokens' heads must be contiguous."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype != dtype:
        raise OrthrosError(1, f"{name} must be a {dtype} {list(shape)} tensor, not {t.dtype} {list(t.shape)}")
    n, H, d = shape
    st = t.stride()
    if (st[2] != 1 or (H > 1 and st[1] != d)) and t.numel():
        raise OrthrosError(1, f"{name}: the heads of a token must be contiguous")
    if t.get_device() != dev:
        raise _elsewhere(t)
    return t.data_ptr(), st[0] if n > 1 else H * d


def _index(name, t, dev, n):
    """Address of a contiguous int32 index tensor of n entries."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous():
        raise OrthrosError(1, f"{name} must be a contiguous int32 tensor of {n} entries")
    if t.get_device() != dev:
        raise _elsewhere(t)
    return t.data_ptr()


def _block(name, t, dev, dtype, shape):
    """Address of a contiguous tensor of this type and shape."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise OrthrosError(1, f"{name} must be a contiguous {dtype} {list(shape)} tensor")
    if t.get_device() != dev:
        raise _elsewhere(t)
    return t.data_ptr()


def _steps(t, dev):
    """(address, rotated channels) of a vector of rotary steps."""
    if t.dtype != torch.int64 or t.dim() != 1 or not t.is_contiguous():
        raise OrthrosError(1, "steps must be a contiguous int64 vector (orthros_rotary_steps)")
    return _addr(t, dev), 2 * t.numel()


def orthros_rotary_frequencies(rot_dim, base, scaling="plain", *, factor=1.0, original_length=0.0, low_turns=1.0,
                               high_turns=4.0):
    """orthros_rotary_frequencies of include/orthros_attn.h: (freq float64 [rot_dim/2] CPU tensor, amplitude)
    of a scaling rule ("plain", "linear", "stretch", "bands", "bands_tempered").

    low_turns and high_turns bound the bands that are blended; their defaults, 1 and 4, are the
    published ones of "bands". YaRN, which "bands_tempered" follows, was published with 1 and
    32: give high_turns=32 for a model that was trained with it.
    """
    lib = load_library()
    if scaling not in _ROPE_SCALINGS:
        raise OrthrosError(1, f"scaling {scaling!r}: one of {sorted(_ROPE_SCALINGS)}")
    freq = np.zeros(max(int(rot_dim) // 2, 1), dtype=np.float64)
    amp = ctypes.c_float(0.0)
    rc = lib.orthros_rotary_frequencies(int(rot_dim), float(base), _ROPE_SCALINGS[scaling], float(factor),
                                        float(original_length), float(low_turns), float(high_turns),
                                        freq.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ctypes.byref(amp))
    _raise_if(rc, lib)
    return torch.from_numpy(freq), float(amp.value)


def orthros_rotary_steps(freq):
    """orthros_rotary_steps of include/orthros_attn.h: frequencies (radians per
    position) -> int64 CPU tensor holding the 64-bit steps; move it to the GPU once."""
    lib = load_library()
    f = freq.detach().cpu().numpy() if isinstance(freq, torch.Tensor) else freq
    f = np.ascontiguousarray(np.asarray(f, dtype=np.float64).ravel())
    steps = np.zeros(f.size, dtype=np.uint64)
    rc = lib.orthros_rotary_steps(f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), int(f.size),
                                  steps.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)))
    _raise_if(rc, lib)
    return torch.from_numpy(steps.view(np.int64))


def orthros_rotate(x, positions, steps, *, layout="half", amplitude=1.0, alpha=None, beta=None, out=None, stream=None):
    """orthros_rotate of include/orthros_attn.h: y = amplitude R(t) (alpha (.) x + beta).

    x [n, H, d] (any token stride), positions [n] int32, steps from
    orthros_rotary_steps on the GPU. Returns y [n, H, d] (`out` may be x).
    """
    if stream is not None:
        with _on(stream):
            return orthros_rotate(x, positions, steps, layout=layout, amplitude=amplitude, alpha=alpha, beta=beta, out=out)
    lib = _lib or load_library()
    dev, here = _here(x)
    shape, dtype = x.shape, x.dtype
    n, H, d = shape
    xa, xs = _rows("x", x, dev, dtype, shape)
    if out is None:
        out = _new(x, shape)
        ya, ys = out.data_ptr(), H * d
    else:
        ya, ys = _rows("out", out, dev, dtype, shape)
    st, rot = _steps(steps, dev)
    pos = _index("positions", positions, dev, n)
    al = _block("alpha", alpha, dev, torch.float32, (H, d))
    be = _block("beta", beta, dev, torch.float32, (H, d))
    rc = lib.orthros_rotate(xa, xs, pos, al, be, st, rot, _rope_layout(layout), amplitude, n, H, d, _dtype(x), ya, ys,
                            here)
    if rc:
        _raise_if(rc, lib)
    return out


def orthros_rotate_backward_workspace_size(n, H, d, dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_rotate_backward_workspace_size(n, H, d, _DTYPES[dtype]))


def orthros_rotate_backward(dy, x, positions, steps, *, layout="half", amplitude=1.0, alpha=None, affine_grads=True,
                            out=None, workspace=None, stream=None):
    """orthros_rotate_backward of include/orthros_attn.h.

    dy, x [n, H, d] (any token strides; x may be None without affine_grads).
    Returns (dx, d_alpha, d_beta), the last two float [H, d], or None without
    affine_grads; `out` gives the three tensors.
    """
    if stream is not None:
        with _on(stream):
            return orthros_rotate_backward(dy, x, positions, steps, layout=layout, amplitude=amplitude, alpha=alpha,
                                           affine_grads=affine_grads, out=out, workspace=workspace)
    lib = _lib or load_library()
    dev, here = _here(dy)
    shape, dtype = dy.shape, dy.dtype
    n, H, d = shape
    if out is None:
        dx, da, db = _new(dy, shape), None, None
        if affine_grads:
            da = torch.empty((H, d), dtype=torch.float32, device=dy.device)
            db = torch.empty_like(da)
        oa, os_ = dx.data_ptr(), H * d
    else:
        dx, da, db = out
        oa, os_ = _rows("dx", dx, dev, dtype, shape)
    if workspace is None and da is not None:
        workspace = torch.empty(max(orthros_rotate_backward_workspace_size(n, H, d, dtype), 256),
                                dtype=torch.uint8, device=dy.device)
    ga, gs = _rows("dy", dy, dev, dtype, shape)
    xa, xs = _rows("x", x, dev, dtype, shape)
    st, rot = _steps(steps, dev)
    rc = lib.orthros_rotate_backward(
        ga, gs, xa, xs, _index("positions", positions, dev, n), _block("alpha", alpha, dev, torch.float32, (H, d)), st, rot,
        _rope_layout(layout), amplitude, n, H, d, _dtype(dy), oa, os_, _block("d_alpha", da, dev, torch.float32, (H, d)),
        _block("d_beta", db, dev, torch.float32, (H, d)), _addr(workspace, dev),
        workspace.numel() if workspace is not None else 0, here)
    _raise_if(rc, lib)
    return dx, da, db


def orthros_rotate_append(q, k_new, v_new, k_cache, v_cache, block_table, token_seq, token_pos, steps, *,
                          layout="half", amplitude=1.0, q_out=None, out_positions=None, alpha_base=None,
                          beta_base=None, alpha_out=None, beta_out=None, out=None, workspace=None, stream=None):
    """orthros_rotate_append of include/orthros_attn.h.

    k_new, v_new [n, Hkv, d] go to their page slots (keys rotated); q [n, Hq,
    d] (or None) and q_out [n_out, Hq, d] are rotated. Returns (q_rot or None,
    q_out_rot or None); k_cache / v_cache are updated in place.
    """
    if stream is not None:
        with _on(stream):
            return orthros_rotate_append(
                q, k_new, v_new, k_cache, v_cache, block_table, token_seq, token_pos, steps, layout=layout,
                amplitude=amplitude, q_out=q_out, out_positions=out_positions, alpha_base=alpha_base, beta_base=beta_base,
                alpha_out=alpha_out, beta_out=beta_out, out=out, workspace=workspace)
    lib = _lib or load_library()
    dev, here = _here(k_cache)
    dtype = k_new.dtype
    n, Hkv, d = k_new.shape
    n_out = q_out.shape[0] if q_out is not None else 0
    Hq = q.shape[1] if q is not None else (q_out.shape[1] if q_out is not None else Hkv)
    num_pages, page_size = k_cache.shape[:2]
    B, max_pages = block_table.shape
    if out is None:
        q_rot = _new(q, (n, Hq, d)) if q is not None else None
        q_out_rot = _new(q_out, (n_out, Hq, d)) if q_out is not None else None
    else:
        q_rot, q_out_rot = out
        _block("q_rot", q_rot, dev, dtype, (n, Hq, d))
        _block("q_out_rot", q_out_rot, dev, dtype, (n_out, Hq, d))
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=k_new.device)
    qa, qs = _rows("q", q, dev, dtype, (n, Hq, d))
    qoa, qos = _rows("q_out", q_out, dev, dtype, (n_out, Hq, d))
    ka, ks = _rows("k_new", k_new, dev, dtype, (n, Hkv, d))
    va, vs = _rows("v_new", v_new, dev, dtype, (n, Hkv, d))
    aff = [_block(name, t, dev, torch.float32, (Hq, d)) for name, t in
           (("alpha_base", alpha_base), ("beta_base", beta_base), ("alpha_out", alpha_out), ("beta_out", beta_out))]
    st, rot = _steps(steps, dev)
    pool = (num_pages, page_size, Hkv, d)
    rc = lib.orthros_rotate_append(
        qa, qs, qoa, qos, ka, ks, va, vs, *aff, st, rot, _rope_layout(layout), amplitude,
        _index("token_seq", token_seq, dev, n), _index("token_pos", token_pos, dev, n),
        _index("out_positions", out_positions, dev, n_out), n, n_out, Hq, Hkv, d, _dtype(k_new),
        _addr(q_rot, dev), _addr(q_out_rot, dev),
        _block("k_cache", k_cache, dev, dtype, pool), _block("v_cache", v_cache, dev, dtype, pool),
        _index("block_table", block_table, dev, B * max_pages), B, max_pages, page_size, num_pages, _addr(workspace, dev),
        workspace.numel(), here)
    _raise_if(rc, lib)
    return q_rot, q_out_rot


def _int32(x) -> int:
    """A bound that may exceed 32 bits, held at their ends (ctypes would drop its upper bits)."""
    return max(-2 ** 31, min(int(x), 2 ** 31 - 1))


def orthros_chunk_attention_workspace_size(B, n, max_new, Hq, Hkv, d, max_pages, page_size,
                                           dtype=torch.bfloat16) -> int:
    return int(load_library().orthros_chunk_attention_workspace_size(B, n, _int32(max_new), Hq, Hkv, d, max_pages,
                                                                     page_size, _DTYPES[dtype]))


def orthros_chunk_attention(q, q_indptr, kv_lens, k_cache, v_cache, block_table, window, scale=None, *, max_new=None,
                            out=None, workspace=None, stream=None):
    """orthros_chunk_attention of include/orthros_attn.h on torch CUDA tensors.

    q [n, Hq, d] with the tokens of sequence b at q_indptr[b] .. q_indptr[b+1];
    q_indptr and kv_lens are int32 tensors on the GPU. max_new bounds the new
    tokens of a sequence (default n). Returns (o [n, Hq, d], lse [n, Hq]).
    """
    if stream is not None:
        with _on(stream):
            return orthros_chunk_attention(q, q_indptr, kv_lens, k_cache, v_cache, block_table, window, scale,
                                           max_new=max_new, out=out, workspace=workspace)
    lib = _lib or load_library()
    dev, here = _here(q)
    shape, dtype = q.shape, q.dtype
    n, Hq, d = shape
    num_pages, page_size, Hkv = k_cache.shape[:3]
    B, max_pages = block_table.shape
    max_new = n if max_new is None else _int32(max_new)
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((n, Hq), dtype=torch.float32, device=q.device)
        oa, la = o.data_ptr(), lse.data_ptr()
    else:
        o, lse = out
        oa, la = _block("o", o, dev, dtype, shape), _block("lse", lse, dev, torch.float32, (n, Hq))
    if workspace is None:
        ws = orthros_chunk_attention_workspace_size(B, n, max_new, Hq, Hkv, d, max_pages, page_size, dtype)
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=q.device)
    pool = (num_pages, page_size, Hkv, d)
    rc = lib.orthros_chunk_attention(
        _block("q", q, dev, dtype, shape), _index("q_indptr", q_indptr, dev, B + 1), _index("kv_lens", kv_lens, dev, B),
        _block("k_cache", k_cache, dev, dtype, pool), _block("v_cache", v_cache, dev, dtype, pool),
        _index("block_table", block_table, dev, B * max_pages), B, n, max_new, Hq, Hkv, d, _int32(window),
        d ** -0.5 if scale is None else scale, _dtype(q), max_pages, page_size, num_pages,
        oa, la, _addr(workspace, dev),
        workspace.numel(), here)
    _raise_if(rc, lib)
    return o, lse


def orthros_selftest_wait_timeout(limit_cycles, workspace, stream=None):
    """orthros_selftest_wait_timeout of include/orthros_attn.h: one kernel whose
    bounded wait on a barrier nothing arms runs out after limit_cycles."""
    lib = load_library()
    rc = lib.orthros_selftest_wait_timeout(int(limit_cycles), _ptr(workspace), workspace.numel(), _stream(stream))
    _raise_if(rc, lib)


def orthros_check(workspace, stream=None):
    """Synchronise and read the device status word. Returns (status, bits)."""
    lib = load_library()
    bits = ctypes.c_uint32(0)
    rc = lib.orthros_check(_ptr(workspace), _stream(stream), ctypes.byref(bits))
    return int(rc), int(bits.value)


def orthros_profile_begin():
    """Start recording per-kernel CUDA-event times of the library's launches."""
    _raise_if(load_library().orthros_profile_begin(), load_library())


def orthros_profile_end():
    """Stop recording; returns {kernel name: (launches, total_ms)} in first-launch order."""
    lib = load_library()
    buf = (KernelTime * 64)()
    n = lib.orthros_profile_end(buf, 64)
    if n < 0:
        raise OrthrosError(3, "orthros_profile_end: CUDA error while reading events")
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(min(n, 64))}
