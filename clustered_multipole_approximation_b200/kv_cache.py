"""The paged K/V cache of an attention layer: write, read back, attend.

    make_cache(pages, Hkv, page_size, D, dtype)      the buffers of one layer
    muse_cache_write(k, v, k_cache, v_cache, table, kv_len, ...)
    muse_cache_read(k_cache, v_cache, table, kv_len, N, ...)
    muse_attn_cache(q, k_cache, v_cache, table, kv_len, ...)

A serving step of a layer writes the new tokens' keys and values and then lets
their queries attend; a prompt's chunk, one token a sequence and a mixed batch
are the same two calls:

    kv_len += new_len
    muse_cache_write(k, v, kc, vc, table, kv_len, new_len=new_len)
    o = muse_attn_cache(q, kc, vc, table, kv_len, new_len=new_len, scale=s)

Shapes: q, k, v [B, H, n, D], bf16 or fp32, the last dimension contiguous and
the others with strides of whole 16 bytes (a transposed view of a projection's
output is fine); k_cache and v_cache [pages, Hkv, page_size, D] in bf16, fp32,
float8_e4m3fn or int8, the 8-bit ones with fp32 k_scale and v_scale [pages,
Hkv, page_size]; table int32 [B, wide], kv_len, new_len and start int32 [B].
All of it lies on one CUDA device.  What each call computes, and what it does
with lengths and table entries out of range, is in include/muse.h.
"""
from __future__ import annotations

import ctypes
import importlib

import torch

import clustered_multipole_approximation_b200 as muse

CACHE_DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float8_e4m3fn: 2, torch.int8: 3}


class muse_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class muse_cache_index(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("new_len", ctypes.c_void_p), ("wide", ctypes.c_int)]


class muse_strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class muse_cache_division(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_longlong)] + [
        (x, ctypes.c_int) for x in ("rows", "splits", "cluster", "quantum", "parts", "keys")]


def declare(lib) -> None:
    """Signatures of the cache entry points."""
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    sh, ca, ix, st = (ctypes.POINTER(t) for t in (muse.muse_shape, muse_cache, muse_cache_index,
                                                   muse_strides))
    lib.muse_cache_write.restype = i32
    lib.muse_cache_write.argtypes = [vp, st, vp, st, sh, ca, ix, vp, vp]
    lib.muse_cache_read.restype = i32
    lib.muse_cache_read.argtypes = [vp, vp, sh, ca, ix, vp, vp, vp]
    lib.muse_attn_cache_workspace_size.restype = sz
    lib.muse_attn_cache_workspace_size.argtypes = [sh, ca, ix]
    lib.muse_debug_inject_cache_fault.restype = None
    lib.muse_debug_inject_cache_fault.argtypes = [i32]
    lib.muse_debug_cache_division.restype = i32
    lib.muse_debug_cache_division.argtypes = [sh, ca, ix, i32, i32, ctypes.POINTER(muse_cache_division)]
    lib.muse_attn_cache.restype = i32
    lib.muse_attn_cache.argtypes = [vp, st, vp, st, vp, sh, ca, ix, ctypes.c_float, i32, i32, vp,
                                    vp, sz, vp]


def make_cache(pages, Hkv, page_size, D, dtype=torch.bfloat16, device="cuda"):
    """Zeroed buffers of one layer's cache, as keyword arguments of the calls
    here: k_cache, v_cache and, for 8-bit dtypes, k_scale and v_scale."""
    if dtype not in CACHE_DTYPES:
        raise TypeError(f"unsupported cache dtype {dtype} (bf16, fp32, float8_e4m3fn or int8)")
    out = {x: torch.zeros(pages, Hkv, page_size, D, dtype=dtype, device=device)
           for x in ("k_cache", "v_cache")}
    if dtype.itemsize == 1:
        out.update({x: torch.ones(pages, Hkv, page_size, device=device)
                    for x in ("k_scale", "v_scale")})
    return out


_bound = None


def _native():
    """The calls on torch tensors (csrc/torch_cache.cpp): argument checks,
    outputs and workspace, launch.  Raises if it is not built."""
    global _bound
    if _bound is None:
        muse.load_library()
        try:
            _bound = importlib.import_module("clustered_multipole_approximation_b200._torch_cache")
        except ImportError as e:
            raise ImportError(f"_torch_cache.so not built or not loadable ({e}); run "
                              "`python -m clustered_multipole_approximation_b200.build`") from e
        _bound.set_error(muse.MuseError)
    return _bound


def _stream(stream, device):
    """A stream other than the current one takes over behind it: memory
    allocated for the call may be memory that work there still uses."""
    if stream is None:
        return None
    if stream.device != device:
        raise ValueError(f"stream must be one of {device}")
    current = torch.cuda.current_stream(device)
    if stream != current:
        stream.wait_stream(current)
    return stream.stream_id, stream.device_index, stream.device_type


def muse_cache_write(k, v, k_cache, v_cache, table, kv_len, *, new_len=None, k_scale=None,
                     v_scale=None, device_error=None, stream=None) -> None:
    """Write the new tokens' rows k, v [B,Hkv,n,D] to their pages, quantising
    them where the cache holds 8 bits.  kv_len counts them already; new_len
    (default: n everywhere) says how many of the n rows each sequence has."""
    if stream is not None:
        stream = _stream(stream, k_cache.device)
    (_bound or _native()).cache_write(k, v, k_cache, v_cache, table, kv_len, new_len, k_scale, v_scale,
                                      device_error, stream)


def muse_cache_read(k_cache, v_cache, table, kv_len, N, *, start=None, k_scale=None, v_scale=None,
                    dtype=torch.bfloat16, out=None, device_error=None, stream=None):
    """Positions start .. start + N - 1 (start [B], default 0) of every
    sequence as contiguous (k, v) [B,Hkv,N,D] in `dtype`, the layout of the
    whole-sequence operators; rows at and past kv_len are zero.  out: a (k, v)
    pair to write to."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    if stream is not None:
        stream = _stream(stream, k_cache.device)
    ok, ov = (None, None) if out is None else out
    return (_bound or _native()).cache_read(k_cache, v_cache, table, kv_len, N, start, k_scale, v_scale,
                                            dtype is torch.bfloat16, ok, ov, device_error, stream)


def attn_cache_workspace_size(q, k_cache, v_cache, table, kv_len, *, k_scale=None, v_scale=None) -> int:
    """Workspace bytes of muse_attn_cache for tensors of these shapes."""
    return _native().attn_workspace(q, k_cache, v_cache, table, kv_len, k_scale, v_scale)


def muse_attn_cache(q, k_cache, v_cache, table, kv_len, *, new_len=None, scale=1.0, causal=True,
                    window=0, k_scale=None, v_scale=None, out=None, lse=None, workspace=None,
                    device_error=None, stream=None):
    """Exact attention of the new tokens' queries q [B,Hq,n,D] over the cache
    (their own keys and values written before): causally by position, within
    the last `window` positions if it is not 0, or over all kv_len positions
    with causal=False (cross attention).  Returns o [B,Hq,n,D] in q's dtype
    or, with lse=True or an fp32 [B,Hq,n] tensor to write to, (o, lse).  Rows
    i >= new_len of tensors that the caller gives are left as they were; of o
    and lse made here they are 0 and -inf (a fill, some 2 us: calls that repeat
    give out).  out may not share memory with q."""
    if stream is not None:
        stream = _stream(stream, k_cache.device)
    return (_bound or _native()).attn_cache(q, k_cache, v_cache, table, kv_len, new_len, scale, causal, window,
                                            k_scale, v_scale, out, None if lse is False else lse, workspace,
                                            device_error, stream)
