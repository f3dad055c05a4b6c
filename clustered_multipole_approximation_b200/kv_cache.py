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

import contextlib
import ctypes

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


def _same(dev, **ts):
    for name, t in ts.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, the device of the cache")


def _cache(k, v, ks, vs, table, kv_len, new_len, B, Hkv, D):
    """Checked descriptors of a cache and of the batch's place in it."""
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("tensors must be CUDA tensors")
    _same(dev, v_cache=v, k_scale=ks, v_scale=vs, table=table, kv_len=kv_len, new_len=new_len)
    if k.dtype not in CACHE_DTYPES or v.dtype != k.dtype:
        raise TypeError("k_cache and v_cache must share a dtype: bf16, fp32, float8_e4m3fn or int8")
    if k.dim() != 4 or v.shape != k.shape or not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous [pages, Hkv, page_size, D]")
    if k.shape[1] != Hkv or k.shape[3] != D:
        raise ValueError(f"the cache holds {k.shape[1]} heads of {k.shape[3]}, the call {Hkv} of {D}")
    for name, s in (("k_scale", ks), ("v_scale", vs)):
        if (s is not None) != (k.dtype.itemsize == 1):
            raise ValueError(f"{name} belongs to an 8-bit cache, and to no other")
        if s is not None and (s.dtype != torch.float32 or s.shape != k.shape[:3]
                              or not s.is_contiguous()):
            raise ValueError(f"{name} must be contiguous fp32 [pages, Hkv, page_size]")
    if table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != B or not table.is_contiguous():
        raise ValueError(f"table must be contiguous int32 [{B}, wide]")
    for name, t in (("kv_len", kv_len), ("new_len", new_len)):
        if t is not None and (t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous int32 [{B}]")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return (muse_cache(p(k), p(v), p(ks), p(vs), k.shape[0], k.shape[2], CACHE_DTYPES[k.dtype]),
            muse_cache_index(p(table), p(kv_len), p(new_len), table.shape[1]))


def _strided(t, name):
    """A tensor's strides, of a [B, H, n, D] view whose rows are contiguous
    (the stride of a dimension of one is never used: 0)."""
    if t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] > 1):
        raise ValueError(f"{name} must be [B, H, n, D] with a contiguous last dimension")
    return muse_strides(*[0 if n == 1 else s for n, s in zip(t.shape[:3], t.stride()[:3])])


def _on(dev):
    """The device the library launches on."""
    return contextlib.nullcontext() if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(stream, dev, *made):
    """The stream's handle; memory allocated here on the current stream is
    kept from reuse until another stream's work with it is done."""
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    if stream.device != dev:
        raise ValueError(f"stream must be one of {dev}")
    current = torch.cuda.current_stream(dev)
    if stream != current:
        stream.wait_stream(current)  # `made` may be memory that work there still uses
        for t in made:
            if t is not None:
                t.record_stream(stream)
    return stream.cuda_stream


def _error_ptr(device_error, dev):
    if device_error is None:
        return None
    if device_error.dtype != torch.int32 or device_error.numel() != 1 or device_error.device != dev:
        raise ValueError(f"device_error must be one int32 on {dev}")
    return device_error.data_ptr()


def muse_cache_write(k, v, k_cache, v_cache, table, kv_len, *, new_len=None, k_scale=None,
                     v_scale=None, device_error=None, stream=None) -> None:
    """Write the new tokens' rows k, v [B,Hkv,n,D] to their pages, quantising
    them where the cache holds 8 bits.  kv_len counts them already; new_len
    (default: n everywhere) says how many of the n rows each sequence has."""
    lib = muse.load_library()
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must be [B, Hkv, n, D] of one shape and dtype")
    B, Hkv, n, D = k.shape
    dev = k_cache.device
    ca, ix = _cache(k_cache, v_cache, k_scale, v_scale, table, kv_len, new_len, B, Hkv, D)
    _same(dev, k=k, v=v)
    sh = muse.muse_shape(B, Hkv, Hkv, n, D, muse._dtype_code(k), 0)
    with _on(dev):
        muse._check(lib, lib.muse_cache_write(
            k.data_ptr(), _strided(k, "k"), v.data_ptr(), _strided(v, "v"), sh, ca, ix,
            _error_ptr(device_error, dev), _stream(stream, dev)))


def muse_cache_read(k_cache, v_cache, table, kv_len, N, *, start=None, k_scale=None, v_scale=None,
                    dtype=torch.bfloat16, out=None, device_error=None, stream=None):
    """Positions start .. start + N - 1 (start [B], default 0) of every
    sequence as contiguous (k, v) [B,Hkv,N,D] in `dtype`, the layout of the
    whole-sequence operators; rows at and past kv_len are zero.  out: a (k, v)
    pair to write to."""
    lib = muse.load_library()
    B = table.shape[0]
    dev = k_cache.device
    Hkv, D = k_cache.shape[1], k_cache.shape[-1]
    ca, ix = _cache(k_cache, v_cache, k_scale, v_scale, table, kv_len, None, B, Hkv, D)
    if start is not None and (start.dtype != torch.int32 or start.shape != (B,)
                              or not start.is_contiguous()):
        raise ValueError(f"start must be contiguous int32 [{B}]")
    made = ()
    if out is None:
        out = made = tuple(torch.empty(B, Hkv, N, D, dtype=dtype, device=dev) for _ in range(2))
    k, v = out
    for t in out:
        if t.shape != (B, Hkv, N, D) or t.dtype != k.dtype or not t.is_contiguous():
            raise ValueError(f"out must be two contiguous [{B}, {Hkv}, {N}, {D}] tensors of one dtype")
    _same(dev, k=k, v=v, start=start)
    sh = muse.muse_shape(B, Hkv, Hkv, N, D, muse._dtype_code(k), 0)
    with _on(dev):
        muse._check(lib, lib.muse_cache_read(
            k.data_ptr(), v.data_ptr(), sh, ca, ix, None if start is None else start.data_ptr(),
            _error_ptr(device_error, dev), _stream(stream, dev, *made)))
    return k, v


def attn_cache_workspace_size(q, k_cache, v_cache, table, kv_len, *, k_scale=None, v_scale=None) -> int:
    """Workspace bytes of muse_attn_cache for tensors of these shapes."""
    lib = muse.load_library()
    B, Hq, n, D = q.shape
    Hkv = k_cache.shape[1]
    ca, ix = _cache(k_cache, v_cache, k_scale, v_scale, table, kv_len, None, B, Hkv, D)
    size = lib.muse_attn_cache_workspace_size(muse.muse_shape(B, Hq, Hkv, n, D, muse._dtype_code(q), 0),
                                              ca, ix)
    if size == 0:
        raise muse.MuseError(1, lib.muse_last_error().decode())
    return int(size)


def muse_attn_cache(q, k_cache, v_cache, table, kv_len, *, new_len=None, scale=1.0, causal=True,
                    window=0, k_scale=None, v_scale=None, out=None, lse=None, workspace=None,
                    device_error=None, stream=None):
    """Exact attention of the new tokens' queries q [B,Hq,n,D] over the cache
    (their own keys and values written before): causally by position, within
    the last `window` positions if it is not 0, or over all kv_len positions
    with causal=False (cross attention).  Returns o [B,Hq,n,D] in q's dtype
    or, with lse=True or an fp32 [B,Hq,n] tensor to write to, (o, lse).  Rows
    i >= new_len of o and lse are left as they were."""
    lib = muse.load_library()
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, n, D]")
    B, Hq, n, D = q.shape
    dev = k_cache.device
    Hkv = k_cache.shape[1]
    ca, ix = _cache(k_cache, v_cache, k_scale, v_scale, table, kv_len, new_len, B, Hkv, D)
    made = []
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        made.append(out)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and dtype")
    if lse is True:
        lse = torch.empty(B, Hq, n, dtype=torch.float32, device=dev)
        made.append(lse)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.shape != (B, Hq, n) or lse.dtype != torch.float32
                              or not lse.is_contiguous()):
        raise ValueError(f"lse must be contiguous fp32 [{B}, {Hq}, {n}]")
    sh = muse.muse_shape(B, Hq, Hkv, n, D, muse._dtype_code(q), 0)
    if workspace is None:
        size = lib.muse_attn_cache_workspace_size(sh, ca, ix)
        if size == 0:
            raise muse.MuseError(1, lib.muse_last_error().decode())
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        made.append(workspace)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _same(dev, q=q, out=out, lse=lse, workspace=workspace)
    with _on(dev):
        muse._check(lib, lib.muse_attn_cache(
            q.data_ptr(), _strided(q, "q"), out.data_ptr(), _strided(out, "out"),
            None if lse is None else lse.data_ptr(), sh, ca, ix, scale, int(causal), int(window),
            _error_ptr(device_error, dev), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(stream, dev, *made)))
    return out if lse is None else (out, lse)
