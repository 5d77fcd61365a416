"""Binding of the paged key/value cache: argument marshalling only, in a native extension (csrc/pi_paged_py.cpp), since a
serving step makes these calls for every layer.

A :class:`PagedCache` holds one layer's pages (bf16, e4m3 or int8; include/pi_attn.h has the
formats).  The calls take the batch as device tensors: a page table [B, width], and, for packed
chunks, offsets cu [B + 1] and positions ctx [B], all int32.  They only enqueue work on the tensors'
device; an index out of range is reported by :func:`structured_sparse_long_gb300.status`.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
from typing import Optional

import torch

from . import _binding
from . import build as _build
from ._binding import MODE_PI, _check

KV_BF16, KV_E4M3, KV_INT8 = 0, 1, 2
_KV_TYPES = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8}
SCALE_BLOCK = 32  # elements per scale byte of an 8-bit cache


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _CacheStruct(ctypes.Structure):  # pi_attn_cache_t
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("kv_type", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("page", ctypes.c_int), ("d", ctypes.c_int)]


class _BatchStruct(ctypes.Structure):  # pi_attn_batch_t
    _fields_ = [("table", ctypes.c_void_p), ("cu", ctypes.c_void_p), ("ctx", ctypes.c_void_p),
                ("B", ctypes.c_int), ("T", ctypes.c_int), ("width", ctypes.c_int)]


class _Handle(ctypes.Structure):  # Handle of csrc/pi_paged_py.cpp
    _fields_ = [("cache", _CacheStruct), ("device", ctypes.c_int)]


_native = None  # the extension module, once loaded and bound to the library


def _load():
    """The library with the prototypes of the paged cache's entry points."""
    lib = _binding.load()
    if lib.pi_attn_extend.argtypes is None:
        P, I, L, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
        C, B = ctypes.POINTER(_CacheStruct), ctypes.POINTER(_BatchStruct)
        lib.pi_attn_cache_append.argtypes = [P, P, L, L, C, B, P]
        lib.pi_attn_cache_read.argtypes = [C, B, P, P, P]
        lib.pi_attn_decode_paged.argtypes = [P, L, C, P, P, I, I, P, I, I, I, I, I, P, P, P]
        lib.pi_attn_extend_workspace_size.argtypes = [C, I, I, I, I, I, I, I, I]
        lib.pi_attn_extend_workspace_size.restype = Z
        lib.pi_attn_extend.argtypes = [P, L, C, B, P, I, I, I, I, I, P, P, P, Z, P]
        for name in ("cache_append", "cache_read", "decode_paged", "extend"):
            getattr(lib, "pi_attn_" + name).restype = I
    return lib


def _load_native():
    global _native
    if _native is None:
        lib, path = _load(), _build.NATIVE_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"native binding not built: {path} is missing; run structured_sparse_long_gb300.build.build()")
        spec = importlib.util.spec_from_file_location("_pi_paged", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, "pi_attn_" + n), ctypes.c_void_p).value
                      for n in ("cache_append", "cache_read", "extend_workspace_size", "extend", "decode_paged")))
        _native = module
    return _native


class PagedCache:
    """The pages of one layer: k and v [n_pages, Hkv, page, d] in bf16, or in float8_e4m3fn or int8 with
    k_scale and v_scale [n_pages, Hkv, page, d / 32] uint8.  Holds the tensors; does not copy them."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4:
            raise ValueError("k must be [n_pages, Hkv, page, d]")
        if k.dtype not in _KV_TYPES:
            raise ValueError(f"unsupported cache dtype {k.dtype}")
        self.kv_type = _KV_TYPES[k.dtype]
        n_pages, Hkv, page, d = k.shape
        scale_shape = (n_pages, Hkv, page, d // SCALE_BLOCK)
        quant = self.kv_type != KV_BF16
        if quant and (k_scale is None or v_scale is None):
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        if not quant and (k_scale is not None or v_scale is not None):
            raise ValueError("a bf16 cache takes no scales")
        for t, name, dtype, shape in ((k, "k", k.dtype, k.shape), (v, "v", k.dtype, k.shape),
                                      (k_scale, "k_scale", torch.uint8, scale_shape),
                                      (v_scale, "v_scale", torch.uint8, scale_shape)):
            if t is not None:
                _binding._expect_like(t, name, k, dtype, shape)
        self._tensors = (k, v, k_scale, v_scale)
        self.device, self.index = k.device, k.get_device()
        self.Hkv, self.page, self.d = Hkv, page, d
        self._struct = _Handle(_CacheStruct(*(None if t is None else t.data_ptr() for t in self._tensors), self.kv_type, n_pages,
                                            Hkv, page, d), self.index)
        self._handle = ctypes.addressof(self._struct)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    @classmethod
    def empty(cls, n_pages: int, Hkv: int, page: int, d: int, dtype=torch.bfloat16, device="cuda") -> "PagedCache":
        """New pages, zero-filled (every row finite)."""
        def new(dt, width):
            return torch.zeros(n_pages, Hkv, page, width, dtype=torch.uint8, device=device).view(dt) \
                if dt != torch.bfloat16 else torch.zeros(n_pages, Hkv, page, width, dtype=dt, device=device)
        if dtype not in _KV_TYPES:
            raise ValueError(f"unsupported cache dtype {dtype}")
        quant = dtype != torch.bfloat16
        return cls(new(dtype, d), new(dtype, d), *((new(torch.uint8, d // SCALE_BLOCK) for _ in range(2)) if quant else ()))


@contextlib.contextmanager
def _place(cache, stream):
    """The cache's device current and, where a stream is given, that stream: a call's new tensors (outputs, workspace) are then
    the stream's own, so that none is handed out again while the call still uses it."""
    if stream is not None and stream.device != cache.device:
        raise ValueError(f"stream must be on {cache.device}, got {stream.device}")
    with torch.cuda.device(cache.index):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def cache_append(k, v, cache: PagedCache, table, cu, ctx, stream=None, check=False) -> None:
    """pi_attn_cache_append: writes the packed rows k, v [T, Hkv, d] bf16 (tokens any stride apart) into the
    pages of their sequences, quantised where the cache holds 8 bits."""
    if stream is not None or cache.index != _current_device():
        with _place(cache, stream):
            return cache_append(k, v, cache, table, cu, ctx, None, check)
    rc = (_native or _load_native()).append(k, v, cache._handle, table, cu, ctx, _raw_stream(cache.index))
    if rc or check:
        _check("pi_attn_cache_append", rc, None, check)


def cache_read(cache: PagedCache, table, cu, start, rows: int, k=None, v=None, stream=None, check=False):
    """pi_attn_cache_read: rows start[b] .. start[b] + cu[b+1] - cu[b] - 1 of every sequence, packed, as
    bf16 (k, v) [rows, Hkv, d]."""
    if stream is not None or cache.index != _current_device():
        with _place(cache, stream):
            return cache_read(cache, table, cu, start, rows, k, v, None, check)
    rc, k, v = (_native or _load_native()).read(cache._handle, table, cu, start, rows, k, v, _raw_stream(cache.index))
    if rc or check:
        _check("pi_attn_cache_read", rc, None, check)
    return k, v


def extend_workspace_size(cache: PagedCache, B: int, T: int, width: int, H: int, k_local: int, period: int, S: int,
                          mode: int = MODE_PI) -> int:
    """pi_attn_extend_workspace_size: bytes of workspace on the cache's device that :func:`extend` needs for B sequences with T
    packed tokens and page tables of `width` entries (0: none, or sizes that it refuses)."""
    if cache.index != _current_device():
        with _place(cache, None):
            return extend_workspace_size(cache, B, T, width, H, k_local, period, S, mode)
    return int(_load().pi_attn_extend_workspace_size(ctypes.byref(cache._struct.cache), B, T, width, H, k_local, period, S, mode))


def extend(q, cache: PagedCache, table, cu, ctx, alpha, k_local: int, period: int, S: int, mode: int = MODE_PI,
           out=None, lse=None, workspace=None, stream=None, check=False):
    """pi_attn_extend: the packed new tokens q [T, H, d] bf16 (any token stride) against their sequences' cached
    rows, which hold the chunk's own already.  alpha [T, H] fp32 (None in ECP mode).  Returns (out, lse)."""
    if stream is not None or cache.index != _current_device():
        with _place(cache, stream):
            return extend(q, cache, table, cu, ctx, alpha, k_local, period, S, mode, out, lse, workspace, None, check)
    rc, out, lse = (_native or _load_native()).extend(q, cache._handle, table, cu, ctx, alpha, k_local, period, S, mode, out, lse,
                                                      workspace, _raw_stream(cache.index))
    if rc or check:
        _check("pi_attn_extend", rc, None, check)
    return out, lse


def decode_paged(q, cache: PagedCache, table, lens, alpha, k_local: int, period: int, S: int, mode: int = MODE_PI,
                 out=None, lse=None, stream=None, check=False):
    """pi_attn_decode_paged: one new token per sequence, q [B, H, d] bf16, against lens[b] cached rows (its own
    among them).  alpha [B, H] fp32 (None in ECP mode).  Returns (out [B, H, d], lse [B, H])."""
    if stream is not None or cache.index != _current_device():
        with _place(cache, stream):
            return decode_paged(q, cache, table, lens, alpha, k_local, period, S, mode, out, lse, None, check)
    rc, out, lse = (_native or _load_native()).decode(q, cache._handle, table, lens, alpha, k_local, period, S, mode, out, lse,
                                                      _raw_stream(cache.index))
    if rc or check:
        _check("pi_attn_decode_paged", rc, None, check)
    return out, lse
