"""ctypes binding of the paged key/value cache: argument marshalling only.

A :class:`PagedCache` holds one layer's pages (bf16, e4m3 or int8; include/pi_attn.h has the
formats).  The calls take the batch as device tensors: a page table [B, width], and, for packed
chunks, offsets cu [B + 1] and positions ctx [B], all int32.  They only enqueue work on the tensors'
device; an index out of range is reported by :func:`structured_sparse_long_gb300.status`.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _binding
from ._binding import MODE_ECP, MODE_PI, PI_OK, _check

KV_BF16, KV_E4M3, KV_INT8 = 0, 1, 2
_KV_TYPES = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8}
SCALE_BLOCK = 32  # elements per scale byte of an 8-bit cache


_INT32, _BF16, _FP32 = torch.int32, torch.bfloat16, torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _CacheStruct(ctypes.Structure):  # pi_attn_cache_t
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("kv_type", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("page", ctypes.c_int), ("d", ctypes.c_int)]


class _BatchStruct(ctypes.Structure):  # pi_attn_batch_t
    _fields_ = [("table", ctypes.c_void_p), ("cu", ctypes.c_void_p), ("ctx", ctypes.c_void_p),
                ("B", ctypes.c_int), ("T", ctypes.c_int), ("width", ctypes.c_int)]


def _load():
    lib = _binding.load()
    if lib.pi_attn_extend.argtypes is None:
        P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        C, B = ctypes.POINTER(_CacheStruct), ctypes.POINTER(_BatchStruct)
        lib.pi_attn_cache_append.argtypes = [P, P, L, L, C, B, P]
        lib.pi_attn_cache_read.argtypes = [C, B, P, P, P]
        lib.pi_attn_decode_paged.argtypes = [P, L, C, P, P, I, I, P, I, I, I, I, I, P, P, P]
        lib.pi_attn_extend.argtypes = [P, L, C, B, P, I, I, I, I, I, P, P, P, ctypes.c_size_t, P]
        lib.pi_attn_extend_workspace_size.argtypes = [C, I, I, I, I, I, I, I, I]
        lib.pi_attn_extend_workspace_size.restype = ctypes.c_size_t
        for name in ("cache_append", "cache_read", "decode_paged", "extend"):
            getattr(lib, "pi_attn_" + name).restype = I
    return lib


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
        self._struct = _CacheStruct(*(None if t is None else t.data_ptr() for t in self._tensors),
                                    self.kv_type, n_pages, Hkv, page, d)
        self._ref = ctypes.byref(self._struct)
        self._workspace = {}  # extend's workspace sizes by the call's sizes
        self.device, self.index = k.device, k.get_device()
        self.Hkv, self.page, self.d = Hkv, page, d

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


def _refuse(t, name, want):
    raise ValueError(f"{name} must be {want}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}"
                     if isinstance(t, torch.Tensor) else f"{name} must be {want}, got {type(t).__name__}")


# Checks of a serving step's hot path: one C call's worth of them costs as much as the launch, so they compare device
# indexes and dtype objects only.

def _int32(t, name, index, *shape):
    if t.dtype is not _INT32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, f"a contiguous int32 tensor of shape {shape} on cuda:{index}")
    return t.data_ptr()


def _dense(t, name, index, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, f"a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _packed(t, name, cache, heads):
    """Number of tokens, heads and the stride between the tokens of a packed [T, heads, d] bf16 tensor whose tokens are
    contiguous."""
    shape = t.shape
    if len(shape) != 3 or t.dtype is not _BF16 or shape[2] != cache.d or t.get_device() != cache.index or (
            heads is not None and shape[1] != heads):
        _refuse(t, name, f"bf16 [T, {heads or 'heads'}, {cache.d}] on cuda:{cache.index}")
    T, heads, d = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != d):
        _refuse(t, name, "a tensor whose tokens have contiguous elements")
    return T, heads, (s0 if T > 1 else heads * d)


def _batch(table, cu, ctx, T, cache):
    if table.dim() != 2:
        _refuse(table, "table", "[B, width]")
    B, width = table.shape
    index = cache.index
    return _BatchStruct(_int32(table, "table", index, B, width), _int32(cu, "cu", index, B + 1), _int32(ctx, "ctx", index, B), B, T,
                        width)


_fns = {}  # entry points, once the library is loaded


def _call(name, cache, stream, check, *args):
    """Calls an entry point with `args` and the stream (the current one of the cache's device, if none is given) on that
    device."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_load(), name)
    index = cache.index
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != PI_OK or check:
        with torch.cuda.device(index):
            _check(name, rc, stream, check)


def cache_append(k, v, cache: PagedCache, table, cu, ctx, stream=None, check=False) -> None:
    """pi_attn_cache_append: writes the packed rows k, v [T, Hkv, d] bf16 (tokens any stride apart) into the
    pages of their sequences, quantised where the cache holds 8 bits."""
    T, _, ks = _packed(k, "k", cache, cache.Hkv)
    Tv, _, vs = _packed(v, "v", cache, cache.Hkv)
    if Tv != T:
        _refuse(v, "v", f"of shape {tuple(k.shape)}")
    batch = _batch(table, cu, ctx, T, cache)
    if T > 0:
        _call("pi_attn_cache_append", cache, stream, check, k.data_ptr(), v.data_ptr(), ks, vs, cache._ref, batch)


def cache_read(cache: PagedCache, table, cu, start, rows: int, k=None, v=None, stream=None, check=False):
    """pi_attn_cache_read: rows start[b] .. start[b] + cu[b+1] - cu[b] - 1 of every sequence, packed, as
    bf16 (k, v) [rows, Hkv, d]."""
    shape, dev = (rows, cache.Hkv, cache.d), cache.device
    k = torch.empty(shape, dtype=torch.bfloat16, device=dev) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=dev) if v is None else v
    pk, pv = _dense(k, "k", cache.index, _BF16, shape), _dense(v, "v", cache.index, _BF16, shape)
    batch = _batch(table, cu, start, rows, cache)
    if rows > 0:
        _call("pi_attn_cache_read", cache, stream, check, cache._ref, batch, pk, pv)
    return k, v


def _rows(T, H, cache, alpha, mode, out, lse):
    """Checks of an attention's packed rows: (alpha's pointer, out, lse)."""
    if alpha is not None:
        alpha = _dense(alpha, "alpha", cache.index, _FP32, (T, H))
    elif mode != MODE_ECP:
        raise ValueError("alpha is needed in pi mode")
    if out is None:
        out = torch.empty((T, H, cache.d), dtype=_BF16, device=cache.device)
    else:
        _dense(out, "out", cache.index, _BF16, (T, H, cache.d))
    if lse is None:
        lse = torch.empty((T, H), dtype=_FP32, device=cache.device)
    else:
        _dense(lse, "lse", cache.index, _FP32, (T, H))
    return alpha, out, lse


def extend_workspace_size(cache: PagedCache, B: int, T: int, width: int, H: int, k_local: int, period: int, S: int,
                          mode: int = MODE_PI) -> int:
    """pi_attn_extend_workspace_size: bytes of device workspace that :func:`extend` needs for B sequences with T packed
    tokens and page tables of `width` entries (0: none, or sizes that it refuses)."""
    return int(_load().pi_attn_extend_workspace_size(cache._ref, B, T, width, H, k_local, period, S, mode))


def extend(q, cache: PagedCache, table, cu, ctx, alpha, k_local: int, period: int, S: int, mode: int = MODE_PI,
           out=None, lse=None, workspace=None, stream=None, check=False):
    """pi_attn_extend: the packed new tokens q [T, H, d] bf16 (any token stride) against their sequences' cached
    rows, which hold the chunk's own already.  alpha [T, H] fp32 (None in ECP mode).  Returns (out, lse)."""
    T, H, qs = _packed(q, "q", cache, None)
    alpha, out, lse = _rows(T, H, cache, alpha, mode, out, lse)
    batch = _batch(table, cu, ctx, T, cache)
    if T > 0:
        key = (batch.B, T, batch.width, H, k_local, period, S, mode)
        nbytes = cache._workspace.get(key)
        if nbytes is None:
            if len(cache._workspace) >= 256:
                cache._workspace.clear()
            nbytes = cache._workspace[key] = extend_workspace_size(cache, *key)
        if workspace is None:
            if nbytes:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
        else:
            _dense(workspace, "workspace", cache.index, torch.uint8, workspace.shape)
            if workspace.numel() < nbytes:
                raise ValueError(f"workspace must hold {nbytes} bytes, got {workspace.numel()}")
        _call("pi_attn_extend", cache, stream, check, q.data_ptr(), qs, cache._ref, batch, alpha, H, k_local, period, S, mode,
              out.data_ptr(), lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
              0 if workspace is None else workspace.numel())
    return out, lse


def decode_paged(q, cache: PagedCache, table, lens, alpha, k_local: int, period: int, S: int, mode: int = MODE_PI,
                 out=None, lse=None, stream=None, check=False):
    """pi_attn_decode_paged: one new token per sequence, q [B, H, d] bf16, against lens[b] cached rows (its own
    among them).  alpha [B, H] fp32 (None in ECP mode).  Returns (out [B, H, d], lse [B, H])."""
    B, H, qs = _packed(q, "q", cache, None)
    alpha, out, lse = _rows(B, H, cache, alpha, mode, out, lse)
    if table.dim() != 2:
        _refuse(table, "table", "[B, width]")
    width = table.shape[1]
    pt, pl = _int32(table, "table", cache.index, B, width), _int32(lens, "lens", cache.index, B)
    if B > 0:
        _call("pi_attn_decode_paged", cache, stream, check, q.data_ptr(), qs, cache._ref, pt, pl, B, width, alpha, H, k_local,
              period, S, mode, out.data_ptr(), lse.data_ptr())
    return out, lse
