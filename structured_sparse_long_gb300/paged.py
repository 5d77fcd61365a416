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
from ._binding import MODE_ECP, MODE_PI, _check

KV_BF16, KV_E4M3, KV_INT8 = 0, 1, 2
_KV_TYPES = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8}
SCALE_BLOCK = 32  # elements per scale byte of an 8-bit cache


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
        self.device = k.device
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


class _on:
    """Makes `device` current for a call (nothing to do where it is already)."""

    __slots__ = ("guard",)

    def __init__(self, device):
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _index_tensor(t, name, cache, shape):
    if t.dtype != torch.int32 or t.device != cache.device or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {cache.device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _packed_rows(t, name, cache, heads=None):
    """[T, heads, d] bf16 with contiguous tokens any stride apart; returns that stride."""
    if t.dim() != 3 or t.dtype != torch.bfloat16 or t.device != cache.device or t.shape[2] != cache.d or (
            heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be bf16 [T, {heads or 'heads'}, {cache.d}] on {cache.device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    rows, heads, d = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != d):
        raise ValueError(f"{name}: the elements of a token must be contiguous, got strides {t.stride()}")
    return s0 if rows > 1 else heads * d


def _batch(table, cu, ctx, T, cache):
    if table.dim() != 2:
        raise ValueError("table must be [B, width]")
    B, width = table.shape
    _index_tensor(table, "table", cache, (B, width))
    _index_tensor(cu, "cu", cache, (B + 1,))
    _index_tensor(ctx, "ctx", cache, (B,))
    return _BatchStruct(table.data_ptr(), cu.data_ptr(), ctx.data_ptr(), B, T, width)


def _stream_of(stream, device):
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def cache_append(k, v, cache: PagedCache, table, cu, ctx, stream=None, check=False) -> None:
    """pi_attn_cache_append: writes the packed rows k, v [T, Hkv, d] bf16 (tokens any stride apart) into the
    pages of their sequences, quantised where the cache holds 8 bits."""
    ks = _packed_rows(k, "k", cache, cache.Hkv)
    vs = _packed_rows(v, "v", cache, cache.Hkv)
    if v.shape != k.shape:
        raise ValueError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    batch = _batch(table, cu, ctx, k.shape[0], cache)
    if k.shape[0] == 0:
        return
    with _on(cache.device):
        rc = _load().pi_attn_cache_append(k.data_ptr(), v.data_ptr(), ks, vs, cache._ref, ctypes.byref(batch),
                                          _stream_of(stream, cache.device))
        _check("pi_attn_cache_append", rc, stream, check)


def cache_read(cache: PagedCache, table, cu, start, rows: int, k=None, v=None, stream=None, check=False):
    """pi_attn_cache_read: rows start[b] .. start[b] + cu[b+1] - cu[b] - 1 of every sequence, packed, as
    bf16 (k, v) [rows, Hkv, d]."""
    shape = (rows, cache.Hkv, cache.d)
    k = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if v is None else v
    _binding._expect_like(k, "k", cache, torch.bfloat16, shape)
    _binding._expect_like(v, "v", cache, torch.bfloat16, shape)
    batch = _batch(table, cu, start, rows, cache)
    if rows > 0:
        with _on(cache.device):
            rc = _load().pi_attn_cache_read(cache._ref, ctypes.byref(batch), k.data_ptr(), v.data_ptr(),
                                            _stream_of(stream, cache.device))
            _check("pi_attn_cache_read", rc, stream, check)
    return k, v


def _outputs(q, cache, alpha, mode, out, lse):
    T, H, d = q.shape
    if alpha is None:
        if mode != MODE_ECP:
            raise ValueError("alpha is needed in pi mode")
    else:
        _binding._expect_like(alpha, "alpha", cache, torch.float32, (T, H))
    if out is None:
        out = torch.empty((T, H, d), dtype=torch.bfloat16, device=cache.device)
    else:
        _binding._expect_like(out, "out", cache, torch.bfloat16, (T, H, d))
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=cache.device)
    else:
        _binding._expect_like(lse, "lse", cache, torch.float32, (T, H))
    return out, lse


def extend_workspace_size(cache: PagedCache, B: int, T: int, width: int, H: int, k_local: int, period: int, S: int,
                          mode: int = MODE_PI) -> int:
    """pi_attn_extend_workspace_size: bytes of device workspace that :func:`extend` needs for B sequences with T packed
    tokens and page tables of `width` entries (0 for sizes that it refuses)."""
    return int(_load().pi_attn_extend_workspace_size(cache._ref, B, T, width, H, k_local, period, S, mode))


def extend(q, cache: PagedCache, table, cu, ctx, alpha, k_local: int, period: int, S: int, mode: int = MODE_PI,
           out=None, lse=None, workspace=None, stream=None, check=False):
    """pi_attn_extend: the packed new tokens q [T, H, d] bf16 (any token stride) against their sequences' cached
    rows, which hold the chunk's own already.  alpha [T, H] fp32 (None in ECP mode).  Returns (out, lse)."""
    qs = _packed_rows(q, "q", cache)
    T, H, _ = q.shape
    out, lse = _outputs(q, cache, alpha, mode, out, lse)
    batch = _batch(table, cu, ctx, T, cache)
    if T > 0:
        with _on(cache.device):
            lib = _load()
            nbytes = lib.pi_attn_extend_workspace_size(cache._ref, batch.B, T, batch.width, H, k_local, period, S, mode)
            if workspace is None:
                workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=cache.device)
            else:
                _binding._expect_like(workspace, "workspace", cache, torch.uint8, None)
                if workspace.numel() < nbytes:
                    raise ValueError(f"workspace must hold {nbytes} bytes, got {workspace.numel()}")
            rc = lib.pi_attn_extend(q.data_ptr(), qs, cache._ref, ctypes.byref(batch),
                                        None if alpha is None else alpha.data_ptr(), H, k_local, period, S, mode,
                                        out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                    _stream_of(stream, cache.device))
            _check("pi_attn_extend", rc, stream, check)
    return out, lse


def decode_paged(q, cache: PagedCache, table, lens, alpha, k_local: int, period: int, S: int, mode: int = MODE_PI,
                 out=None, lse=None, stream=None, check=False):
    """pi_attn_decode_paged: one new token per sequence, q [B, H, d] bf16, against lens[b] cached rows (its own
    among them).  alpha [B, H] fp32 (None in ECP mode).  Returns (out [B, H, d], lse [B, H])."""
    qs = _packed_rows(q, "q", cache)
    B, H, _ = q.shape
    out, lse = _outputs(q, cache, alpha, mode, out, lse)
    if table.dim() != 2:
        raise ValueError("table must be [B, width]")
    _index_tensor(table, "table", cache, (B, table.shape[1]))
    _index_tensor(lens, "lens", cache, (B,))
    if B > 0:
        with _on(cache.device):
            rc = _load().pi_attn_decode_paged(q.data_ptr(), qs, cache._ref, table.data_ptr(), lens.data_ptr(), B,
                                              table.shape[1], None if alpha is None else alpha.data_ptr(), H, k_local,
                                              period, S, mode, out.data_ptr(), lse.data_ptr(),
                                              _stream_of(stream, cache.device))
            _check("pi_attn_decode_paged", rc, stream, check)
    return out, lse
