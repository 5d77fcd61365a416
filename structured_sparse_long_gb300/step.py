"""Binding of rotary positions and of a speculative serving step: argument marshalling only, in the same native extension as the
paged cache's (csrc/pi_paged_py.cpp; include/pi_attn.h has the operations).

A step over drafted trees: :func:`rotary_append` writes the nodes into the cache, :func:`extend_tree` attends, :func:`verify_tree`
finds the accepted path and the next token, :func:`cache_keep` moves the path's rows together.  All only enqueue work on
the tensors' device; an index out of range is reported by :func:`structured_sparse_long_gb300.status`.
"""
from __future__ import annotations

import ctypes
import math
from collections import namedtuple
from fractions import Fraction
from typing import Optional, Sequence

import torch

from . import paged
from ._binding import MODE_PI, _check
from .paged import PagedCache, _CacheStruct, _current_device, _Handle, _load_native, _place, _raw_stream

TREE_MAX = 256  # nodes of a sequence's tree

# pi to 69 digits, as a rational number: frequencies become turns without a rounding of their own
_PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816, 10 ** 69)


class _RotaryStruct(ctypes.Structure):  # pi_attn_rotary_t
    _fields_ = [("step", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("scale", ctypes.c_float)]


class _Rope(ctypes.Structure):  # Rope of csrc/pi_paged_py.cpp
    _fields_ = [("rotary", _RotaryStruct), ("device", ctypes.c_int)]


class _Layers(ctypes.Structure):  # Layers of csrc/pi_paged_py.cpp
    _fields_ = [("first", _Handle), ("caches", ctypes.POINTER(_CacheStruct)), ("n", ctypes.c_int)]


def _layers(caches) -> _Layers:
    array = (_CacheStruct * len(caches))(*(c._struct.cache for c in caches))
    s = _Layers(caches[0]._struct, array, len(caches))
    s.array = array  # (lives as long as the struct)
    return s


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: int = 0,
                       low: float = 1.0, high: float = 32.0):
    """Radians per position of the rot / 2 pairs, as a list, and the factor of the turned elements.

    f_t = base^(-2 t / rot), scaled for contexts `factor` times as long as trained on:
      "linear"  f_t / factor (positions interpolated);
      "ntk"     with base * factor^(rot / (rot - 2)): the slowest pair is interpolated, the fastest kept;
      "yarn"    pairs that make at least `high` turns over the `original` length kept, those with at most `low` interpolated, in
                between a mix that is linear in the number of turns, as the method was published; the factor is 0.1 ln(factor) + 1.
                Much model code mixes linearly in the pair's number t instead, between two rounded bounds: the frequencies in
                between differ by up to three times, so a checkpoint trained with that code needs its own list (Rotary's `freqs`).
    """
    if rot <= 0 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot of at least 4")
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * t / rot) for t in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "yarn":
        return f, 1.0
    if original <= 0 or not high > low:
        raise ValueError("yarn scaling needs the original length, and high above low")
    keep = [min(1.0, max(0.0, (original * x / (2 * math.pi) - low) / (high - low))) for x in f]
    return [x * g + x * (1 - g) / factor for x, g in zip(f, keep)], 0.1 * math.log(factor) + 1.0


class Rotary:
    """Frequencies of rotary positions on a device: a row's first `rot` elements turn in pairs, (t, t + rot / 2) or, interleaved,
    (2 t, 2 t + 1).  Frequencies from :func:`rotary_frequencies`, or given in radians per position (`freqs`, rot / 2 of them);
    `scale` multiplies the turned elements (default: the scaling's own factor).
    Its device memory is not handed out again before calls enqueued with it are done, whatever their stream; a captured graph
    of such calls reads it at every replay, so keep the object as long as the graph."""

    def __init__(self, rot: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                 original: int = 0, low: float = 1.0, high: float = 32.0, freqs: Optional[Sequence[float]] = None,
                 scale: Optional[float] = None, device="cuda"):
        if rot <= 0 or rot % 16:
            raise ValueError("rot must be a positive multiple of 16")
        own = 1.0
        if freqs is None:
            freqs, own = rotary_frequencies(rot, base, scaling, factor, original, low, high)
        self.freqs = [float(f) for f in freqs]
        if len(self.freqs) != rot // 2 or not all(map(math.isfinite, self.freqs)):
            raise ValueError("freqs must be rot / 2 finite numbers")
        self.rot, self.interleaved, self.scale = rot, bool(interleaved), own if scale is None else float(scale)
        if not math.isfinite(self.scale):
            raise ValueError("scale must be finite")
        steps = [round(Fraction(f) * 2 ** 63 / _PI) % 2 ** 64 for f in self.freqs]  # turns per position in 2^-64
        self.steps = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in steps], dtype=torch.int64, device=device)
        self.device, self.index = self.steps.device, self.steps.get_device()
        self._struct = _Rope(_RotaryStruct(self.steps.data_ptr(), rot, int(self.interleaved), self.scale), self.index)
        self._handle = ctypes.addressof(self._struct)
        self._streams = {_raw_stream(self.index)} if self.index >= 0 else {0}  # that the allocator knows to read the steps

    def _used_on(self, raw: int) -> None:
        """The steps are about to be read on the current stream, `raw`, which is not the one that they were made on."""
        self.steps.record_stream(torch.cuda.current_stream(self.index))
        self._streams.add(raw)


class CacheLayers:
    """The layers of a model whose caches have the same type and sizes and share their page tables."""

    def __init__(self, caches: Sequence[PagedCache]):
        self.caches = tuple(caches)
        if not self.caches:
            raise ValueError("no caches")
        first = self.caches[0]
        for c in self.caches:
            if c.index != first.index or c.kv_type != first.kv_type or c.k.shape != first.k.shape:
                raise ValueError("the layers' caches must have the same type and sizes and lie on one device")
        self.device, self.index = first.device, first.index
        self._struct = _layers(self.caches)
        self._handle = ctypes.addressof(self._struct)


_Where = namedtuple("_Where", "device index")


def _turn(q, k, rope, start, pos, q_out, k_out, back, stream, check):
    if stream is not None or rope.index != _current_device():
        with _place(rope, stream):
            return _turn(q, k, rope, start, pos, q_out, k_out, back, None, check)
    raw = _raw_stream(rope.index)
    if raw not in rope._streams:
        rope._used_on(raw)
    rc, q_out, k_out = (paged._native or _load_native()).rotary(q, k, rope._handle, start, pos, q_out, k_out, back, raw)
    if rc or check:
        _check("pi_attn_rotary", rc, None, check)
    return q_out, k_out


def rotary(q, k, rope: Rotary, start: int = 0, pos=None, q_out=None, k_out=None, stream=None, check=False):
    """pi_attn_rotary: q [B, H, N, d] and k [B, Hkv, N, d] (or None), bf16 or fp32, turned by their positions: start, start + 1,
    ..., or pos [B, N] int32.  Any strides of whole rows; new outputs are contiguous, as :func:`fwd` takes them.  An output
    may be its input.  Returns (q, k)."""
    return _turn(q, k, rope, start, pos, q_out, k_out, 0, stream, check)


def rotary_bwd(dq, dk, rope: Rotary, start: int = 0, pos=None, q_out=None, k_out=None, stream=None, check=False):
    """pi_attn_rotary's transpose: the gradients of :func:`rotary`'s inputs, given those of its outputs.  Arguments as there."""
    return _turn(dq, dk, rope, start, pos, q_out, k_out, 1, stream, check)


def rotary_append(q, k, v, rope: Rotary, cache: PagedCache, table, cu, ctx, parent=None, q_out=None, stream=None, check=False):
    """pi_attn_rotary_append: the packed new tokens q [T, H, d], k, v [T, Hkv, d] bf16 (tokens any stride apart): keys turned by their
    positions and values go into the pages, the turned queries are returned (into q_out, which may be q).  parent [T] int32:
    the tokens are nodes of trees, and a position is ctx plus the node's depth; None: they follow one another."""
    if stream is not None or cache.index != _current_device():
        with _place(cache, stream):
            return rotary_append(q, k, v, rope, cache, table, cu, ctx, parent, q_out, None, check)
    raw = _raw_stream(cache.index)
    if raw not in rope._streams and rope.index == cache.index:  # (else the call refuses it)
        rope._used_on(raw)
    rc, q_out = (paged._native or _load_native()).rotary_append(q, k, v, rope._handle, cache._handle, table, cu, ctx, parent, q_out, raw)
    if rc or check:
        _check("pi_attn_rotary_append", rc, None, check)
    return q_out


def extend_tree(q, cache: PagedCache, table, cu, ctx, parent, alpha, k_local: int, period: int, S: int, mode: int = MODE_PI,
                out=None, lse=None, stream=None, check=False):
    """pi_attn_extend_tree: :func:`extend` for trees of drafted tokens, whose rows the cache holds: node j of sequence b in row
    ctx[b] + j, with parent [T] int32 (a node number, or -1).  Returns (out, lse)."""
    if stream is not None or cache.index != _current_device():
        with _place(cache, stream):
            return extend_tree(q, cache, table, cu, ctx, parent, alpha, k_local, period, S, mode, out, lse, None, check)
    rc, out, lse = (paged._native or _load_native()).extend_tree(q, cache._handle, table, cu, ctx, parent, alpha, k_local, period, S, mode, out,
                                                                 lse, _raw_stream(cache.index))
    if rc or check:
        _check("pi_attn_extend_tree", rc, None, check)
    return out, lse


def verify_tree(target, draft, tokens, cu, parent, u, u_next, path=None, count=None, next=None, stream=None, check=False):
    """pi_attn_verify_tree: target [T, V] fp32 probabilities after every node, draft [T, V] those that its children were drawn from
    (None: chosen tokens), tokens, parent [T] int32, cu [B + 1] int32, random numbers u [T], u_next [B] fp32 in [0, 1).
    Returns (path [T], count [B], next [B]) int32: sequence b's accepted nodes from path[cu[b]] on, how many, and its next token."""
    if not isinstance(target, torch.Tensor):
        raise ValueError(f"target must be fp32 [T, V], got {type(target).__name__}")
    index = target.get_device()
    if stream is not None or index != _current_device():
        with _place(_Where(target.device, index), stream):
            return verify_tree(target, draft, tokens, cu, parent, u, u_next, path, count, next, None, check)
    rc, path, count, next = (paged._native or _load_native()).verify(target, draft, tokens, cu, parent, u, u_next, path, count, next,
                                                                     _raw_stream(index))
    if rc or check:
        _check("pi_attn_verify_tree", rc, None, check)
    return path, count, next


def cache_keep(cache, table, cu, ctx, path, count, stream=None, check=False) -> None:
    """pi_attn_cache_keep: in a :class:`PagedCache` or all :class:`CacheLayers`, row ctx[b] + path[cu[b] + j] goes to row
    ctx[b] + j for j < count[b]: the accepted path's rows lie together, and the next step's ctx is ctx + count."""
    if stream is not None or cache.index != _current_device():
        with _place(cache, stream):
            return cache_keep(cache, table, cu, ctx, path, count, None, check)
    handle = cache._handle
    if isinstance(cache, PagedCache):
        alone = cache._layers  # (held by this call: another thread's first one may put its own in the cache's place meanwhile)
        if alone is None:
            alone = cache._layers = _layers((cache,))
        handle = ctypes.addressof(alone)
    rc = (paged._native or _load_native()).keep(handle, table, cu, ctx, path, count, _raw_stream(cache.index))
    if rc or check:
        _check("pi_attn_cache_keep", rc, None, check)
