"""Host tests of rotary positions and of the speculative step: refusals of the C ABI and of the binding before anything is launched,
frequencies and fixed-point turns, the reference of the verification, and what the binding hands to the library."""
import ctypes
import gc
import math
import weakref

import numpy as np
import pytest
import torch

import step_ref as sref
import structured_sparse_long_gb300 as pa
from structured_sparse_long_gb300 import build as pbuild
from structured_sparse_long_gb300 import paged, step

PI_ERR_NULL, PI_ERR_SHAPE, PI_ERR_UNSUPPORTED, PI_ERR_ALIGN = -1, -2, -3, -4
A16 = 0x10000  # fake, 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return paged._load()


def cache(k=A16, v=A16, ks=None, vs=None, kv_type=0, n_pages=4, Hkv=2, page=32, d=64):
    return paged._CacheStruct(k, v, ks, vs, kv_type, n_pages, Hkv, page, d)


def batch(table=A16, cu=A16, ctx=A16, B=2, T=5, width=4):
    return ctypes.byref(paged._BatchStruct(table, cu, ctx, B, T, width))


def turns(step_=A16, rot=32, inter=0, scale=1.0):
    return ctypes.byref(step._RotaryStruct(step_, rot, inter, scale))


def strides(*s):
    return (ctypes.c_longlong * 3)(*s)


DENSE_Q, DENSE_K = (4 * 10 * 64, 10 * 64, 64), (2 * 10 * 64, 10 * 64, 64)


def rotary(lib, q=A16, qs=DENSE_Q, k=A16, ks=DENSE_K, r=None, pos=None, start=0, B=3, H=4, Hkv=2, N=10, d=64, f32=0, qo=A16, qos=DENSE_Q,
           ko=A16, kos=DENSE_K):
    s = [x and strides(*x) for x in (qs, ks, qos, kos)]
    return lib.pi_attn_rotary(q, s[0], k, s[1], r or turns(), pos, start, B, H, Hkv, N, d, f32, 0, qo, s[2], ko, s[3], None)


def append(lib, q=A16, qs=256, k=A16, ks=128, v=A16, vs=128, r=None, c=None, b=None, parent=None, H=4, qo=A16 + 4096, qos=256):
    return lib.pi_attn_rotary_append(q, qs, k, ks, v, vs, r or turns(), ctypes.byref(c or cache()), b or batch(), parent, H, qo, qos, None)


def tree(lib, q=A16, qs=256, c=None, b=None, parent=A16, alpha=A16, H=4, kl=8, per=16, S=1, mode=0, out=A16, lse=A16):
    return lib.pi_attn_extend_tree(q, qs, ctypes.byref(c or cache()), b or batch(), parent, alpha, H, kl, per, S, mode, out, lse, None)


def verify(lib, target=A16, ts=100, draft=A16, ds=100, tokens=A16, cu=A16, parent=A16, u=A16, un=A16, B=2, T=5, V=100, path=A16, count=A16,
           nxt=A16):
    return lib.pi_attn_verify_tree(target, ts, draft, ds, tokens, cu, parent, u, un, B, T, V, path, count, nxt, None)


def keep(lib, caches=None, n=None, b=None, path=A16, count=A16):
    caches = [cache()] if caches is None else caches
    array = (paged._CacheStruct * max(1, len(caches)))(*caches)
    return lib.pi_attn_cache_keep(array, len(caches) if n is None else n, b or batch(), path, count, None)


def test_rotary_is_checked(lib):
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(qs=None), dict(kos=None), dict(r=turns(None))):
        assert rotary(lib, **kw) == PI_ERR_NULL
    for kw in (dict(B=0), dict(H=0), dict(Hkv=-1), dict(N=0), dict(start=-1), dict(start=2 ** 31 - 9), dict(r=turns(rot=0)), dict(r=turns(rot=24)),
               dict(r=turns(rot=80)), dict(r=turns(scale=math.inf)), dict(r=turns(scale=math.nan)), dict(qs=(4 * 640, 640, 60)),
               dict(qs=(-64, 640, 64)), dict(ks=(1 << 38, 640, 64)), dict(qos=(2560, 0, 64)), dict(kos=(1280, 640, 32))):
        assert rotary(lib, **kw) == PI_ERR_SHAPE, kw
    assert rotary(lib, f32=1, qs=(2560, 640, 62)) == PI_ERR_SHAPE
    assert rotary(lib, qos=(2568, 640, 64)) == PI_ERR_SHAPE and rotary(lib, kos=(1280, 648, 64)) == PI_ERR_SHAPE  # in place
    for kw in (dict(d=96), dict(d=16), dict(d=256), dict(H=65536), dict(B=1 << 20, N=1 << 11), dict(B=1 << 14, N=1 << 16, H=60000),
               dict(B=1 << 24, qs=(1 << 37, 640, 64))):
        assert rotary(lib, **kw) == PI_ERR_UNSUPPORTED, kw
    for kw in (dict(q=A16 + 8), dict(ko=A16 + 4), dict(pos=A16 + 2), dict(r=turns(A16 + 4))):
        assert rotary(lib, **kw) == PI_ERR_ALIGN


@pytest.mark.parametrize("call", [append, tree, keep], ids=lambda f: f.__name__)
def test_cache_and_batch_are_checked(lib, call):
    for kw, code in ((dict(k=None), PI_ERR_NULL), (dict(kv_type=3), PI_ERR_UNSUPPORTED), (dict(kv_type=1), PI_ERR_NULL),
                     (dict(n_pages=0), PI_ERR_SHAPE), (dict(d=32), PI_ERR_UNSUPPORTED), (dict(page=48), PI_ERR_UNSUPPORTED),
                     (dict(v=A16 + 8), PI_ERR_ALIGN)):
        assert (call(lib, caches=[cache(**kw)]) if call is keep else call(lib, c=cache(**kw))) == code
    for kw, code in ((dict(table=None), PI_ERR_NULL), (dict(cu=None), PI_ERR_NULL), (dict(B=0), PI_ERR_SHAPE), (dict(T=0), PI_ERR_SHAPE),
                     (dict(width=0), PI_ERR_SHAPE), (dict(B=2 ** 30 + 1), PI_ERR_UNSUPPORTED), (dict(ctx=A16 + 2), PI_ERR_ALIGN)):
        assert call(lib, b=batch(**kw)) == code


def test_append_is_checked(lib):
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(r=turns(None))):
        assert append(lib, **kw) == PI_ERR_NULL
    for kw in (dict(H=0), dict(qs=248), dict(ks=120), dict(vs=132), dict(qos=252), dict(r=turns(rot=72)), dict(qo=A16, qos=512)):
        assert append(lib, **kw) == PI_ERR_SHAPE
    assert append(lib, H=65536, qs=1 << 23, qos=1 << 23) == PI_ERR_UNSUPPORTED
    for kw in (dict(q=A16 + 8), dict(k=A16 + 2), dict(v=A16 + 8), dict(qo=A16 + 8), dict(parent=A16 + 2)):
        assert append(lib, **kw) == PI_ERR_ALIGN


def test_tree_is_checked(lib):
    for kw in (dict(q=None), dict(parent=None), dict(out=None), dict(lse=None), dict(alpha=None)):
        assert tree(lib, **kw) == PI_ERR_NULL
    for kw in (dict(H=3), dict(kl=-1), dict(S=-1), dict(per=0), dict(mode=1, kl=0, S=0), dict(mode=1, S=1), dict(qs=260)):
        assert tree(lib, **kw) == PI_ERR_SHAPE
    for kw in (dict(mode=2), dict(b=batch(T=1 << 29)), dict(H=34, qs=34 * 64, b=batch(B=1 << 30))):
        assert tree(lib, **kw) == PI_ERR_UNSUPPORTED
    for kw in (dict(out=A16 + 8), dict(lse=A16 + 2), dict(alpha=A16 + 1), dict(parent=A16 + 3), dict(q=A16 + 4)):
        assert tree(lib, **kw) == PI_ERR_ALIGN


def test_verify_is_checked(lib):
    for name in ("target", "tokens", "cu", "parent", "u", "un", "path", "count", "nxt"):
        assert verify(lib, **{name: None}) == PI_ERR_NULL
        assert verify(lib, **{name: A16 + 2}) == PI_ERR_ALIGN
    assert verify(lib, draft=A16 + 2) == PI_ERR_ALIGN
    for kw in (dict(B=0), dict(T=0), dict(V=0), dict(ts=99), dict(ds=99), dict(ts=1 << 38)):
        assert verify(lib, **kw) == PI_ERR_SHAPE
    for kw in (dict(B=65536), dict(V=2 ** 30 + 1, ts=1 << 31, ds=1 << 31), dict(T=2 ** 30, ts=2 ** 37)):
        assert verify(lib, **kw) == PI_ERR_UNSUPPORTED


def test_keep_is_checked(lib):
    assert keep(lib, n=0) == PI_ERR_SHAPE and keep(lib, path=None) == PI_ERR_NULL and keep(lib, count=None) == PI_ERR_NULL
    assert keep(lib, path=A16 + 2) == PI_ERR_ALIGN
    for kw in (dict(n_pages=5), dict(Hkv=1), dict(page=64), dict(d=128), dict(kv_type=1, ks=A16, vs=A16)):
        assert keep(lib, caches=[cache(), cache(**kw)]) == PI_ERR_SHAPE
    # the same rows twice: keys and values of one layer, of two (4 pages x 2 heads x 32 rows x 64 elements; their scales)
    step_, scales = 4 * 2 * 32 * 64, 4 * 2 * 32 * 2
    assert keep(lib) == PI_ERR_SHAPE and keep(lib, caches=[cache(v=A16 + 2 * step_ - 16)]) == PI_ERR_SHAPE
    two = [cache(v=A16 + 2 * step_), cache(k=A16 + 4 * step_, v=A16 + 6 * step_)]
    for other in (two[0], cache(k=A16 + 4 * step_, v=A16 + 16), cache(k=A16 + 4 * step_, v=A16 + 6 * step_ - 16)):
        assert keep(lib, caches=two[:1] + [other]) == PI_ERR_SHAPE
    at = A16 + 2 * step_
    assert keep(lib, caches=[cache(v=A16 + step_, ks=at, vs=at + scales - 16, kv_type=1)]) == PI_ERR_SHAPE
    assert keep(lib, caches=[cache(v=A16 + step_, ks=at - 16, vs=at + scales, kv_type=2)]) == PI_ERR_SHAPE
    assert keep(lib, caches=[cache(Hkv=65535, n_pages=1)], b=batch(B=1 << 20)) == PI_ERR_UNSUPPORTED


# ------------------------------------------------------------------ frequencies

def test_frequencies():
    f, scale = pa.rotary_frequencies(64, 10000.0)
    assert scale == 1 and f[0] == 1 and f[16] == pytest.approx(0.01, rel=1e-14) and len(f) == 32
    assert pa.rotary_frequencies(64, scaling="linear", factor=4)[0] == [x / 4 for x in f]
    n, _ = pa.rotary_frequencies(64, scaling="ntk", factor=8)
    assert n[0] == 1 and n[-1] == pytest.approx(f[-1] / 8, rel=1e-13)  # the fastest kept, the slowest interpolated
    y, m = pa.rotary_frequencies(64, scaling="yarn", factor=16, original=4096)
    assert m == pytest.approx(0.1 * math.log(16) + 1)
    for a, b in zip(f, y):
        r = 4096 * a / (2 * math.pi)
        assert b == pytest.approx(a if r >= 32 else a / 16 if r <= 1 else a * (r - 1) / 31 + a / 16 * (32 - r) / 31, rel=1e-13)
    for kw in (dict(rot=63), dict(rot=64, scaling="other"), dict(rot=64, scaling="yarn"), dict(rot=64, base=-1.0), dict(rot=2, scaling="ntk"),
               dict(rot=64, scaling="yarn", original=10, low=3.0, high=2.0)):
        with pytest.raises(ValueError):
            pa.rotary_frequencies(**kw)
    for kw in (dict(rot=24), dict(rot=0), dict(rot=32, freqs=[1.0] * 15), dict(rot=32, freqs=[math.nan] * 16), dict(rot=32, scale=math.inf)):
        with pytest.raises(ValueError):
            pa.Rotary(**kw, device="cpu")


def test_turns_in_fixed_point():
    """position * step mod 2^64 is the angle to 2^-65 turns per position, however far, for either sign; the kernel's arithmetic, restated."""
    from fractions import Fraction
    freqs = [1.0, 0.3, 1e-6, 5.5, 0.0, -0.25, math.pi, 2 ** -40]
    r = pa.Rotary(16, freqs=freqs, device="cpu")
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    for f, s in zip(freqs, r.steps.tolist()):
        for p in (0, 1, -1, 12345, 2 ** 20 + 7, 2 ** 31 - 1, -2 ** 31):
            part = Fraction((p * s) % 2 ** 64, 2 ** 64)
            want = Fraction(f) / (2 * pi) * p
            off = abs(part - want) % 1
            assert min(off, 1 - off) <= Fraction(abs(p) + 1, 2 ** 65) + Fraction(1, 2 ** 100)


# ------------------------------------------------------------------ the verification's reference

def test_reference_is_distributed_as_the_target():
    """Two children drawn from q, numbers integrated over a fine grid: the first new token's distribution is p."""
    p, q, g = np.array([0.05, 0.45, 0.3, 0.2]), np.array([0.4, 0.1, 0.2, 0.3]), 24
    grid = (np.arange(g) + 0.5) / g
    first = np.zeros(4)
    rows = np.stack([p] * 3)
    for v in range(4):
        for w in range(4):
            for a in grid:
                for b in grid[:: 2] + 0.25 / g:
                    path, _ = sref.verify(rows, np.stack([q] * 3), [0, v, w], [-1, 0, 0], [0, a, b], 0.5)
                    if len(path) == 2:
                        first[[0, v, w][path[1]]] += q[v] * q[w] / g / (g // 2)
                    else:  # the whole residual, at once
                        left = np.maximum(p - q, 0)
                        left = np.maximum(left / left.sum() - q, 0)
                        first += left / left.sum() * q[v] * q[w] / g / (g // 2)
    assert np.abs(first - p).max() < 3.0 / g


# ------------------------------------------------------------------ the binding

@pytest.fixture
def calls(monkeypatch):
    """Arguments of the step's C functions as the binding makes them, on host tensors."""
    pbuild.build()
    paged._load()
    monkeypatch.setattr(paged._binding, "_expect_like", lambda t, name, like, dtype, shape: None)
    for m in (paged, step):
        monkeypatch.setattr(m, "_current_device", lambda: -1)
        monkeypatch.setattr(m, "_raw_stream", lambda index: 0)
    seen = {}
    P, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.CFUNCTYPE

    def record(name, *types):
        f = F(I, *types)(lambda *a: seen.__setitem__(name, a) or 0)
        seen.setdefault("keep", []).append(f)
        return ctypes.cast(f, P).value

    native = paged._load_native()
    native.bind_step(record("rotary", P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P),
                     record("append", P, L, P, L, P, L, P, P, P, P, I, P, L, P),
                     record("tree", P, L, P, P, P, P, I, I, I, I, I, P, P, P),
                     record("verify", P, L, P, L, P, P, P, P, P, I, I, I, P, P, P, P), record("cache_keep", P, I, P, P, P, P))
    yield seen
    monkeypatch.setattr(paged, "_native", None)
    paged._load_native()


def three(address):
    return list((ctypes.c_longlong * 3).from_address(address))


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_rotary_binding(calls):
    r = pa.Rotary(32, device="cpu")
    x = torch.zeros(2, 5, 8, 64, dtype=torch.bfloat16).transpose(1, 2)
    q, k = pa.rotary(x[:, :4], x[:, 4:6], r, 3)
    a = calls["rotary"]
    assert a[0] == x.data_ptr() and a[2] == x.data_ptr() + 4 * 64 * 2 and a[6:14] == (3, 2, 4, 2, 5, 64, 0, 0)
    assert q.shape == (2, 4, 5, 64) and k.shape == (2, 2, 5, 64) and q.is_contiguous() and a[14] == q.data_ptr() and a[16] == k.data_ptr()
    q, k = pa.rotary_bwd(torch.zeros(2, 4, 5, 64), None, r, pos=ints(2, 5))
    a = calls["rotary"]
    assert k is None and a[9] == 0 and a[12:14] == (1, 1) and a[5]
    pa.rotary(x[:, :0], x[:, 4:6], r)  # (for the call to refuse)
    assert calls["rotary"][8:10] == (0, 2)
    f = torch.zeros(2, 4, 5, 64)
    for bad in (dict(q=f.double()), dict(q=f[0]), dict(q=f[..., ::2]), dict(q=f, k=f.bfloat16()), dict(q=f, k=f[:, :, :4]), dict(q=f, pos=ints(5)),
                dict(q=f, pos=ints(2, 5).long()), dict(q=f, q_out=f[:, :3]), dict(q=f, k_out=f), dict(q=f, start=2 ** 40), dict(q=None)):
        with pytest.raises((ValueError, TypeError)):
            pa.rotary(bad.pop("q"), bad.pop("k", None), r, **bad)


def test_step_binding(calls):
    z = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    c, r = pa.PagedCache(z, z), pa.Rotary(32, device="cpu")
    x = torch.zeros(5, 8, 64, dtype=torch.bfloat16)
    t, cu, ctx, par = ints(3, 4), ints(4), ints(3), ints(5)
    out = pa.rotary_append(x[:, :4], x[:, 4:6], x[:, 6:], r, c, t, cu, ctx)
    a = calls["append"]
    assert out.shape == (5, 4, 64) and a[1] == a[3] == a[5] == 512 and a[9] is None and a[10] == 4 and a[12] == 256
    assert pa.rotary_append(x[:, :4], x[:, 4:6], x[:, 6:], r, c, t, cu, ctx, par, x[:, :4]) is not None
    assert calls["append"][9] == par.data_ptr() and calls["append"][11] == x.data_ptr() and calls["append"][12] == 512
    out, lse = pa.extend_tree(x[:, :4], c, t, cu, ctx, par, torch.zeros(5, 4), 8, 16, 1)
    assert calls["tree"][4] == par.data_ptr() and out.shape == (5, 4, 64) and lse.shape == (5, 4)
    p = torch.zeros(5, 103)[:, :100]
    path, count, nxt = pa.verify_tree(p, None, par, cu, par, torch.zeros(5), torch.zeros(3))
    a = calls["verify"]
    assert a[1] == 103 and a[2] is None and a[9:12] == (3, 5, 100) and path.shape == (5,) and count.shape == nxt.shape == (3,)
    pa.cache_keep(c, t, cu, ctx, path, count)
    assert calls["cache_keep"][1] == 1
    pa.cache_keep(pa.CacheLayers([c, c, c]), t, cu, ctx, path, count)
    assert calls["cache_keep"][1] == 3
    calls.clear()
    al = torch.zeros(5, 4)
    for f in (lambda: pa.rotary_append(x[:, :4], x[:4, 4:6], x[:, 6:], r, c, t, cu, ctx), lambda: pa.rotary_append(x[:, :4], x[:, 4:7], x[:, 6:], r, c, t, cu, ctx),
              lambda: pa.rotary_append(x[:, :4], x[:, 4:6], x[:, 6:], r, c, t, cu, ctx, ints(4)),
              lambda: pa.rotary_append(x[:, :4], x[:, 4:6], x[:, 6:], r, c, t, cu, ctx, None, x[:, :3]),
              lambda: pa.extend_tree(x[:, :4], c, t, cu, ctx, None, al, 8, 16, 1), lambda: pa.extend_tree(x[:, :4], c, t, cu, ctx, ints(6), al, 8, 16, 1),
              lambda: pa.extend_tree(x[:, :4], c, t, cu, ctx, par.long(), al, 8, 16, 1), lambda: pa.extend_tree(x[:, :4], c, t, cu, ctx, par, None, 8, 16, 1),
              lambda: pa.verify_tree(p.double(), None, par, cu, par, torch.zeros(5), torch.zeros(3)),
              lambda: pa.verify_tree(p, p[:, :99], par, cu, par, torch.zeros(5), torch.zeros(3)),
              lambda: pa.verify_tree(p, p, par, cu, par, torch.zeros(4), torch.zeros(3)),
              lambda: pa.verify_tree(p, p, par, cu, par, torch.zeros(5), torch.zeros(2)),
              lambda: pa.verify_tree(p, p, par, cu, par, torch.zeros(5), torch.zeros(3), count=ints(4)),
              lambda: pa.verify_tree(None, p, par, cu, par, torch.zeros(5), torch.zeros(3)),
              lambda: pa.cache_keep(c, t, cu, ctx, path.long(), count), lambda: pa.cache_keep(c, t, cu, ctx, path, count[:2]),
              lambda: pa.CacheLayers([]), lambda: pa.CacheLayers([c, pa.PagedCache(z[:1], z[:1])])):
        with pytest.raises(ValueError):
            f()
    assert not calls


def test_a_cache_goes_with_its_last_reference(calls):
    """No cycle keeps pages until the collector runs, also not once their rows were moved."""
    c = pa.PagedCache(torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16))
    pages, layers = weakref.ref(c), pa.CacheLayers([c])
    for x in (c, layers):
        pa.cache_keep(x, ints(3, 4), ints(4), ints(3), ints(5), ints(3))
        assert calls["cache_keep"][1] == 1 and paged._CacheStruct.from_address(calls["cache_keep"][0]).k == c.k.data_ptr()
    gc.disable()
    try:
        del x, c, layers
        assert pages() is None
    finally:
        gc.enable()


def test_tensors_on_the_host_are_refused(monkeypatch):
    """With another device current (a call that would change to theirs and look again)."""
    for m in (paged, step):
        monkeypatch.setattr(m, "_current_device", lambda: 0)
    for f in (lambda: pa.rotary(torch.zeros(1, 1, 2, 32), None, pa.Rotary(32, device="cpu")),
              lambda: pa.verify_tree(torch.zeros(2, 3), None, ints(2), ints(2), ints(2), torch.zeros(2), torch.zeros(1))):
        with pytest.raises(ValueError, match="CUDA device"):
            f()
