"""Host tests of what the step's binding keeps alive while a call, or a stream, still reads it."""
import ctypes
import threading
import weakref

import pytest
import torch

import structured_sparse_long_gb300 as pa
from structured_sparse_long_gb300 import build as pbuild
from structured_sparse_long_gb300 import paged, step


@pytest.fixture
def native(monkeypatch):
    """The extension module with the step's C functions as a test gives them (`native(rotary=..., cache_keep=...)`), on host tensors."""
    pbuild.build()
    paged._load()
    monkeypatch.setattr(paged._binding, "_expect_like", lambda t, name, like, dtype, shape: None)
    for m in (paged, step):
        monkeypatch.setattr(m, "_current_device", lambda: -1)
        monkeypatch.setattr(m, "_raw_stream", lambda index: 0)
    P, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.CFUNCTYPE
    types = dict(rotary=(P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P), rotary_append=(P, L, P, L, P, L, P, P, P, P, I, P, L, P),
                 extend_tree=(P, L, P, P, P, P, I, I, I, I, I, P, P, P), verify_tree=(P, L, P, L, P, P, P, P, P, I, I, I, P, P, P, P),
                 cache_keep=(P, I, P, P, P, P))
    held = []

    def bind(**given):
        for name, t in types.items():
            held.append(F(I, *t)(given.get(name, lambda *a: 0)))
        paged._load_native().bind_step(*(ctypes.cast(f, P).value for f in held[-len(types):]))

    yield bind
    monkeypatch.setattr(paged, "_native", None)
    paged._load_native()


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def pages(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_two_threads_keep_paths_in_a_cache_for_the_first_time(native, monkeypatch):
    """Both make the cache's descriptor before either has stored it, and then both are in the library: what each reads there is alive."""
    made, both_made, both_in, dead, seen = [], threading.Barrier(2), threading.Barrier(2), [], []
    own = step._layers

    def layers(caches):
        s = own(caches)
        made.append(weakref.ref(s))
        both_made.wait(5)
        return s

    def keep(caches, n, *rest):
        both_in.wait(5)
        dead.append(sum(r() is None for r in made))
        seen.append(paged._CacheStruct.from_address(caches).k)
        both_in.wait(5)
        return 0

    native(cache_keep=keep)
    monkeypatch.setattr(step, "_layers", layers)
    c = pa.PagedCache(pages(2, 2, 16, 64), pages(2, 2, 16, 64))
    args = (ints(3, 4), ints(4), ints(3), ints(5), ints(3))
    threads = [threading.Thread(target=pa.cache_keep, args=(c, *args)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert dead == [0, 0] and seen == [c.k.data_ptr()] * 2


def test_a_rotarys_steps_are_known_to_every_stream_that_reads_them(native, monkeypatch):
    """Else the allocator hands their memory out again once the object is gone, although another stream's call has yet to read it.  Once for
    each stream, and not for the one that they were made on."""
    native()
    r = pa.Rotary(32, device="cpu")
    known, raw = [], [0]

    class Steps:
        def record_stream(self, stream):
            known.append(stream)

    r.steps = Steps()
    monkeypatch.setattr(step, "_raw_stream", lambda index: raw[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: raw[0])
    x = pages(5, 8, 64)
    c = pa.PagedCache(pages(2, 2, 16, 64), pages(2, 2, 16, 64))
    calls = (lambda: pa.rotary(pages(1, 2, 3, 64), None, r), lambda: pa.rotary_bwd(pages(1, 2, 3, 64), None, r),
             lambda: pa.rotary_append(x[:, :4], x[:, 4:6], x[:, 6:], r, c, ints(3, 4), ints(4), ints(3)))
    for i, call in enumerate(calls):
        raw[0] = 0
        call()
        assert known == list(range(1, i + 1))
        raw[0] = i + 1
        call()
        call()
        assert known == list(range(1, i + 2))


def test_the_trees_kernel_is_told_for_the_sizes_of_a_call():
    """And a call's own errors for sizes that it refuses; as if on one SM where there is no device."""
    pbuild.build()
    f, a16 = paged._load().pi_attn_debug_tree_kernel, 0x10000

    def ask(B=1, T=26, width=1100, H=16, kl=256, per=1024, S=4, mode=0, **kw):
        c = paged._CacheStruct(*(kw.get(x, y) for x, y in (("k", a16), ("v", a16), ("ks", None), ("vs", None), ("kv", 0), ("pages", 4), ("Hkv", 4),
                                                           ("page", 64), ("d", 128))))
        return f(ctypes.byref(c), B, T, width, H, kl, per, S, mode)

    assert ask() in (0, 1) and ask(H=80) == 1  # (20 heads on one)
    assert ask(k=None) == -1 and ask(B=0) == ask(T=0) == ask(H=6) == ask(per=0) == -2
    assert ask(d=96) == ask(mode=2) == ask(T=1 << 28) == -3 and ask(v=a16 + 8) == -4
