"""Host tests of what the paged cache's calls hand to the library: the C functions are replaced by ones that record their
arguments, so that nothing is launched, here or on a machine with a GPU."""
import ctypes

import pytest
import torch

from structured_sparse_long_gb300 import build as pbuild
from structured_sparse_long_gb300 import paged


@pytest.fixture
def calls(monkeypatch):
    """Arguments of every pi_attn_extend that the binding makes, on host tensors: (workspace, bytes)."""
    pbuild.build()
    lib = paged._load()
    monkeypatch.setattr(paged._binding, "_expect_like", lambda t, name, like, dtype, shape: None)
    monkeypatch.setattr(paged, "_current_device", lambda: -1)
    monkeypatch.setattr(paged, "_raw_stream", lambda index: 0)
    seen = []
    P, I, L, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    extend_t = ctypes.CFUNCTYPE(I, P, L, P, P, P, I, I, I, I, I, P, P, P, Z, P)
    record = extend_t(lambda *a: seen.append((a[12], a[13])) or 0)
    never = ctypes.CFUNCTYPE(I)(lambda: 1 / 0)
    address = lambda f: ctypes.cast(f, P).value  # noqa: E731
    native = paged._load_native()
    native.bind(address(never), address(never), address(lib.pi_attn_extend_workspace_size), address(record), address(never))
    yield seen
    monkeypatch.setattr(paged, "_native", None)
    paged._load_native()


def short_call(workspace):
    """One token of four heads on two: a call that needs no workspace."""
    z = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    cache = paged.PagedCache(z, z)
    q, a = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 4)
    table, cu, ctx = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    assert paged.extend_workspace_size(cache, 1, 1, 4, 4, 8, 16, 1) == 0
    paged.extend(q, cache, table, cu, ctx, a, 8, 16, 1, workspace=workspace)


def test_an_empty_workspace_is_no_workspace(calls):
    """What extend_workspace_size() asks for is accepted, zero bytes as well: an empty tensor goes in as a null pointer (it has no
    address of its own, and any other may lie on no multiple of 256)."""
    room = torch.zeros(1024, dtype=torch.uint8)
    for workspace in (None, torch.empty(0, dtype=torch.uint8), room[256:256]):
        short_call(workspace)
        assert calls.pop() == (None, 0)
    short_call(room)
    assert calls.pop() == (room.data_ptr(), 1024)


def test_a_workspace_that_is_needed_is_handed_on(calls):
    """20 query heads on one KV head: always the long chunks' kernels, which need a workspace of the size asked for."""
    z = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    cache = paged.PagedCache(z, z)
    q, a = torch.zeros(1, 20, 64, dtype=torch.bfloat16), torch.zeros(1, 20)
    batch = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    need = paged.extend_workspace_size(cache, 1, 1, 4, 20, 8, 16, 1)
    assert need > 0
    paged.extend(q, cache, *batch, a, 8, 16, 1)
    pointer, size = calls.pop()
    assert pointer and size == need
    mine = torch.zeros(need, dtype=torch.uint8)
    paged.extend(q, cache, *batch, a, 8, 16, 1, workspace=mine)
    assert calls.pop() == (mine.data_ptr(), need)
    for small in (mine[:need - 1], mine[:0]):
        with pytest.raises(ValueError, match="workspace must hold"):
            paged.extend(q, cache, *batch, a, 8, 16, 1, workspace=small)
    assert not calls


# ------------------------------------------------------------------ sizes past the kernels' limits, through the C ABI

PI_ERR_UNSUPPORTED = -3
A16 = 0x10000  # fake, 256-byte aligned, never dereferenced: validation fails first


def sizes(T, B=1, Hkv=1, width=4, kv_type=1):
    cache = paged._CacheStruct(A16, A16, A16, A16, kv_type, 4, Hkv, 256, 128)
    return ctypes.byref(cache), ctypes.byref(paged._BatchStruct(A16, A16, A16, B, T, width))


def test_rows_past_the_grids_are_refused():
    """A launch has at most 2^31 - 1 warps, of 256 elements of a token each."""
    pbuild.build()
    lib = paged._load()
    for T, Hkv in ((2 ** 31 - 1, 64), (2 ** 30, 5), (2 ** 16, 65535)):
        for kv_type in (0, 1, 2):
            c, b = sizes(T, Hkv=Hkv, kv_type=kv_type)
            assert lib.pi_attn_cache_append(A16, A16, Hkv * 128, Hkv * 128, c, b, None) == PI_ERR_UNSUPPORTED
            assert lib.pi_attn_cache_read(c, b, A16, A16, None) == PI_ERR_UNSUPPORTED


@pytest.mark.parametrize("T,B,H,Hkv,width,k_local", [
    (2 ** 16, 2 ** 16, 20, 1, 2 ** 12, 2 ** 20),      # 2^31 converted tiles
    (2 ** 20, 2 ** 20, 128, 128, 2 ** 13, 2 ** 11),   # 2^26 of each of 128 heads
    (2 ** 30, 2 ** 30, 1, 1, 2 ** 22, 2 ** 30),       # a workspace of 2^68 bytes
    (2 ** 31 - 1, 5, 2, 1, 4, 8),                     # 2^32 rows
])
def test_chunks_past_the_conversion_are_refused(T, B, H, Hkv, width, k_local):
    """What the 8-bit kernels cannot number is refused as unsupported, and no workspace size is made up for it.  (All of these are
    calls of the long chunks' kernels, whatever the device: 20 heads on one, or more than 65535 groups of tokens.)"""
    pbuild.build()
    lib = paged._load()
    for kv_type in (1, 2):
        c, b = sizes(T, B, Hkv, width, kv_type)
        assert lib.pi_attn_extend_workspace_size(c, B, T, width, H, k_local, 1, 0, 0) == 0
        args = (A16, H * 128, c, b, A16, H, k_local, 1, 0, 0, A16, A16, A16, 2 ** 64 - 1, None)
        assert lib.pi_attn_extend(*args) == PI_ERR_UNSUPPORTED


def test_skips_are_counted_as_far_as_the_table_reaches():
    """A token attends no more skips than lie before it: 128 of 2^20 positions under a table of 2^27 positions, however
    large S is, so a single token stays a short call, which needs no workspace."""
    pbuild.build()
    lib = paged._load()
    for S in (128, 2 ** 20, 2 ** 27, 2 ** 31 - 1):
        for H, Hkv in ((4, 4), (16, 4)):
            c, _ = sizes(1, 1, Hkv, 2 ** 19)
            assert lib.pi_attn_extend_workspace_size(c, 1, 1, 2 ** 19, H, 8, 2 ** 20, S, 0) == 0


def test_the_workspace_size_is_the_cache_devices(calls, monkeypatch):
    """The size depends on the device (its SMs choose the kernel): it is asked for with the cache's device current, as the call's is."""
    import contextlib
    current, asked = [3], []

    @contextlib.contextmanager
    def place(cache, stream):
        before, current[0] = current[0], cache.index
        yield
        current[0] = before

    lib = paged._load()
    real = lib.pi_attn_extend_workspace_size

    class Library:
        @staticmethod
        def pi_attn_extend_workspace_size(*args):
            asked.append(current[0])
            return real(*args)

    z = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    cache = paged.PagedCache(z, z)
    with monkeypatch.context() as m:
        m.setattr(paged, "_current_device", lambda: current[0])
        m.setattr(paged, "_place", place)
        m.setattr(paged, "_load", lambda: Library)
        assert paged.extend_workspace_size(cache, 1, 1, 4, 20, 8, 16, 1) > 0
    assert asked == [cache.index] and current == [3]


def test_more_sequences_than_the_search_can_number():
    """The search's probes lie up to 32 times a 32nd of B, rounded up, which has to fit an int."""
    pbuild.build()
    lib = paged._load()
    for B in (2 ** 30 + 1, 2 ** 31 - 31, 2 ** 31 - 1):
        c, b = sizes(20, B=B)
        assert lib.pi_attn_cache_append(A16, A16, 128, 128, c, b, None) == PI_ERR_UNSUPPORTED
        assert lib.pi_attn_cache_read(c, b, A16, A16, None) == PI_ERR_UNSUPPORTED
        assert lib.pi_attn_extend(A16, 128, c, b, A16, 1, 8, 1, 0, 0, A16, A16, A16, 2 ** 64 - 1, None) == PI_ERR_UNSUPPORTED
        assert lib.pi_attn_extend_workspace_size(c, B, 20, 4, 1, 8, 1, 0, 0) == 0
