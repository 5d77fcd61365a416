"""Host tests of the paged kernels' own work-list arithmetic: csrc/pi_plan.cuh, which the kernels include, compiled for the
host.  Blocks cover every token, tiles every attended key once, slots every attended tile within the workspace's bound, groups
every token, and the search finds every sequence without leaving its array."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from structured_sparse_long_gb300 import build as pbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    target = str(tmp_path_factory.mktemp("paged_arithmetic") / "libpaged_arithmetic.so")
    cmd = [pbuild.nvcc(), "-shared", os.path.join(HERE, "paged_arithmetic.cu"), "-o", target] + pbuild.ARCH_FLAGS + pbuild.NVCC_FLAGS
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(target)
    L = ctypes.c_longlong
    lib.block_bound.restype = lib.slot_bound.restype = lib.token_group.restype = L
    lib.block_bound.argtypes = [L, L, ctypes.c_int]
    lib.slot_bound.argtypes = [ctypes.c_int] * 4 + [L] * 3
    return lib


def numbers(f, *args, n):
    out = (ctypes.c_int * n)()
    f(*(int(a) for a in args), out)
    return list(out)


def attended(i, k, period, S, ecp):
    lo = max(0, (i // k - 1) * k) if ecp else max(0, i - k)
    far = [] if ecp else [i - m * period for m in range(1, S + 1) if m * period > k and i >= m * period]
    return list(range(lo, i + 1)), far


def draw(rng):
    ecp = rng.random() < 0.2
    k = int(rng.integers(1 if ecp else 0, 300))
    return k, int(rng.choice([1, 7, 31, 32, 33, 64, 100, 256, 1024])), 0 if ecp else int(rng.integers(0, 7)), ecp


@pytest.mark.parametrize("R", [32, 64, 128])
def test_blocks_cover_every_token(lib, R):
    rng = np.random.default_rng(R)
    for n in list(range(1, 3 * R + 2)) + [1000, 65536]:
        ctx, t0 = int(rng.integers(0, 1000)), int(rng.integers(0, 1000))
        if n % 3 == 0:
            ctx = ctx // R * R
        count, at = lib.n_blocks(n, ctx, R), ctx
        for x in range(count):
            p0, tq, first, last, *_ = numbers(lib.block, 20, 32, 2, 0, R, t0, n, ctx, x, n=8)
            assert first == at and p0 <= first <= last < p0 + R and tq == t0 + p0 - ctx
            at = last + 1
        assert at == ctx + n and count <= lib.block_bound(n, 1, R)
    for _ in range(200):  # a batch's blocks, empty sequences among them
        n = rng.integers(0, 3 * R, int(rng.integers(1, 40))) * (rng.random() < 0.9)
        ctx = rng.integers(0, 1000, len(n))
        T = int(n.sum()) + int(rng.integers(0, 9))
        used = sum(lib.n_blocks(int(m), int(c), R) for m, c in zip(n, ctx) if m)
        assert used <= lib.block_bound(T, len(n), R)


@pytest.mark.parametrize("R", [32, 64, 128])
def test_tiles_hold_every_attended_key_once(lib, R):
    """Of every block the tiles' ranges, cut to what a query attends, are its keys, each once; and tiles without masks lie inside
    the band of every query of the block."""
    rng = np.random.default_rng(100 + R)
    for _ in range(150):
        k, period, S, ecp = p = draw(rng)
        n, ctx = int(rng.integers(1, 300)), int(rng.integers(0, 3000))
        x = int(rng.integers(0, lib.n_blocks(n, ctx, R)))
        _, _, first, last, tiles, n_band, full_lo, full_hi = numbers(lib.block, *p, R, 0, n, ctx, x, n=8)
        ranges = [numbers(lib.tile, *p, R, n, ctx, x, t, 0, n=5) for t in range(tiles)]
        for t, (key0, back, lo, hi, _) in enumerate(ranges):
            assert (key0 % 32 == 0 and key0 <= lo and hi < key0 + 32 and lo >= 0) or lo > hi
            assert (back == 0) == (t < n_band)
            if full_lo <= t <= full_hi and t < n_band:
                for i in (first, last):
                    band, _ = attended(i, k, period, S, ecp)
                    assert band[0] <= key0 and key0 + 31 <= band[-1]
        for i in {first, last, int(rng.integers(first, last + 1))}:
            band, far = attended(i, k, period, S, ecp)
            got = []
            for key0, back, lo, hi, _ in ranges:
                if back == 0:
                    got += range(max(lo, band[0]), min(hi, i) + 1)
                elif lo <= i - back <= hi:
                    got.append(i - back)
            assert sorted(got) == sorted(band + far)


def test_slots_hold_every_attended_tile_within_the_bound(lib):
    """The slot that the attention looks a tile up in is the one that the conversion fills with it, and a batch's slots fit."""
    rng = np.random.default_rng(0)
    for _ in range(300):
        k, period, S, ecp = p = draw(rng)
        used, T, B = 0, 0, int(rng.integers(1, 5))
        for _ in range(B):
            ctx, n, R = int(rng.integers(0, 2000)), int(rng.integers(1, 400)), int(rng.choice([32, 64, 128]))
            slots = lib.n_slots(*p, n, ctx)
            held = [lib.tile_of_slot(*p, n, ctx, x) for x in range(slots)]
            for x in {0, lib.n_blocks(n, ctx, R) - 1, int(rng.integers(0, lib.n_blocks(n, ctx, R)))}:
                tiles = numbers(lib.block, *p, R, 0, n, ctx, x, n=8)[4]
                for t in range(tiles):
                    key0, _, lo, hi, slot = numbers(lib.tile, *p, R, n, ctx, x, t, used, n=5)
                    if lo <= hi:  # (a tile without an attended key is not looked up)
                        assert 0 <= slot - used < slots and held[slot - used] == key0 >> 5
            used, T = used + slots, T + n
        assert used <= lib.slot_bound(*p, B, T, 2500)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 8])
def test_token_groups_have_their_places(lib, group):
    rng = np.random.default_rng(group)
    for B in (1, 2, 7, 40):
        n = rng.integers(0, 12, B)
        cu = np.concatenate([[0], np.cumsum(n)])
        T = int(cu[-1]) + int(rng.integers(0, 5))
        start = lambda j: lib.token_group(j, int(cu[j]), group)  # noqa: E731
        seen = []
        for i in range((T + B * (group - 1)) // group):  # the grid
            b = sum(start(j) <= i for j in range(1, B + 1))
            if b < B and 0 <= (i - start(b)) * group < n[b]:
                seen.append((b, (i - start(b)) * group))
        assert seen == [(b, x) for b in range(B) for x in range(0, n[b], group)]


def test_sequence_search(lib):
    """Finds every token's sequence in sorted offsets, and stays inside cu[1 .. B] and ends for any others."""
    rng = np.random.default_rng(0)

    def search(cu, B, t):
        cu, outside = np.ascontiguousarray(cu, dtype=np.int32), ctypes.c_int()
        found = lib.search(cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), B, int(t), ctypes.byref(outside))
        assert outside.value == 0
        return found

    for B in list(range(1, 70)) + [300, 1024, 1100, 5000, 65535]:
        cu = np.concatenate([[0], np.cumsum(rng.integers(0, 3, B))])
        for t in rng.integers(0, cu[-1] + 3, 20):
            assert search(cu, B, t) == np.searchsorted(cu[1:], t, side="right")
        wild = rng.integers(-2 ** 31, 2 ** 31, B + 1)
        for t in rng.integers(0, 1000, 5):
            assert 0 <= search(wild, B, t) <= B
