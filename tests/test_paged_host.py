"""Host-only tests of the paged cache: refusals of the C ABI and of the binding before anything is launched,
the 64-bit format reference against torch's own conversions, and the sequence search's arithmetic."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
from structured_sparse_long_gb300 import build as pbuild
from structured_sparse_long_gb300 import paged

PI_ERR_NULL, PI_ERR_SHAPE, PI_ERR_UNSUPPORTED, PI_ERR_ALIGN, PI_ERR_WORKSPACE = -1, -2, -3, -4, -5
A16 = 0x10000  # fake, 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return paged._load()


def cache(k=A16, v=A16, ks=None, vs=None, kv_type=0, n_pages=4, Hkv=2, page=32, d=64):
    return ctypes.byref(paged._CacheStruct(k, v, ks, vs, kv_type, n_pages, Hkv, page, d))


def batch(table=A16, cu=A16, ctx=A16, B=2, T=5, width=4):
    return ctypes.byref(paged._BatchStruct(table, cu, ctx, B, T, width))


def append(lib, k=A16, v=A16, ks=128, vs=128, c=None, b=None):
    return lib.pi_attn_cache_append(k, v, ks, vs, c or cache(), b or batch(), None)


def read(lib, k=A16, v=A16, c=None, b=None):
    return lib.pi_attn_cache_read(c or cache(), b or batch(), k, v, None)


def extend(lib, q=A16, qs=256, c=None, b=None, alpha=A16, H=4, kl=8, per=16, S=1, mode=0, out=A16, lse=A16, ws=A16,
           ws_bytes=1 << 20):
    return lib.pi_attn_extend(q, qs, c or cache(), b or batch(), alpha, H, kl, per, S, mode, out, lse, ws, ws_bytes, None)


def decode(lib, q=A16, qs=256, c=None, table=A16, lens=A16, B=2, width=4, alpha=A16, H=4, kl=8, per=16, S=1, mode=0,
           out=A16, lse=A16):
    return lib.pi_attn_decode_paged(q, qs, c or cache(), table, lens, B, width, alpha, H, kl, per, S, mode, out, lse, None)


CALLS = [append, read, extend, decode]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), PI_ERR_NULL), (dict(v=None), PI_ERR_NULL), (dict(kv_type=3), PI_ERR_UNSUPPORTED),
    (dict(kv_type=1), PI_ERR_NULL), (dict(kv_type=2, ks=A16), PI_ERR_NULL), (dict(n_pages=0), PI_ERR_SHAPE),
    (dict(Hkv=0), PI_ERR_SHAPE), (dict(d=32), PI_ERR_UNSUPPORTED), (dict(d=96), PI_ERR_UNSUPPORTED),
    (dict(page=8), PI_ERR_UNSUPPORTED), (dict(page=48), PI_ERR_UNSUPPORTED), (dict(page=512), PI_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 26, page=16), PI_ERR_UNSUPPORTED),  # 2^31 rows
    (dict(k=A16 + 8), PI_ERR_ALIGN), (dict(v=A16 + 4), PI_ERR_ALIGN),
    (dict(kv_type=1, ks=A16, vs=A16 + 8), PI_ERR_ALIGN)])
def test_cache_is_checked(lib, call, kw, code):
    assert call(lib, c=cache(**kw)) == code


@pytest.mark.parametrize("call", [append, read, extend], ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw,code", [
    (dict(table=None), PI_ERR_NULL), (dict(cu=None), PI_ERR_NULL), (dict(ctx=None), PI_ERR_NULL), (dict(B=0), PI_ERR_SHAPE),
    (dict(T=0), PI_ERR_SHAPE), (dict(width=0), PI_ERR_SHAPE), (dict(width=1 << 26), PI_ERR_UNSUPPORTED),
    (dict(cu=A16 + 2), PI_ERR_ALIGN)])
def test_batch_is_checked(lib, call, kw, code):
    assert call(lib, b=batch(**kw)) == code


def test_rows_are_checked(lib):
    for call, first in ((append, "k"), (read, "k"), (extend, "q"), (decode, "q")):
        assert call(lib, **{first: None}) == PI_ERR_NULL
        assert call(lib, **{first: A16 + 8}) == PI_ERR_ALIGN
    assert append(lib, v=None) == PI_ERR_NULL and read(lib, v=A16 + 2) == PI_ERR_ALIGN
    for bad in (127, 120, 132, 0, -128, 1 << 38):  # below a token's elements, not a multiple of 8, absurd
        assert append(lib, ks=bad) == PI_ERR_SHAPE and append(lib, vs=bad) == PI_ERR_SHAPE
    for call in (extend, decode):
        assert call(lib, qs=248) == PI_ERR_SHAPE and call(lib, qs=260) == PI_ERR_SHAPE


@pytest.mark.parametrize("call", [extend, decode], ids=lambda f: f.__name__)
def test_attention_is_checked(lib, call):
    assert call(lib, out=None) == PI_ERR_NULL and call(lib, lse=None) == PI_ERR_NULL
    assert call(lib, alpha=None) == PI_ERR_NULL                       # pi mode needs alpha
    assert call(lib, H=3) == PI_ERR_SHAPE and call(lib, H=0) == PI_ERR_SHAPE
    assert call(lib, kl=-1) == PI_ERR_SHAPE and call(lib, S=-1) == PI_ERR_SHAPE
    assert call(lib, per=0) == PI_ERR_SHAPE
    assert call(lib, mode=2) == PI_ERR_UNSUPPORTED and call(lib, mode=5) == PI_ERR_UNSUPPORTED
    assert call(lib, mode=1, kl=0, S=0) == PI_ERR_SHAPE and call(lib, mode=1, kl=8, S=1) == PI_ERR_SHAPE
    assert call(lib, out=A16 + 8) == PI_ERR_ALIGN and call(lib, lse=A16 + 2) == PI_ERR_ALIGN
    assert call(lib, alpha=A16 + 1) == PI_ERR_ALIGN


def test_sizes_past_the_limits(lib):
    assert extend(lib, b=batch(T=1 << 29), H=4) == PI_ERR_UNSUPPORTED    # 2^31 rows of lse
    assert decode(lib, H=34, qs=34 * 64) == PI_ERR_UNSUPPORTED           # 17 query heads per KV head
    assert decode(lib, B=70000) == PI_ERR_UNSUPPORTED and decode(lib, B=0) == PI_ERR_SHAPE
    for call, kw in ((extend, dict(b=batch(width=1 << 25))), (decode, dict(width=1 << 25))):  # 2^30 positions, as many skips
        assert call(lib, per=1, S=1 << 30, **kw) == PI_ERR_UNSUPPORTED
    assert decode(lib, width=0) == PI_ERR_SHAPE and decode(lib, lens=None) == PI_ERR_NULL
    assert decode(lib, table=A16 + 2) == PI_ERR_ALIGN


def workspace(lib, c=None, B=2, T=5, width=4, H=4, kl=8, per=16, S=1, mode=0):
    return lib.pi_attn_extend_workspace_size(c or cache(), B, T, width, H, kl, per, S, mode)


def test_extend_workspace(lib):
    """A plan of at most T / R + 2 min(B, T) blocks of 80 bytes and its head; refused where the call would be."""
    for B, T in ((1, 65536), (16, 8000), (300, 30000)):
        need = workspace(lib, B=B, T=T, width=1 << 20)
        plan = 32 + 80 * (T // 64 + 2 * min(B, T))  # two query heads per KV head: 64 positions per block
        assert need == -(-plan // 256) * 256
        for ws in (dict(ws_bytes=need - 1), dict(ws=None)):
            assert extend(lib, b=batch(B=B, T=T, width=1 << 20), **ws) == PI_ERR_WORKSPACE
    quant, big = cache(kv_type=1, ks=A16, vs=A16), dict(T=8000, width=1 << 20)
    assert workspace(lib, quant, **big) > workspace(lib, **big) > 0
    assert extend(lib, c=quant, b=batch(**big), ws_bytes=workspace(lib, quant, **big) - 1) == PI_ERR_WORKSPACE
    for B, T in ((1, 1), (1000, 30)):  # short chunks need none
        assert workspace(lib, B=B, T=T) == 0
    for bad in (dict(B=0), dict(T=0), dict(width=0), dict(H=3), dict(kl=-1), dict(mode=2), dict(c=cache(d=96))):
        assert workspace(lib, **bad) == 0
    assert extend(lib, ws=A16 + 16) == PI_ERR_ALIGN


def seq_tiles(n, ctx, k, period, S, ecp):
    """The plan kernel's bf16 tiles of one sequence over an 8-bit cache: their list, and the slot of a band tile or of
    tile x of the window at distance back."""
    last = ctx + n - 1
    band0 = max(0, (ctx // k - 1) * k) if ecp else max(0, ctx - k)
    m_first = 1 if ecp or not S else min(k // period + 1, S + 1)
    windows = 0 if ecp or not S else max(0, min(S, last // period) - m_first + 1)
    lo, per_window = band0 >> 5, ((n - 1) >> 5) + 2
    band = (last >> 5) - lo + 1
    if windows:
        first = min(lo, max(0, ctx - (m_first + windows - 1) * period) >> 5)
        if (last >> 5) - first + 1 <= band + windows * per_window:
            return list(range(first, (last >> 5) + 1)), lambda x, back: x - first
    tiles = list(range(lo, (last >> 5) + 1))
    for m in range(m_first, m_first + windows):
        start = (ctx - m * period) >> 5
        tiles += [x if x <= (last - m * period) >> 5 else -1 for x in range(start, start + per_window)]
    return tiles, lambda x, back: x - lo if not back else band + (back // period - m_first) * per_window + x - ((ctx - back) >> 5)


def test_converted_tiles_hold_every_attended_key_within_the_bound(lib):
    """Every attended key's tile has a slot that holds it, and a batch's slots fit the workspace whatever its lengths."""
    rng = np.random.default_rng(0)
    for _ in range(400):
        ecp = rng.random() < 0.2
        k, period, S = int(rng.integers(1, 300)), int(rng.integers(1, 400)), 0 if ecp else int(rng.integers(0, 6))
        used, T, B = 0, 0, int(rng.integers(1, 4))
        for _ in range(B):
            ctx, n = int(rng.integers(0, 2000)), int(rng.integers(1, 400))
            tiles, slot = seq_tiles(n, ctx, k, period, S, ecp)
            used, T = used + len(tiles), T + n
            for i in {ctx, ctx + n - 1, int(rng.integers(ctx, ctx + n))}:
                lo = max(0, (i // k - 1) * k) if ecp else max(0, i - k)
                for j in range(lo, i + 1):
                    assert tiles[slot(j >> 5, 0)] == j >> 5
                for m in range(1, S + 1):
                    if m * period > k and i >= m * period:
                        assert tiles[slot((i - m * period) >> 5, m * period)] == (i - m * period) >> 5
        # (20 query heads on one: the long chunks' kernels, whatever the lengths)
        c = dict(Hkv=1, d=64, page=16)
        kw = dict(B=B, T=T, width=150, H=20, kl=k, per=period, S=S, mode=int(ecp))
        room = workspace(lib, cache(kv_type=1, ks=A16, vs=A16, **c), **kw) - workspace(lib, cache(**c), **kw)
        assert used * (8 + 2 * 32 * 64 * 2) <= room


@pytest.mark.parametrize("group", [1, 2, 3, 4, 8])
def test_token_groups_have_their_places(group):
    """The short chunks' kernel: every group of tokens of every sequence gets a CTA number of its own below the grid's size."""
    rng = np.random.default_rng(group)
    for B in (1, 2, 7, 40):
        n = rng.integers(0, 12, B)
        cu = np.concatenate([[0], np.cumsum(n)])
        T = int(cu[-1]) + int(rng.integers(0, 5))
        start = lambda j: (cu[j] + j * (group - 1)) // group  # noqa: E731
        seen = []
        for i in range((T + B * (group - 1)) // group):
            b = sum(start(j) <= i for j in range(1, B + 1))
            if b < B and 0 <= (i - start(b)) * group < n[b]:
                seen.append((b, (i - start(b)) * group))
        assert seen == [(b, x) for b in range(B) for x in range(0, n[b], group)]


def plan(n, ctx, R):
    """The plan kernel's blocks of one sequence: (p0, first, last)."""
    p = ctx if n <= R else ctx // R * R
    return [(x, max(x, ctx), min(x + R, ctx + n) - 1) for x in range(p, ctx + n, R)]


@pytest.mark.parametrize("R", [32, 64, 128])
def test_plan_covers_every_token_within_the_bound(R):
    rng = np.random.default_rng(R)
    for n in list(range(1, 3 * R + 2)) + [1000, 65536]:
        ctx = int(rng.integers(0, 1000))
        blocks = plan(n, ctx, R)
        assert [i for _, f, la in blocks for i in range(f, la + 1)] == list(range(ctx, ctx + n))
        assert len(blocks) <= n // R + 2


@pytest.mark.parametrize("period", [1, 7, 31, 32, 33, 64, 100, 1024])
def test_key_tiles_cover_what_the_queries_attend(period):
    """The 32-key tiles of a block (band, then skip windows) hold every attended key once, whatever the period."""
    rng = np.random.default_rng(period)
    for _ in range(200):
        first = int(rng.integers(0, 3000))
        last = first + int(rng.integers(0, 128))
        k, S = int(rng.integers(0, 200)), int(rng.integers(0, 6))
        m_first = min(k // period + 1, S + 1)
        lo = max(0, first - k)
        band = [(lo & ~31) + 32 * t for t in range((last - (lo & ~31)) // 32 + 1)]
        windows = max(0, min(S, last // period) - m_first + 1) if S else 0
        cpb = (last >> 5) - (first >> 5) + 1 if period % 32 == 0 else ((last - first) >> 5) + 2
        inv = 0xFFFFFFFF // cpb + 1 & 0xFFFFFFFF
        for i in (first, last, int(rng.integers(first, last + 1))):
            got = [j for t in band for j in range(max(t, max(0, i - k)), min(t + 31, i) + 1)]
            for x in range(windows * cpb):
                w = x * inv >> 32 if inv else x
                assert w == x // cpb
                back = (m_first + w) * period
                key0 = ((first - back) & ~31) + 32 * (x - w * cpb)
                if i - back >= 0 and key0 <= i - back < key0 + 32:
                    got.append(i - back)
            want = list(range(max(0, i - k), i + 1)) + [i - m * period for m in range(1, S + 1) if m * period > k and i >= m * period]
            assert sorted(got) == sorted(want)


def test_strerror_names_the_index_error(lib):
    assert lib.pi_attn_strerror(-8).startswith(b"PI_ERR_INDEX")


def test_binding_refuses_host_tensors_and_wrong_types(monkeypatch):
    z = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        paged.PagedCache(z, z)
    with pytest.raises(ValueError, match="dtype"):
        paged.PagedCache(z.float(), z.float())
    with pytest.raises(ValueError, match="k_scale"):
        paged.PagedCache(z.to(torch.int8), z.to(torch.int8))
    with pytest.raises(ValueError, match="no scales"):
        paged.PagedCache(z, z, z, z)
    # past the device check (stubbed: no GPU here; host tensors answer get_device() with -1, as their cache does),
    # everything else is still checked before the library is called
    monkeypatch.setattr(paged._binding, "_expect_like", lambda t, name, like, dtype, shape: None)
    monkeypatch.setattr(paged, "_current_device", lambda: -1)
    monkeypatch.setattr(paged, "_raw_stream", lambda index: 0)
    native = paged._load_native()
    calls = []
    never = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: calls.append(1) or 0)
    addresses = [ctypes.cast(never, ctypes.c_void_p).value] * 5
    addresses[2] = ctypes.cast(paged._load().pi_attn_extend_workspace_size, ctypes.c_void_p).value
    native.bind(*addresses)
    try:
        c = paged.PagedCache(z, z)
        table, cu = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
        ctx = torch.zeros(1, dtype=torch.int32)
        q, a = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 4)
        kv = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
        for bad in (dict(table=table.long()), dict(table=table[0]), dict(cu=cu[:1]), dict(ctx=ctx.float()), dict(ctx=[0]),
                    dict(table=table.expand(1, 4)[:, ::2]), dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)),
                    dict(q=q[0]), dict(q=None), dict(alpha=None), dict(alpha=a[:4]), dict(alpha=a.double()), dict(alpha=a.T),
                    dict(k_local=2 ** 31), dict(S=-2 ** 40), dict(out=a), dict(out=q[:4]), dict(out=q.float()), dict(lse=q),
                    dict(lse=torch.zeros(4, 5).T), dict(workspace=a), dict(workspace=torch.zeros(3, 3, dtype=torch.uint8))):
            kw = dict(q=q, cache=c, table=table, cu=cu, ctx=ctx, alpha=a, k_local=8, period=16, S=1, out=q.clone(), lse=a.clone())
            with pytest.raises(ValueError):
                paged.extend(**{**kw, **bad})
            if not {"cu", "ctx", "workspace"} & set(bad):
                del kw["cu"], kw["ctx"]
                with pytest.raises(ValueError):
                    paged.decode_paged(lens=torch.zeros(5, dtype=torch.int32), **{**kw, "table": table.expand(5, 4).contiguous(), **bad})
        for k, v in ((kv[:, :1], kv), (kv, kv[:4]), (kv[:, :, ::2], kv), (kv.float(), kv), (kv, 3)):
            with pytest.raises(ValueError):
                paged.cache_append(k, v, c, table, cu, ctx)
        for bad in (dict(k=kv.float()), dict(v=kv[:4]), dict(rows=-1), dict(start=cu)):
            with pytest.raises(ValueError):
                paged.cache_read(**{**dict(cache=c, table=table, cu=cu, start=ctx, rows=5, k=kv, v=kv), **bad})
        with pytest.raises(ValueError):
            paged.decode_paged(q, c, table, ctx, a, 8, 16, 1)  # five queries, one sequence
        # an empty call is none, and one that is right reaches the library
        assert paged.cache_append(kv[:0], kv[:0], c, table, cu, ctx) is None
        out, lse = paged.decode_paged(q[:0], c, table[:0], ctx[:0], a[:0], 8, 16, 1, out=q[:0], lse=a[:0])
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4) and not calls
        paged.cache_append(kv, kv, c, table, cu, ctx)
        assert calls == [1]
    finally:
        monkeypatch.setattr(paged, "_native", None)
        paged._load_native()


def test_reference_codes_are_torch_codes():
    """The reference's own rounding against torch's conversions, on scaled values."""
    gen = torch.Generator().manual_seed(0)
    x = (torch.randn(300, 64, generator=gen) * torch.exp2(torch.randint(-125, 110, (300, 1), generator=gen).float()))
    x = x.to(torch.bfloat16)
    for kv in ("e4m3", "int8"):
        codes, s = ref.encode(x.float().numpy(), kv)
        y = x.double().unflatten(-1, (-1, 32)) * torch.exp2(127.0 - torch.from_numpy(s).double())[..., None]
        assert (y.abs() <= ref.QMAX[kv]).all()
        grown = (y.abs().amax(-1) * 2 > ref.QMAX[kv]) | (torch.from_numpy(s) == 7)
        assert grown.all(), "a smaller scale would have done"
        y = y.flatten(-2)
        want = y.float().to(torch.float8_e4m3fn).view(torch.uint8) if kv == "e4m3" else torch.round(y).to(torch.int8).view(torch.uint8)
        assert np.array_equal(codes, want.numpy())
        held = ref.decode(codes, s, kv)
        assert np.array_equal(held, torch.from_numpy(held).to(torch.bfloat16).double().numpy())  # bf16 holds them
        # half a step of the code's grid: 2^-4 of an e4m3 value (2^-10 below its normals), 1/2 of an int8 step
        step = np.repeat(np.exp2(s.astype(float) - 127), 32, -1)
        off = np.abs(held - x.double().numpy())
        assert (off <= (np.maximum(2.0 ** -4 * np.abs(x.double().numpy()), 2.0 ** -10 * step) if kv == "e4m3" else step / 2)).all()


def search(cu, B, t, seen):
    """The kernels' sequence search (find_sequence), probe by probe."""
    lo, length = 0, B
    while length > 0:
        step = (length + 31) >> 5
        below = []
        for lane in range(32):
            k = (lane + 1) * step
            if k <= length:
                seen.append(lo + k)
            below.append(k <= length and cu[lo + k] <= t)
        c = sum(below)
        lo += c * step
        length = min(step - 1, length - c * step)
    return lo


def test_sequence_search():
    """Finds every token's sequence in sorted offsets, and stays inside cu[1 .. B] and ends for any others."""
    rng = np.random.default_rng(0)
    for B in list(range(1, 70)) + [300, 1024, 1100, 5000]:
        n = rng.integers(0, 3, B)
        cu = np.concatenate([[0], np.cumsum(n)])
        for t in rng.integers(0, cu[-1] + 3, 20):
            seen = []
            b = search(cu, B, t, seen)
            assert b == np.searchsorted(cu[1:], t, side="right")
            assert min(seen) >= 1 and max(seen) <= B
        wild = rng.integers(-2 ** 31, 2 ** 31, B + 1)
        for t in rng.integers(0, 1000, 5):
            seen = []
            assert 0 <= search(wild, B, t, seen) <= B
            assert min(seen) >= 1 and max(seen) <= B
