"""GPU parity of the paged key/value cache: append, read back, chunk attention, single-token attention.

Codes, scales and read-back values are compared bit for bit with a 64-bit restatement of the formats;
attention with the fp64 oracle, sequence by sequence, on the values the cache holds.  Page tables are
shuffled, contexts ragged; every page row that no query attends holds NaN."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import structured_sparse_long_gb300 as pa
from structured_sparse_long_gb300 import build as pbuild

pytestmark = pytest.mark.gpu

PI, ECP = pa.MODE_PI, pa.MODE_ECP
ERR_INDEX = -8


@pytest.fixture(scope="module", autouse=True)
def built():
    pbuild.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    pa.load()
    yield
    assert pa.status() == 0


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def nan_cache(pages, Hkv, page, d, kv):
    """A cache whose every row reads as NaN."""
    if kv == "bf16":
        return pa.PagedCache(*(torch.full((pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16).cuda() for _ in range(2)))
    k, v = (torch.full((pages, Hkv, page, d), 0x7F, dtype=torch.uint8).cuda().view(ref.DTYPE[kv]) for _ in range(2))
    return pa.PagedCache(k, v, *(torch.full((pages, Hkv, page, d // 32), 255, dtype=torch.uint8).cuda() for _ in range(2)))


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen).to(torch.bfloat16)


class Batch:
    """Sequences with ctx cached rows and n new ones, their values, and a cache of NaN rows."""

    def __init__(self, ctx, n, Hkv, d, page, kv, seed, extra_tokens=0):
        self.rng, self.gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.ctx, self.n, self.kv, self.page, self.Hkv, self.d = ctx, n, kv, page, Hkv, d
        self.table, pages = ref.make_table(ctx, n, page, self.rng)
        self.cache = nan_cache(pages, Hkv, page, d, kv)
        self.cu = ref.offsets(n)
        self.T = int(self.cu[-1]) + extra_tokens
        self.k = [normal(self.gen, c + m, Hkv, d) for c, m in zip(ctx, n)]
        self.v = [normal(self.gen, c + m, Hkv, d) for c, m in zip(ctx, n)]

    def write(self, what="all", keep=None):
        """Appends rows 0 .. ctx + n of every sequence (those of the pages in keep[b], if given)."""
        for b, (c, m) in enumerate(zip(self.ctx, self.n)):
            for p in range(0, c + m, self.page):
                if keep is not None and p // self.page not in keep[b]:
                    continue
                rows = slice(p, min(p + self.page, c + m))
                cnt = rows.stop - rows.start
                pa.cache_append(self.k[b][rows].cuda(), self.v[b][rows].cuda(), self.cache, dev(self.table[b:b + 1]),
                                dev([0, cnt]), dev([p]))

    def held(self):
        """The values the cache holds for each sequence's rows, as bf16 tensors."""
        if self.kv == "bf16":
            return self.k, self.v
        return tuple([torch.from_numpy(ref.decode(*ref.encode(x.float().numpy(), self.kv), self.kv)).to(torch.bfloat16)
                      for x in xs] for xs in (self.k, self.v))


# ------------------------------------------------------------------ append and read

APPEND = [
    # kv, d, Hkv, page, ctx, n, tokens of no sequence behind the last
    ("e4m3", 128, 4, 64, [0, 63, 64, 100], [1, 1, 1, 1], 0),
    ("int8", 64, 1, 16, [5], [70], 0),
    ("bf16", 128, 2, 32, [0, 31, 7], [33, 0, 1], 5),
    ("e4m3", 64, 3, 16, [15, 0, 16, 2, 9], [0, 17, 0, 47, 1], 3),
    ("int8", 128, 12, 256, [250, 1], [7, 300], 1),
    ("bf16", 64, 16, 128, [127], [130], 0),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"{c[0]}-d{c[1]}-h{c[2]}-p{c[3]}" for c in APPEND])
def test_append_writes_the_new_rows_and_nothing_else(case):
    kv, d, Hkv, page, ctx, n, extra = case
    bt = Batch(ctx, n, Hkv, d, page, kv, seed=d + page, extra_tokens=extra)
    H = 2 * Hkv  # the projection's output: queries in front of the keys and values
    qkv = normal(bt.gen, bt.T, H + 2 * Hkv, d)
    before = [None if t is None else ref.bits(t).copy() for t in (bt.cache.k, bt.cache.v, bt.cache.k_scale, bt.cache.v_scale)]
    x = qkv.cuda()
    pa.cache_append(x[:, H:H + Hkv], x[:, H + Hkv:], bt.cache, dev(bt.table), dev(bt.cu), dev(bt.ctx))
    torch.cuda.synchronize()
    for i, (pages, scales, first) in enumerate(((bt.cache.k, bt.cache.k_scale, H), (bt.cache.v, bt.cache.v_scale, H + Hkv))):
        rows = qkv[:, first:first + Hkv]
        want, want_s = before[i], before[i + 2]
        codes, sc = (ref.bits(rows), None) if kv == "bf16" else ref.encode(rows.float().numpy(), kv)
        for b in range(len(ctx)):
            for t in range(bt.cu[b], bt.cu[b + 1]):
                pos = ctx[b] + t - bt.cu[b]
                at = (bt.table[b, pos // page], slice(None), pos % page)
                want[at] = codes[t]
                if sc is not None:
                    want_s[at] = sc[t]
        assert np.array_equal(ref.bits(pages), want)
        if sc is not None:
            assert np.array_equal(ref.bits(scales), want_s)
    # and back: exactly what the codes stand for, nothing of the tokens of no sequence
    k, v = (torch.full((bt.T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = pa.cache_read(bt.cache, dev(bt.table), dev(bt.cu), dev(bt.ctx), bt.T, k=k, v=v)
    torch.cuda.synchronize()
    m = int(bt.cu[-1])
    for t, first in zip(got, (H, H + Hkv)):
        rows = qkv[:m, first:first + Hkv].float().numpy()
        want = rows if kv == "bf16" else ref.decode(*ref.encode(rows, kv), kv)
        assert np.array_equal(t[:m].float().cpu().numpy().astype(np.float64), want)
        assert (t[m:] == 7.0).all()


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_quantisation_at_the_edges(kv):
    """Blocks whose largest magnitude is zero, the type's smallest and largest, exactly a scaled code's largest
    and just above it; every tie between codes; an infinity or a NaN in one block only."""
    q = ref.QMAX[kv]
    rows = []
    for amax in (0.0, 2.0 ** -133, 2.0 ** -120, q * 2.0 ** -120, 2.0 ** -100, 1.0, q, q * 2, 2.0 ** 100, 3.3895e38, q * 2.0 ** 110):
        for up in (1.0, 1 + 2.0 ** -7, 1 - 2.0 ** -7):
            x = np.linspace(-1, 1, 128) * amax * up
            x[::32] = amax * up
            rows.append(x)
    ties = np.concatenate([np.arange(128) + 0.5, -(np.arange(128) + 0.5)]).reshape(2, 128) * (1 if kv == "int8" else 2.0 ** -9)
    rows += [np.clip(t, -q, q) for t in ties]
    bad = np.ones((3, 128))
    bad[0, 40], bad[1, 127], bad[2, 0] = np.inf, np.nan, -np.inf
    x = torch.from_numpy(np.concatenate([np.stack(rows), bad])).to(torch.bfloat16)[:, None].contiguous()
    T = x.shape[0]
    cache = pa.PagedCache.empty(-(-T // 16), 1, 16, 128, ref.DTYPE[kv])
    table, cu, ctx = dev(np.arange(-(-T // 16))[None]), dev([0, T]), dev([0])
    pa.cache_append(x.cuda(), (-x).cuda(), cache, table, cu, ctx)
    k, v = pa.cache_read(cache, table, cu, ctx, T)
    torch.cuda.synchronize()
    for got, pages, scales, src in ((k, cache.k, cache.k_scale, x), (v, cache.v, cache.v_scale, -x)):
        codes, sc = ref.encode(src.float().numpy(), kv)
        assert np.array_equal(ref.bits(pages).reshape(-1, 1, 128)[:T], codes)
        assert np.array_equal(ref.bits(scales).reshape(-1, 1, 4)[:T], sc)
        assert np.array_equal(got.float().cpu().numpy().astype(np.float64), ref.decode(codes, sc, kv), equal_nan=True)


@pytest.mark.parametrize("B", [1, 31, 32, 33, 300, 1100])
def test_tokens_find_their_sequence(B):
    """Batches up to several rounds of the search, empty sequences among them."""
    rng = np.random.default_rng(B)
    n = rng.integers(0, 3, B)
    n[rng.integers(0, B)] = 40
    ctx = rng.integers(0, 20, B)
    bt = Batch(list(ctx), list(n), 1, 64, 16, "bf16", seed=B)
    pos = np.concatenate([c + np.arange(m) for c, m in zip(ctx, n)])
    seq = np.repeat(np.arange(B), n)
    x = (torch.from_numpy(seq * 64.0 + pos)[:, None, None] % 251 + torch.arange(64)).to(torch.bfloat16)
    pa.cache_append(x.cuda(), x.cuda(), bt.cache, dev(bt.table), dev(bt.cu), dev(ctx))
    k, _ = pa.cache_read(bt.cache, dev(bt.table), dev(bt.cu), dev(ctx), len(x))
    torch.cuda.synchronize()
    assert torch.equal(k.cpu(), x)
    got = bt.cache.k.cpu()[bt.table[seq, pos // 16], 0, pos % 16]
    assert torch.equal(got, x[:, 0])


@pytest.mark.parametrize("kv,Hkv,d", [("e4m3", 1, 64), ("int8", 3, 64), ("e4m3", 2, 128), ("bf16", 1, 64)])
def test_append_of_a_long_call(kv, Hkv, d):
    """Calls long enough for two tokens per warp: sequences that start and end between the two, empty ones, tokens behind
    the last sequence, a bad page in the middle."""
    n, ctx = [7001, 0, 12990, 1, 1, 33, 4000], [5, 0, 16, 3, 0, 15, 1]
    bt = Batch(ctx, n, Hkv, d, 16, kv, seed=d + Hkv, extra_tokens=4)
    k, v = normal(bt.gen, bt.T, Hkv, d), normal(bt.gen, bt.T, Hkv, d)
    table = bt.table.copy()
    table[2, 100] = 2 ** 30
    before = ref.bits(bt.cache.k).copy()
    pa.cache_append(k.cuda(), v.cuda(), bt.cache, dev(table), dev(bt.cu), dev(ctx))
    assert pa.status() == ERR_INDEX
    seq = np.repeat(np.arange(len(n)), n)
    pos = np.concatenate([c + np.arange(m) for c, m in zip(ctx, n)])
    kept = ~((seq == 2) & (pos // 16 == 100))
    at = bt.table[seq, pos // 16][kept], pos[kept] % 16
    for x, pages, scales in ((k, bt.cache.k, bt.cache.k_scale), (v, bt.cache.v, bt.cache.v_scale)):
        rows = x[:len(seq)][torch.from_numpy(kept)]
        codes, sc = (ref.bits(rows), None) if kv == "bf16" else ref.encode(rows.float().numpy(), kv)
        got = ref.bits(pages)
        assert np.array_equal(got[at[0], :, at[1]], codes)
        assert sc is None or np.array_equal(ref.bits(scales)[at[0], :, at[1]], sc)
        rest = np.ones(got.shape[:1] + got.shape[2:3], dtype=bool)  # [page, row]
        rest[at] = False
        assert np.array_equal(got.transpose(0, 2, 1, 3)[rest], before.transpose(0, 2, 1, 3)[rest])


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
def test_read_of_a_long_call(kv):
    """Calls long enough for four tokens per warp, across sequences' ends, empty sequences and a bad page."""
    Hkv, d, n, ctx = 16, 128, [7001, 0, 3990, 1, 1, 2, 33], [5, 0, 16, 3, 0, 7, 15]
    bt = Batch(ctx, n, Hkv, d, 64, kv, seed=3, extra_tokens=3)
    k, v = normal(bt.gen, bt.T, Hkv, d), normal(bt.gen, bt.T, Hkv, d)
    pa.cache_append(k.cuda(), v.cuda(), bt.cache, dev(bt.table), dev(bt.cu), dev(ctx))
    assert pa.status() == 0
    table = bt.table.copy()
    table[2, 30] = -5
    out = [torch.full((bt.T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.cache_read(bt.cache, dev(table), dev(bt.cu), dev(ctx), bt.T, k=out[0], v=out[1])
    assert pa.status() == ERR_INDEX
    seq = np.repeat(np.arange(len(n)), n)
    pos = np.concatenate([c + np.arange(m) for c, m in zip(ctx, n)])
    kept = np.append(~((seq == 2) & (pos // 64 == 30)), np.zeros(bt.T - len(seq), dtype=bool))
    for x, got in zip((k, v), out):
        x, got = x.float().numpy(), got.float().cpu().numpy()
        want = x[kept] if kv == "bf16" else ref.decode(*ref.encode(x[kept], kv), kv)
        assert np.array_equal(got[kept], want) and (got[~kept] == 7.0).all()


# ------------------------------------------------------------------ attention

EXTEND = [
    # name, kv, H, Hkv, d, page, ctx, n, k_local, period, S, mode
    ("one-token", "bf16", 4, 2, 64, 16, [0], [1], 8, 16, 2, PI),
    ("one-after-many", "bf16", 16, 4, 128, 64, [777], [1], 256, 128, 4, PI),
    ("draft", "bf16", 16, 4, 128, 32, [30, 64, 500, 31], [5, 3, 6, 2], 100, 150, 3, PI),
    ("aligned-chunk", "bf16", 8, 2, 128, 64, [256], [256], 128, 128, 3, PI),
    ("odd-all", "bf16", 4, 1, 64, 16, [37, 0, 5], [133, 71, 1], 45, 67, 3, PI),
    ("mha", "bf16", 3, 3, 64, 32, [129, 3], [200, 140], 64, 96, 2, PI),
    ("gqa2", "bf16", 4, 2, 128, 128, [70], [161], 33, 50, 4, PI),
    ("gqa3", "bf16", 6, 2, 64, 64, [11, 90], [64, 40], 50, 64, 2, PI),
    ("gqa7", "bf16", 7, 1, 128, 16, [40], [130], 31, 37, 5, PI),
    ("empty-sequences", "bf16", 4, 2, 64, 16, [0, 10, 0, 99], [0, 20, 0, 64], 20, 32, 2, PI),
    ("no-skips", "bf16", 4, 4, 64, 256, [300], [100], 70, 1, 0, PI),
    ("band-of-one", "bf16", 4, 2, 128, 32, [50], [90], 0, 7, 6, PI),
    ("skips-in-band", "bf16", 4, 2, 64, 32, [100], [70], 40, 16, 6, PI),
    ("many-skips", "bf16", 4, 2, 64, 64, [900], [40], 5, 9, 90, PI),
    ("band-over-everything", "bf16", 8, 2, 128, 64, [200], [150], 100000, 64, 2, PI),
    ("period-over-everything", "bf16", 4, 2, 64, 16, [60], [60], 10, 100000, 4, PI),
    ("ecp", "bf16", 4, 4, 64, 32, [100, 0], [150, 65], 64, 0, 0, ECP),
    ("ecp-odd", "bf16", 4, 2, 128, 16, [61], [77], 27, 0, 0, ECP),
    ("e4m3", "e4m3", 8, 2, 128, 64, [333, 5], [130, 31], 128, 96, 3, PI),
    ("e4m3-d64-page16", "e4m3", 6, 2, 64, 16, [90, 17], [40, 70], 50, 70, 3, PI),
    ("int8", "int8", 8, 2, 128, 32, [200, 64], [64, 100], 100, 128, 2, PI),
    ("int8-ecp-d64", "int8", 4, 4, 64, 128, [300], [200], 96, 0, 0, ECP),
    ("int8-one-token", "int8", 16, 1, 128, 16, [400, 3], [1, 1], 64, 100, 3, PI),
    ("long", "e4m3", 16, 4, 128, 64, [2500], [700], 256, 1024, 4, PI),
    ("ragged-batch", "bf16", 16, 4, 128, 64, [0, 1500, 31, 640, 77], [300, 1, 33, 128, 5], 256, 512, 2, PI),
]


# The same call has two kernels, for chunks of few tokens and for long ones; the cases above are small enough for the
# first, these long enough for the second, with padding where they have to be.
EXTEND_LONG = [
    ("aligned", "bf16", 8, 2, 128, 64, [256], [512], 128, 128, 3, PI),
    ("one-block-and-one-token", "bf16", 16, 4, 128, 64, [0, 7], [320, 1], 100, 96, 2, PI),
    ("odd-all", "bf16", 16, 4, 64, 16, [37, 0, 5], [233, 171, 1], 45, 67, 3, PI),
    ("mha", "bf16", 6, 6, 64, 32, [129, 3], [400, 340], 64, 96, 2, PI),
    ("gqa2", "bf16", 8, 4, 128, 128, [70, 900], [361, 63], 33, 50, 4, PI),
    ("gqa3", "bf16", 12, 4, 64, 64, [11, 90, 31], [264, 140, 2], 50, 64, 2, PI),
    ("gqa7", "bf16", 14, 2, 128, 16, [40, 8], [230, 130], 31, 37, 5, PI),
    ("gqa16", "bf16", 32, 2, 64, 16, [100], [200], 64, 100, 3, PI),
    ("gqa20", "bf16", 20, 1, 64, 32, [5, 3], [40, 9], 20, 30, 3, PI),
    ("empty-sequences", "bf16", 16, 4, 64, 16, [0, 10, 0, 99, 3], [0, 220, 0, 164, 0], 20, 32, 2, PI),
    ("no-skips", "bf16", 8, 8, 64, 256, [300], [500], 70, 1, 0, PI),
    ("band-of-one", "bf16", 8, 4, 128, 32, [50], [390], 0, 7, 6, PI),
    ("skips-in-band", "bf16", 8, 4, 64, 32, [100], [370], 40, 16, 6, PI),
    ("many-skips", "bf16", 20, 1, 64, 64, [900], [340], 5, 9, 90, PI),
    ("band-over-everything", "bf16", 16, 4, 128, 64, [200], [350], 100000, 64, 2, PI),
    ("period-over-everything", "bf16", 8, 4, 64, 16, [60], [360], 10, 100000, 4, PI),
    ("ecp", "bf16", 8, 8, 64, 32, [100, 0], [250, 265], 64, 0, 0, ECP),
    ("ecp-odd", "bf16", 8, 4, 128, 16, [61], [377], 27, 0, 0, ECP),
    ("ecp-long", "bf16", 8, 4, 64, 64, [1000], [400], 700, 0, 0, ECP),
    ("e4m3", "e4m3", 16, 4, 128, 64, [333, 5], [430, 31], 128, 96, 3, PI),
    ("e4m3-d64-page16", "e4m3", 12, 4, 64, 16, [90, 17], [240, 170], 50, 70, 3, PI),
    ("e4m3-far-skips", "e4m3", 16, 4, 64, 16, [3000, 100], [130, 40], 40, 900, 3, PI),
    ("int8", "int8", 16, 4, 128, 32, [200, 64], [264, 100], 100, 128, 2, PI),
    ("int8-ecp-d64", "int8", 8, 8, 64, 128, [300], [500], 96, 0, 0, ECP),
    ("int8-empty", "int8", 16, 4, 128, 256, [0, 500, 3], [0, 300, 1], 64, 50, 3, PI),
    ("long", "e4m3", 16, 4, 128, 64, [2500], [700], 256, 1024, 4, PI),
    ("long-bf16", "bf16", 16, 4, 128, 64, [2500], [700], 256, 1024, 4, PI),
]


def few_rows(case, extra=0):
    """Whether a case, with so many tokens of no sequence behind the last, takes the kernel of few tokens, which alone needs no
    workspace."""
    _, kv, H, Hkv, d, page, ctx, n, kl, per, S, mode = case
    width = max(max(-(-(c + m) // page) for c, m in zip(ctx, n)), 1) + 1
    return pa.extend_workspace_size(pa.PagedCache.empty(1, Hkv, page, d, ref.DTYPE[kv]), len(n), int(sum(n)) + extra, width, H, kl, per, S, mode) == 0


def padding(case, extra=2):
    """Tokens of no sequence that make a case a long one: the choice goes by the tokens of the call."""
    while few_rows(case, extra):
        extra *= 2
        assert extra < 10 ** 5
    return extra


def run_attention(case, decode=False, seed=0, extra=2):
    name, kv, H, Hkv, d, page, ctx, n, kl, per, S, mode = case
    bt = Batch(ctx, n, Hkv, d, page, kv, seed=seed + len(name) + d, extra_tokens=0 if decode else extra)
    keep = [ref.attended_pages(c, c + m - 1, page, kl, per, S, mode == ECP) if m else set() for c, m in zip(ctx, n)]
    bt.write(keep=keep)
    for b, pages in enumerate(keep):  # pages that no query attends are gone from the table
        for p in range(bt.table.shape[1]):
            if p not in pages:
                bt.table[b, p] = -1 if p % 2 else 2 ** 30
    q = normal(bt.gen, bt.T, H, d)
    alpha = None if mode == ECP else torch.sigmoid(1.5 * torch.randn(bt.T, H, generator=bt.gen))
    if alpha is not None:
        alpha[0, 0], alpha[-1, -1] = 1.0, 0.0
    wide = torch.full((bt.T, H + 3, d), float("nan"), dtype=torch.bfloat16)
    wide[:, :H] = q
    qd, ad = wide.cuda()[:, :H], None if alpha is None else alpha.cuda()
    out = torch.full((bt.T, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((bt.T, H), 9.0, device="cuda")
    if decode:
        call = lambda: pa.decode_paged(qd, bt.cache, dev(bt.table), dev(np.array(ctx) + 1), ad, kl, per, S, mode,  # noqa: E731
                                       out=out, lse=lse)
    else:
        call = lambda: pa.extend(qd, bt.cache, dev(bt.table), dev(bt.cu), dev(ctx), ad, kl, per, S, mode,  # noqa: E731
                                 out=out, lse=lse)
    call()
    torch.cuda.synchronize()
    assert pa.status() == 0
    K, V = bt.held()
    for b, (c, m) in enumerate(zip(ctx, n)):
        if m:
            t = slice(bt.cu[b], bt.cu[b + 1])
            want = ref.attention(q[t], K[b], V[b], None if alpha is None else alpha[t], c, kl, per, S, mode)
            ref.check_attention(f"{name} sequence {b}", out[t], lse[t], want)
    assert (out[bt.cu[-1]:] == 9.0).all() and (lse[bt.cu[-1]:] == 9.0).all()
    first = out.clone(), lse.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse), "not the same twice"


@pytest.mark.parametrize("case", EXTEND, ids=[c[0] for c in EXTEND])
def test_extend_matches_the_oracle(case):
    run_attention(case)


@pytest.mark.parametrize("case", EXTEND_LONG, ids=[c[0] for c in EXTEND_LONG])
def test_extend_of_long_chunks_matches_the_oracle(case):
    run_attention(case, extra=padding(case))


DECODE = [
    ("first-token", "bf16", 4, 2, 64, 16, [0, 0], [1, 1], 8, 4, 2, PI),
    ("short", "bf16", 4, 4, 64, 32, [19, 3, 15], [1] * 3, 40, 16, 2, PI),
    ("ragged", "bf16", 16, 4, 128, 64, [999, 4, 63, 64, 300], [1] * 5, 256, 150, 3, PI),
    ("gqa16", "bf16", 16, 1, 128, 16, [700, 31], [1, 1], 64, 90, 5, PI),
    ("gqa8", "bf16", 8, 1, 64, 128, [500], [1], 64, 100, 4, PI),
    ("gqa9", "e4m3", 9, 1, 64, 64, [321, 7], [1, 1], 50, 60, 4, PI),
    ("gqa3", "int8", 6, 2, 128, 256, [400, 255], [1, 1], 90, 100, 3, PI),
    ("mha-e4m3", "e4m3", 12, 12, 64, 16, [127, 128, 129], [1] * 3, 128, 64, 1, PI),
    ("e4m3", "e4m3", 16, 4, 128, 64, [1200, 90, 0], [1] * 3, 256, 300, 4, PI),
    ("int8", "int8", 16, 4, 128, 32, [600, 2], [1, 1], 77, 128, 4, PI),
    ("band-of-one", "bf16", 4, 2, 128, 16, [50], [1], 0, 7, 6, PI),
    ("no-skips", "int8", 4, 2, 64, 16, [333], [1], 70, 1, 0, PI),
    ("many-skips", "bf16", 4, 2, 64, 64, [1500], [1], 5, 9, 160, PI),
    ("long-band", "bf16", 8, 2, 128, 64, [2500], [1], 2400, 64, 2, PI),
    ("ecp", "bf16", 4, 2, 64, 32, [776, 127, 128], [1] * 3, 128, 0, 0, ECP),
    ("ecp-e4m3-d128", "e4m3", 4, 4, 128, 64, [512, 1], [1, 1], 256, 0, 0, ECP),
    ("big-batch", "bf16", 4, 2, 64, 16, list(range(0, 300, 4)), [1] * 75, 64, 96, 2, PI),
]


@pytest.mark.parametrize("case", DECODE, ids=[c[0] for c in DECODE])
def test_decode_matches_the_oracle(case):
    run_attention(case, decode=True)


def test_decode_without_rows():
    """A sequence of length zero among others: out 0 and lse -inf, as for a row without a finite logit."""
    bt = Batch([40, 7], [1, 1], 2, 64, 16, "bf16", seed=3)
    bt.write()
    q, a = normal(bt.gen, 2, 4, 64).cuda(), torch.full((2, 4), 0.5, device="cuda")
    out, lse = pa.decode_paged(q, bt.cache, dev(bt.table), dev([41, 0]), a, 16, 8, 2)
    torch.cuda.synchronize()
    assert pa.status() == 0
    assert torch.isfinite(out[0].float()).all() and torch.isfinite(lse[0]).all()
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


MASKED = [
    # kv, H, Hkv, d, page, ctx, n, k_local, period, S, mode
    ("bf16", 16, 4, 128, 64, [300, 64], [320, 40], 100, 96, 2, PI),
    ("bf16", 12, 4, 64, 16, [90], [640], 50, 70, 3, PI),
    ("e4m3", 16, 4, 128, 64, [300, 64], [420, 40], 100, 128, 2, PI),
    ("int8", 8, 8, 64, 128, [300], [500], 96, 0, 0, ECP),
    ("bf16", 16, 4, 128, 32, [130, 164, 500], [5, 3, 6], 100, 150, 3, PI),
    ("e4m3", 12, 4, 64, 16, [90], [30], 20, 25, 3, PI),
    ("int8", 4, 2, 128, 64, [300], [40], 96, 0, 0, ECP),
]


@pytest.mark.parametrize("case", MASKED, ids=[f"{c[0]}-d{c[3]}-{sum(c[6])}" for c in MASKED])
def test_a_row_is_made_of_its_own_keys(case):
    """Values that are not finite, inside the chunk, in its band and under its skips, and one such key: exactly the rows
    that attend them have them in their results, in their columns (8 bits: blocks); every other is the oracle's."""
    kv, H, Hkv, d, page, ctx, n, kl, per, S, mode = case
    extra = padding(("",) + case) if sum(n) > 300 else 0
    assert few_rows(("",) + case, extra) == (sum(n) < 300)
    bt = Batch(ctx, n, Hkv, d, page, kv, seed=d + sum(n), extra_tokens=extra)
    odd = [float("nan"), float("inf"), float("-inf")]
    planted = []  # sequence, position, KV head, first column, columns
    for b, (c, m) in enumerate(zip(ctx, n)):
        far = [c + m // 3 - per] if S and c + m // 3 >= per else []
        for x, pos in enumerate([c - 3, c, c + m // 2, c + m - 1] + far):
            g, col = x % Hkv, (37 * x + 5) % d
            bt.v[b][pos, g, col] = odd[x % 3]
            planted.append((b, pos, g, col, 1) if kv == "bf16" else (b, pos, g, col // 32 * 32, 32))
    key_at = ctx[0] + 2 * n[0] // 3
    bt.k[0][key_at, Hkv - 1, 7] = odd[0]
    bt.write()
    q = normal(bt.gen, bt.T, H, d)
    alpha = None if mode == ECP else torch.sigmoid(torch.randn(bt.T, H, generator=bt.gen))
    out, lse = pa.extend(q.cuda(), bt.cache, dev(bt.table), dev(bt.cu), dev(ctx), None if alpha is None else alpha.cuda(), kl, per, S, mode)
    torch.cuda.synchronize()
    assert pa.status() == 0
    K, V = ([torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in xs] for xs in bt.held())
    bad, bad_lse = np.zeros((bt.T, H, d), dtype=bool), np.zeros((bt.T, H), dtype=bool)
    G = H // Hkv
    for b, (c, m) in enumerate(zip(ctx, n)):
        for i in range(c, c + m):
            t = bt.cu[b] + i - c
            keys = set(range(max(0, (i // kl - 1) * kl if mode == ECP else i - kl), i + 1))
            keys |= {i - x * per for x in range(1, S + 1) if x * per > kl and i >= x * per}
            for pb, pos, g, col, w in planted:
                if pb == b and pos in keys:
                    bad[t, g * G:(g + 1) * G, col:col + w] = True
            if b == 0 and key_at in keys:
                bad[t, H - G:] = bad_lse[t, H - G:] = True
    assert bad.any() and not bad.all()
    got, got_lse = out.float().cpu(), lse.cpu()
    assert not torch.isfinite(got[torch.from_numpy(bad)]).any(), "a row without a value that it attends"
    assert torch.isnan(got_lse[torch.from_numpy(bad_lse)]).all()
    for b, (c, m) in enumerate(zip(ctx, n)):
        t = slice(bt.cu[b], bt.cu[b + 1])
        ro, rl, size = ref.attention(q[t], K[b], V[b], None if alpha is None else alpha[t], c, kl, per, S, mode)
        o = np.where(bad[t], ro, got[t].numpy().astype(np.float64))
        z = np.where(bad_lse[t], rl, got_lse[t].numpy().astype(np.float64))
        off = np.abs(o - ro)
        assert np.isfinite(o).all(), f"sequence {b}: {int((~np.isfinite(o)).sum())} outputs have another row's value"
        # rounding as in check_attention; what stands in for a bad result is the oracle's own
        assert (off <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -12) * size + 1e-30).all()
        assert (np.abs(z - rl) <= 2.0 ** -12 + 2.0 ** -22 * np.abs(rl)).all()


@pytest.mark.parametrize("n,H,shape,strides", [(5, 4, (5, 4, 64), (576, 64, 1)), (1, 4, (1, 4, 64), (1, 64, 1)), (4, 1, (4, 1, 64), (64, 1000, 1)),
                                               (1, 1, (1, 1, 64), (8, 7, 1)), (300, 4, (300, 4, 64), (264, 64, 1))])
def test_new_outputs_are_contiguous(n, H, shape, strides):
    """Whatever the strides between the queries' tokens (and of dimensions of size one)."""
    bt = Batch([40], [n], 1, 64, 16, "bf16", seed=n)
    bt.write()
    q = torch.empty_strided(shape, strides, dtype=torch.bfloat16, device="cuda").copy_(normal(bt.gen, *shape))
    a = torch.full((n, H), 0.5, device="cuda")
    call = lambda x: pa.extend(x, bt.cache, dev(bt.table), dev(bt.cu), dev([40]), a, 20, 16, 2)  # noqa: E731
    out, lse = call(q)
    want, want_lse = call(q.clone(memory_format=torch.contiguous_format))
    assert out.is_contiguous() and lse.is_contiguous() and torch.equal(out, want) and torch.equal(lse, want_lse)
    if n == 1:
        out, lse = pa.decode_paged(q, bt.cache, dev(bt.table), dev([41]), a, 20, 16, 2)
        assert out.is_contiguous() and lse.is_contiguous() and out.shape == q.shape


# ------------------------------------------------------------------ indexes out of range

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bad_indexes_of_long_chunks(kv):
    """The same for the kernels of long chunks: a bad sequence is left out, a bad page reported, decreasing offsets end
    the call's work."""
    n, H, Hkv = 250, 16, 4
    bt = Batch([20] * 3, [n] * 3, Hkv, 64, 16, kv, seed=6)
    bt.write()
    q, a = normal(bt.gen, bt.T, H, 64).cuda(), torch.full((bt.T, H), 0.5, device="cuda")
    args = (a, 16, 8, 2)
    good, good_lse = pa.extend(q, bt.cache, dev(bt.table), dev(bt.cu), dev(bt.ctx), *args)
    torch.cuda.synchronize()
    assert pa.status() == 0
    ok = [0, n, 2 * n, 3 * n]
    for cu, ctx, kept in ((ok[:3] + [3 * n + 1], [20] * 3, 2 * n), (ok[:3] + [2 ** 31 - 1], [20] * 3, 2 * n),
                          (ok, [20, 20, -1], 2 * n), (ok, [20, 20, 2 ** 31 - 1], 2 * n),
                          (ok, [20, 20, 16 * bt.table.shape[1] - n + 1], 2 * n), ([0, n, n - 1, 3 * n], [20] * 3, 0)):
        out, lse = torch.full_like(good, 9.0), torch.full_like(good_lse, 9.0)
        pa.extend(q, bt.cache, dev(bt.table), dev(cu), dev(ctx), *args, out=out, lse=lse)
        assert pa.status() == ERR_INDEX and pa.status() == 0
        assert torch.equal(out[:kept], good[:kept]) and torch.equal(lse[:kept], good_lse[:kept])
        assert (out[kept:] == 9.0).all() and (lse[kept:] == 9.0).all()
    for bad in (2 ** 31 - 1, -1):
        table = bt.table.copy()
        table[2, 3] = bad
        out, lse = pa.extend(q, bt.cache, dev(table), dev(ok), dev(bt.ctx), *args)
        assert pa.status() == ERR_INDEX and pa.status() == 0
        assert torch.equal(out[:2 * n], good[:2 * n]) and torch.equal(lse[:2 * n], good_lse[:2 * n])


def test_bad_indexes_are_reported_and_left_out():
    """Offsets, contexts, lengths and pages out of range: reported once by status(), the rest of the batch
    served, nothing written for the sequences concerned."""
    bt = Batch([20, 20, 20], [10, 10, 10], 2, 64, 16, "bf16", seed=5)
    bt.write()
    q, a = normal(bt.gen, 30, 4, 64).cuda(), torch.full((30, 4), 0.5, device="cuda")
    args = (a, 16, 8, 2)
    pa.extend(q, bt.cache, dev(bt.table), dev([0, 10, 9, 30]), dev(bt.ctx), *args)  # decreasing offsets
    assert pa.status() == ERR_INDEX and pa.status() == 0
    good, good_lse = pa.extend(q, bt.cache, dev(bt.table), dev(bt.cu), dev(bt.ctx), *args)
    rows = torch.zeros(30, 2, 64, dtype=torch.bfloat16, device="cuda")
    ok = [0, 10, 20, 30]
    for cu, ctx in (([0, 10, 20, 31], [20] * 3), ([0, 10, 20, 2 ** 31 - 1], [20] * 3), (ok, [20, 20, -1]),
                    (ok, [20, 20, 2 ** 31 - 1]), (ok, [20, 20, 16 * bt.table.shape[1] - 9])):
        out, lse = torch.full_like(good, 9.0), torch.full_like(good_lse, 9.0)
        pa.extend(q, bt.cache, dev(bt.table), dev(cu), dev(ctx), *args, out=out, lse=lse)
        assert pa.status() == ERR_INDEX and pa.status() == 0
        assert torch.equal(out[:20], good[:20]) and torch.equal(lse[:20], good_lse[:20])
        assert (out[20:] == 9.0).all() and (lse[20:] == 9.0).all()
    before = [x.clone() for x in (bt.cache.k, bt.cache.v)]
    table = bt.table.copy()
    table[2] = 2 ** 31 - 1
    pa.cache_append(rows[20:], rows[20:], bt.cache, dev(table[2:]), dev([0, 10]), dev([20]))
    assert pa.status() == ERR_INDEX
    assert torch.equal(before[0].view(torch.int16), bt.cache.k.view(torch.int16))
    assert torch.equal(before[1].view(torch.int16), bt.cache.v.view(torch.int16))
    k, _ = pa.cache_read(bt.cache, dev(table), dev(ok), dev([20, 20, 20]), 30, k=torch.full_like(rows, 9.0))
    assert pa.status() == ERR_INDEX
    assert (k[20:] == 9.0).all() and torch.equal(k[:10].cpu(), bt.k[0][20:30])
    pa.extend(q, bt.cache, dev(table), dev(ok), dev(bt.ctx), *args)
    assert pa.status() == ERR_INDEX
    d3, a3 = q[:3].contiguous(), a[:3].contiguous()
    want = pa.decode_paged(d3, bt.cache, dev(bt.table), dev([30, 30, 0]), a3, 16, 8, 2)
    for lens in ([30, 30, -1], [30, 30, 16 * bt.table.shape[1] + 1], [30, 30, 2 ** 31 - 1]):
        got = pa.decode_paged(d3, bt.cache, dev(bt.table), dev(lens), a3, 16, 8, 2)
        assert pa.status() == ERR_INDEX and pa.status() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    pa.decode_paged(d3, bt.cache, dev(table), dev([30, 30, 30]), a3, 16, 8, 2)
    assert pa.status() == ERR_INDEX and pa.status() == 0


# ------------------------------------------------------------------ as they are used together

@pytest.mark.parametrize("kv,H,Hkv,d,page,kl,per,S,mode", [
    ("bf16", 8, 2, 128, 32, 64, 96, 3, PI), ("e4m3", 8, 2, 128, 64, 64, 100, 3, PI),
    ("int8", 4, 4, 64, 16, 48, 0, 0, ECP)])
def test_serving_run(kv, H, Hkv, d, page, kl, per, S, mode):
    """Prompts written and attended chunk by chunk, then tokens one by one, in one batch: every output row is
    the whole sequence's forward's on the values the cache holds."""
    gen = torch.Generator().manual_seed(7)
    chunks = [[130, 40], [77, 0], [1, 64], [1, 1], [1, 1], [1, 1]]  # new rows of the two sequences per step
    total = np.sum(chunks, 0)
    rng = np.random.default_rng(1)
    table, pages = ref.make_table([0, 0], list(total), page, rng)
    cache = nan_cache(pages, Hkv, page, d, kv)
    seqs = [dict(q=normal(gen, m, H, d), k=normal(gen, m, Hkv, d), v=normal(gen, m, Hkv, d),
                 a=None if mode == ECP else torch.sigmoid(torch.randn(m, H, generator=gen)), out=[], lse=[]) for m in total]
    at = [0, 0]
    for n in chunks:
        part = lambda name: torch.cat([s[name][p:p + m] for s, p, m in zip(seqs, at, n)]).cuda()  # noqa: E731
        cu, ctx = ref.offsets(n), list(at)
        pa.cache_append(part("k"), part("v"), cache, dev(table), dev(cu), dev(ctx))
        a = None if mode == ECP else part("a")
        if n == [1, 1]:
            out, lse = pa.decode_paged(part("q"), cache, dev(table), dev(np.add(ctx, 1)), a, kl, per, S, mode)
        else:
            out, lse = pa.extend(part("q"), cache, dev(table), dev(cu), dev(ctx), a, kl, per, S, mode)
        for b, s in enumerate(seqs):
            s["out"].append(out[cu[b]:cu[b + 1]].cpu())
            s["lse"].append(lse[cu[b]:cu[b + 1]].cpu())
            at[b] += n[b]
    K, V = pa.cache_read(cache, dev(table), dev(ref.offsets(total)), dev([0, 0]), int(total.sum()))
    assert pa.status() == 0
    for b, s in enumerate(seqs):
        rows = slice(*ref.offsets(total)[b:b + 2])
        held = K[rows].cpu(), V[rows].cpu()
        if kv == "bf16":
            assert torch.equal(held[0], s["k"]) and torch.equal(held[1], s["v"])
        want = ref.attention(s["q"], *held, s["a"], 0, kl, per, S, mode)
        ref.check_attention(f"sequence {b}", torch.cat(s["out"]), torch.cat(s["lse"]), want)


@pytest.mark.parametrize("T,sizes", [(50, ([30, 20], [0, 45], [7, 1])), (2000, ([500, 300], [0, 777], [700, 3]))])
def test_captured_step_follows_its_inputs(T, sizes):
    """Append, extend and decode captured into one graph on a stream of their own and replayed with other offsets,
    contexts and values in the same tensors, an empty sequence and padding tokens among them."""
    H, Hkv, d, page, kl, per, S = 8, 2, 64, 16, 40, 50, 2
    bt = Batch([100, 60], [T, T], Hkv, d, page, "e4m3", seed=11)  # pages for every step's rows
    bt.write()
    k, v, q = (normal(bt.gen, T, h, d).cuda() for h in (Hkv, Hkv, H))
    a = torch.rand(T, H, generator=bt.gen).cuda()
    table, cu, ctx, lens = dev(bt.table), dev(ref.offsets(sizes[0])), dev([100, 60]), dev([130, 80])
    out, lse = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")
    dout, dlse = torch.zeros(2, H, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, H, device="cuda")

    def step():
        pa.cache_append(k, v, bt.cache, table, cu, ctx)
        pa.extend(q, bt.cache, table, cu, ctx, a, kl, per, S, out=out, lse=lse)
        pa.decode_paged(q[:2], bt.cache, table, lens, a[:2], kl, per, S, out=dout, lse=dlse)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for n, c in zip(sizes, ([100, 60], [100, 10], [64, 79])):
        for t in (k, v, q):
            t.copy_(normal(bt.gen, *t.shape))
        cu.copy_(dev(ref.offsets(n)))
        ctx.copy_(dev(c))
        lens.copy_(dev(np.minimum(np.add(c, n), 130)))
        results = []
        for run in (step, graph.replay):
            for t in (out, lse, dout, dlse):
                t.fill_(5.0)
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            results.append([t.clone() for t in (out, lse, dout, dlse)] + [bt.cache.k.clone().view(torch.uint8)])
        assert all(torch.equal(x, y) for x, y in zip(*results))
        assert (results[0][0][sum(n):] == 5.0).all()
    assert pa.status() == 0


@pytest.mark.parametrize("n", [[364, 240], [3, 5]])
def test_streams_run_side_by_side(n):
    """Calls on two streams at once, each with inputs of its own, new outputs and (long chunks) a workspace made in the call:
    what each alone gives."""
    bt = Batch([300, 200], n, 2, 128, 64, "e4m3", seed=13)
    bt.write()
    sets = [(normal(bt.gen, bt.T, 8, 128).cuda(), torch.rand(bt.T, 8, generator=bt.gen).cuda()) for _ in range(2)]
    table, cu, ctx, lens = dev(bt.table), dev(bt.cu), dev(bt.ctx), dev(np.add(bt.ctx, n))
    calls = [lambda q, a, **kw: pa.extend(q, bt.cache, table, cu, ctx, a, 100, 64, 3, **kw),
             lambda q, a, **kw: pa.decode_paged(q[:2], bt.cache, table, lens, a[:2], 100, 64, 3, **kw)]
    want = [[call(*x) for call in calls] for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            got[i].append([call(*sets[i], stream=st) for call in calls])
    torch.cuda.synchronize()
    for i in range(2):
        for results in got[i]:
            for (o, ls), (wo, wl) in zip(results, want[i]):
                assert torch.equal(o, wo) and torch.equal(ls, wl)
    assert pa.status() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("H,Hkv,d,B", [(16, 4, 128, 3), (4, 4, 64, 40)])
def test_steps_without_a_pause(kv, H, Hkv, d, B):
    """A hundred generation steps enqueued one behind the other, and as a replayed graph of single steps, give what steps with a
    synchronisation after each call give: every call sees what the calls before it wrote (its kernel starts early)."""
    page, steps, first = 16, 100, 37
    gen = torch.Generator().manual_seed(B)
    width = (first + steps) // page + 1
    order = torch.randperm(B * width, generator=gen).int().view(B, width).cuda()
    new = normal(gen, steps, B, H + 2 * Hkv, d).cuda()
    alpha = torch.rand(steps, B, H, generator=gen).cuda()
    draft = torch.arange(B + 1, dtype=torch.int32, device="cuda")

    def run(pause=False, graph=False):
        cache = pa.PagedCache.empty(B * width, Hkv, page, d, ref.DTYPE[kv])
        lens = torch.full((B,), first, dtype=torch.int32, device="cuda")
        table = torch.full_like(order, -1)
        table[:, :first // page + 1] = order[:, :first // page + 1]
        at = torch.zeros(1, dtype=torch.int64, device="cuda")
        out = [torch.zeros(steps, B, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        x, a = torch.empty_like(new[0]), torch.empty_like(alpha[0])

        def step():
            stop = torch.cuda.synchronize if pause else lambda: None
            x.copy_(new.index_select(0, at)[0])
            a.copy_(alpha.index_select(0, at)[0])
            table.scatter_(1, (lens // page).long()[:, None], order.gather(1, (lens // page).long()[:, None]))
            stop()
            pa.cache_append(x[:, H:H + Hkv], x[:, H + Hkv:], cache, table, draft, lens)
            stop()
            o1, _ = pa.extend(x[:, :H], cache, table, draft, lens, a, 20, 16, 2)
            stop()
            lens.add_(1)
            o2, _ = pa.decode_paged(x[:, :H], cache, table, lens, a, 20, 16, 2)
            stop()
            out[0].index_copy_(0, at, o1[None])
            out[1].index_copy_(0, at, o2[None])
            at.add_(1)

        if graph:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                step()  # a first step outside the capture
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            for _ in range(steps - 1):
                g.replay()
        else:
            for _ in range(steps):
                step()
        torch.cuda.synchronize()
        assert pa.status() == 0
        return out + [cache.k.view(torch.uint8), cache.v.view(torch.uint8)]

    want = run(pause=True)
    for got in (run(), run(graph=True)):
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_threads_call_side_by_side():
    """Four host threads, each with a cache, a stream and outputs of its own, make the same calls at once that one makes alone."""
    from concurrent.futures import ThreadPoolExecutor

    def work(x, stream):
        bt, q, a = x
        with torch.cuda.stream(stream):
            got = []
            for _ in range(20):
                pa.cache_append(bt.k[0][:64].cuda(), bt.v[0][:64].cuda(), bt.cache, dev(bt.table), dev([0, 64]), dev([0]))
                got.append(pa.extend(q, bt.cache, dev(bt.table), dev(bt.cu), dev(bt.ctx), a, 64, 32, 3))
                got.append(pa.decode_paged(q[-1:], bt.cache, dev(bt.table), dev([bt.ctx[0] + bt.n[0]]), a[-1:], 64, 32, 3))
                got.append(pa.cache_read(bt.cache, dev(bt.table), dev([0, 100]), dev([0]), 100))
        stream.synchronize()
        return got

    jobs = []
    for x in range(4):
        bt = Batch([100], [3 if x % 2 else 700], 4, 64, 32, ["bf16", "e4m3", "int8"][x % 3], seed=x)
        bt.write()
        jobs.append((bt, normal(bt.gen, bt.T, 16, 64).cuda(), torch.rand(bt.T, 16, generator=bt.gen).cuda()))
    torch.cuda.synchronize()
    want = [work(x, torch.cuda.current_stream()) for x in jobs]
    with ThreadPoolExecutor(4) as pool:
        got = list(pool.map(work, jobs, [torch.cuda.Stream() for _ in jobs]))
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for u, v in zip(w, g) for x, y in zip(u, v))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_sequences(kv):
    """More sequences than the plan takes in one round, empty ones among them, through the long chunks' kernels; and through
    the short ones'."""
    rng, B, H, Hkv, d = np.random.default_rng(8), 600, 16, 4, 64
    for n in (rng.integers(0, 30, B), rng.integers(0, 3, B)):
        n[100:140] = 0
        ctx = rng.integers(0, 50, B)
        case = ("", kv, H, Hkv, d, 16, list(ctx), list(n), 20, 32, 2, PI)
        assert few_rows(case, 2) == (n.max() < 3)
        bt = Batch(list(ctx), list(n), Hkv, d, 16, kv, seed=9, extra_tokens=2)
        whole = np.add(ctx, n)
        k, v = (torch.cat([x for x in xs if len(x)]).cuda() for xs in (bt.k, bt.v))
        pa.cache_append(k, v, bt.cache, dev(bt.table), dev(ref.offsets(whole)), dev(np.zeros(B)))
        q, a = normal(bt.gen, bt.T, H, d), torch.rand(bt.T, H, generator=bt.gen)
        out, lse = pa.extend(q.cuda(), bt.cache, dev(bt.table), dev(bt.cu), dev(ctx), a.cuda(), 20, 32, 2)
        assert pa.status() == 0
        K, V = bt.held()
        for b in np.concatenate([np.flatnonzero(n)[::9], np.flatnonzero(n)[-3:]]):
            t = slice(bt.cu[b], bt.cu[b + 1])
            ref.check_attention(f"sequence {b}", out[t], lse[t], ref.attention(q[t], K[b], V[b], a[t], ctx[b], 20, 32, 2, PI))


def test_offsets_past_32_bits():
    """Rows whose byte and element offsets in the pool pass 2^32: the last pages of a large 8-bit pool."""
    page, Hkv, d = 256, 8, 128
    pages = (1 << 32) // (page * Hkv * d) + 40  # codes alone pass 4 GiB, K and V each
    cache = pa.PagedCache.empty(pages, Hkv, page, d, torch.int8)
    gen = torch.Generator().manual_seed(2)
    n, H = 500, 16
    k, v, q = (normal(gen, n, h, d) for h in (Hkv, Hkv, H))
    a = torch.rand(n, H, generator=gen)
    table, cu, ctx = dev([[pages - 1, pages - 3]]), dev([0, n]), dev([0])
    pa.cache_append(k.cuda(), v.cuda(), cache, table, cu, ctx)
    out, lse = pa.extend(q.cuda(), cache, table, cu, ctx, a.cuda(), 64, 100, 2)
    o1, l1 = pa.decode_paged(q[-1:].cuda(), cache, table, dev([n]), a[-1:].cuda(), 64, 100, 2)
    K, V = pa.cache_read(cache, table, cu, ctx, n)
    assert pa.status() == 0
    held = [torch.from_numpy(ref.decode(*ref.encode(x.float().numpy(), "int8"), "int8")).to(torch.bfloat16) for x in (k, v)]
    assert torch.equal(K.cpu(), held[0]) and torch.equal(V.cpu(), held[1])
    want = ref.attention(q, *held, a, 0, 64, 100, 2, PI)
    ref.check_attention("extend", out, lse, want)
    ref.check_attention("decode", o1, l1, [x[-1:] for x in want])


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attention_with_scales_of_any_size(kv, where):
    """Keys (against queries that make up for it) and values 2^-100 to 2^100 times their usual size: the kernels'
    conversions hold over the whole range of the scales."""
    Hkv, H, d, page, N, n = 2, 8, 128, 16, 150, 40
    gen = torch.Generator().manual_seed(4)
    table, cu, ctx = dev(np.arange(10)[None]), dev([0, n]), dev([N - n])
    for power in (-100, -20, 10, 60, 100):
        size = 2.0 ** power
        k, v, q = (normal(gen, m, h, d) for m, h in ((N, Hkv), (N, Hkv), (n, H)))
        if where == "k":
            k, q = k * size, q / size
        else:
            v = v * size
        cache = pa.PagedCache.empty(10, Hkv, page, d, ref.DTYPE[kv])
        pa.cache_append(k.cuda(), v.cuda(), cache, table, dev([0, N]), dev([0]))
        a = torch.rand(n, H, generator=gen)
        out, lse = pa.extend(q.cuda(), cache, table, cu, ctx, a.cuda(), 64, 50, 2)
        o1, l1 = pa.decode_paged(q[-1:].cuda(), cache, table, dev([N]), a[-1:].cuda(), 64, 50, 2)
        torch.cuda.synchronize()
        held = [torch.from_numpy(ref.decode(*ref.encode(x.float().numpy(), kv), kv)).to(torch.bfloat16) for x in (k, v)]
        want = ref.attention(q, *held, a, N - n, 64, 50, 2, PI)
        ref.check_attention(f"extend 2^{power}", out, lse, want)
        ref.check_attention(f"decode 2^{power}", o1, l1, [x[-1:] for x in want])
