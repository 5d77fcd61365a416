"""GPU parity of rotary positions and of a speculative serving step: rotation, append, tree attention, verification, kept paths."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import step_ref as sref
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


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rope(rot, inter, kind="none", **kw):
    more = dict(linear=dict(factor=4.0), ntk=dict(factor=8.0), yarn=dict(factor=16.0, original=4096), none={})[kind]
    return pa.Rotary(rot, 10000.0, interleaved=inter, scaling=kind, **more, **kw)


# ------------------------------------------------------------------ rotary

ROTARY = [
    # B, H, Hkv, N, d, rot, interleaved, scaling, type, start or None (given positions)
    (2, 4, 2, 37, 64, 64, False, "none", torch.bfloat16, 0),
    (1, 3, 1, 130, 128, 128, True, "yarn", torch.bfloat16, 1000003),
    (3, 5, 5, 1, 128, 64, False, "linear", torch.float32, None),
    (1, 1, 0, 300, 32, 16, True, "none", torch.float32, 5),
    (2, 9, 3, 33, 128, 48, False, "ntk", torch.bfloat16, None),
    (1, 2, 2, 65, 32, 32, False, "none", torch.bfloat16, None),
    (1, 6, 2, 41, 64, 16, False, "yarn", torch.float32, 2 ** 21 - 41),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: f"d{c[4]}-r{c[5]}-{c[7]}-n{c[3]}")
def test_rotary(case, back):
    B, H, Hkv, N, d, rot, inter, kind, dt, start = case
    gen = torch.Generator().manual_seed(N + d)
    r = rope(rot, inter, kind)
    pos = None if start is not None else torch.randint(-(2 ** 20), 2 ** 20, (B, N), generator=gen, dtype=torch.int32)
    x = torch.randn(B, N, H + 2 * max(Hkv, 1), d, generator=gen).to(dt)  # a projection's output
    xd = x.cuda().transpose(1, 2)
    call = pa.rotary_bwd if back else pa.rotary
    q, k = call(xd[:, :H], xd[:, H:H + Hkv] if Hkv else None, r, start or 0, None if pos is None else pos.cuda())
    torch.cuda.synchronize()
    at = np.arange(N)[None] + start if pos is None else pos.numpy()
    at = np.broadcast_to(at, (B, N))[:, None]
    for name, y, lo, hi in (("q", q, 0, H), ("k", k, H, H + Hkv)):
        if hi == lo:
            assert y is None
            continue
        assert y.is_contiguous() and y.dtype == dt
        want, size = sref.rotate(f64(x[:, :, lo:hi].transpose(1, 2)), at, r, -1 if back else 1)
        sref.check_rotated(name, f64(y), want, size, torch.finfo(dt).eps)
        assert torch.equal(y[..., rot:].cpu(), x[:, :, lo:hi, rot:].transpose(1, 2))


def test_rotary_into_a_projection_and_in_place():
    """Outputs with strides of their own, and an output that is its input: the same bits as a new one."""
    B, N, H, Hkv, d = 2, 70, 6, 3, 64
    r = rope(32, False, "ntk")
    dq, dk = (torch.randn(B, h, N, d, device="cuda").bfloat16() for h in (H, Hkv))
    want = pa.rotary_bwd(dq, dk, r, 7)
    g = torch.full((B, N, H + 2 * Hkv, d), 3.0, device="cuda", dtype=torch.bfloat16)
    v = g.transpose(1, 2)
    got = pa.rotary_bwd(dq, dk, r, 7, None, v[:, :H], v[:, H:H + Hkv])
    assert got[0].data_ptr() == g.data_ptr()
    assert torch.equal(v[:, :H], want[0]) and torch.equal(v[:, H:H + Hkv], want[1]) and (v[:, H + Hkv:] == 3).all()
    x = torch.randn(B, N, H + 2 * Hkv, d, device="cuda").bfloat16()
    w = x.transpose(1, 2)
    want = pa.rotary(w[:, :H], w[:, H:H + Hkv], r, 7)
    rest = w[:, H + Hkv:].clone()
    pa.rotary(w[:, :H], w[:, H:H + Hkv], r, 7, None, w[:, :H], w[:, H:H + Hkv])
    assert torch.equal(w[:, :H], want[0]) and torch.equal(w[:, H:H + Hkv], want[1]) and torch.equal(w[:, H + Hkv:], rest)


def test_rotary_gradient_is_the_transpose():
    """<rotary(x), g> = <x, rotary_bwd(g)>, and differences of a linear function of x."""
    r = rope(64, True, "yarn")
    gen = torch.Generator().manual_seed(3)
    x, g = (torch.randn(1, 2, 50, 64, generator=gen, dtype=torch.float32).cuda() for _ in range(2))
    y, _ = pa.rotary(x, None, r, 100)
    dx, _ = pa.rotary_bwd(g, None, r, 100)
    a, b = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    size = (y.double().abs() * g.double().abs()).sum() + (x.double().abs() * dx.double().abs()).sum()
    assert abs(a - b) <= 2 * sref.SLACK * size
    for i in (0, 1, 17, 63):  # the loss sum y g along one element: an exact difference, the function being linear
        e = torch.zeros_like(x)
        e[0, 1, 13, i] = 1.0
        ye, _ = pa.rotary(e, None, r, 100)
        d = (ye.double() * g.double()).sum()
        assert abs(d - dx[0, 1, 13, i].double()) <= 4 * sref.SLACK * g[0, 1, 13].abs().sum()


def test_rotary_with_values_that_are_not_finite():
    """An infinity or NaN stays in its pair; elements past rot keep their bits."""
    r = rope(32, False)
    x = torch.randn(1, 1, 4, 64, device="cuda").bfloat16()
    x[0, 0, 1, 5], x[0, 0, 2, 40], x[0, 0, 3, 16] = float("inf"), float("nan"), float("nan")
    y, _ = pa.rotary(x, None, r, 3)
    bad = ~torch.isfinite(y[0, 0])
    want = torch.zeros(4, 64, dtype=torch.bool)
    want[1, 5] = want[1, 21] = want[2, 40] = want[3, 0] = want[3, 16] = True
    assert torch.equal(bad.cpu(), want)


# ------------------------------------------------------------------ append

APPEND = [
    # type, d, H, Hkv, page, rot, interleaved, ctx, n, trees, tokens of no sequence
    ("bf16", 128, 8, 2, 32, 128, False, [0, 31, 7, 90], [5, 0, 1, 40], False, 3),
    ("e4m3", 128, 4, 4, 64, 64, True, [100000, 63], [20, 17], True, 0),
    ("int8", 64, 3, 3, 16, 64, False, [5], [70], True, 1),
    ("e4m3", 64, 7, 1, 16, 48, False, [15, 0, 16, 2, 9], [0, 17, 0, 47, 1], False, 0),
    ("int8", 128, 16, 12, 256, 32, True, [250, 1], [7, 300], False, 2),
    ("int8", 128, 2, 1, 128, 128, False, [9], [256], True, 0),
    ("bf16", 64, 1, 1, 16, 16, False, [3] * 40, [1] * 40, True, 0),
    ("e4m3", 128, 16, 4, 64, 96, False, [77, 4000], [2600, 11], False, 5),  # several tokens per CTA
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0]}-d{c[1]}-h{c[3]}-r{c[5]}-T{sum(c[8])}")
def test_rotary_append(case):
    kv, d, H, Hkv, page, rot, inter, ctx, n, trees, extra = case
    rng, gen = np.random.default_rng(d + rot), torch.Generator().manual_seed(d + rot)
    table, pages = ref.make_table(ctx, n, page, rng)
    cu, T = ref.offsets(n), sum(n) + extra
    r = rope(rot, inter, "yarn")
    cache = pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv])
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(7)
    before = [None if t is None else ref.bits(t).copy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=gen).to(torch.bfloat16)
    x = qkv.cuda()
    parents = [sref.random_tree(m, rng, roots=1 + (m > 9)) for m in n]
    parent = dev(sum(parents, []) + [99] * extra) if trees else None
    out = torch.full((T, H, d), 5.0, device="cuda", dtype=torch.bfloat16)
    got = pa.rotary_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], r, cache, dev(table), dev(cu), dev(ctx), parent, out)
    torch.cuda.synchronize()
    assert got is out and (out[sum(n):] == 5).all()
    pos = np.concatenate([c + np.array(sref.depths(p) if trees else range(m), dtype=np.int64) for c, m, p in zip(ctx, n, parents)])
    m = sum(n)
    want, size = sref.rotate(f64(qkv[:m, :H]), pos[:, None], r)
    sref.check_rotated("q", f64(out[:m]), want, size, 2.0 ** -7)
    want, size = sref.rotate(f64(qkv[:m, H:H + Hkv]), pos[:, None], r)
    at = [(table[b, (ctx[b] + j) // page], slice(None), (ctx[b] + j) % page) for b in range(len(n)) for j in range(n[b])]
    rows = lambda t: np.stack([ref.bits(t)[i] for i in at])  # noqa: E731
    if kv == "bf16":
        sref.check_rotated("k", f64(torch.from_numpy(rows(cache.k)).view(torch.bfloat16)), want, size, 2.0 ** -7)
    else:
        sref.check_quantised("k", rows(cache.k), rows(cache.k_scale), want, size, kv)
    v = qkv[:m, H + Hkv:]
    codes, sc = (ref.bits(v), None) if kv == "bf16" else ref.encode(f64(v), kv)
    assert np.array_equal(rows(cache.v), codes)
    assert sc is None or np.array_equal(rows(cache.v_scale), sc)
    for t, old in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):  # and nothing else
        if t is not None:
            now = ref.bits(t).copy()
            for i in at:
                now[i] = old[i]
            assert np.array_equal(now, old)


def test_rotary_append_in_place_and_values_that_are_not_finite():
    d, H, Hkv = 64, 4, 2
    r, table = rope(64, False), dev([[0, 1, 2]])
    x = torch.randn(20, H + 2 * Hkv, d, device="cuda").bfloat16()
    x[3, H, 40] = float("nan")
    x[4, H + Hkv + 1, 2] = float("inf")
    for kv in ("bf16", "int8", "e4m3"):
        c1, c2 = (pa.PagedCache.empty(3, Hkv, 16, d, ref.DTYPE[kv]) for _ in range(2))
        y = x.clone()
        want = pa.rotary_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], r, c1, table, dev([0, 20]), dev([10]))
        got = pa.rotary_append(y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:], r, c2, table, dev([0, 20]), dev([10]), q_out=y[:, :H])
        assert got.data_ptr() == y.data_ptr() and torch.equal(got, want)
        k, v = pa.cache_read(c2, table, dev([0, 20]), dev([10]), 20)
        bad_k, bad_v = ~torch.isfinite(k).cpu(), ~torch.isfinite(v).cpu()
        want_k, want_v = torch.zeros_like(bad_k), torch.zeros_like(bad_v)
        if kv == "bf16":
            want_k[3, 0, 40] = want_k[3, 0, 8] = want_v[4, 1, 2] = True
        else:  # their blocks of 32
            want_k[3, 0], want_v[4, 1, :32] = True, True
        assert torch.equal(bad_k, want_k) and torch.equal(bad_v, want_v)


# ------------------------------------------------------------------ tree attention

MANY, NODES = 60, 256  # further trees, of 256 nodes: enough for the tensor-core kernel, whatever the other sizes


def tree_case(kv, d, H, Hkv, page, ctx, n, seed, deep=6, roots=1, extra=0, ecp=False):
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    table, pages = ref.make_table(ctx, n, page, rng)
    parents = [sref.random_tree(m, rng, deep, roots) if b < 80 and (m < NODES or b < 2) else [(j - 1) // 3 if j else -1 for j in range(m)]
               for b, m in enumerate(n)]
    T = sum(n) + extra
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=gen).to(torch.bfloat16)
    cache = pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv])
    for t in (cache.k, cache.v):  # rows that nobody writes read as NaN
        t.view(torch.uint8).fill_(0x7F if kv != "bf16" else 0xFF)
    for t in (cache.k_scale, cache.v_scale):
        if t is not None:
            t.fill_(255)
    old = [torch.randn(2, max(c, 1), Hkv, d, generator=gen).to(torch.bfloat16) for c in ctx]
    for b, c in enumerate(ctx):
        if c:
            pa.cache_append(old[b][0].cuda(), old[b][1].cuda(), cache, dev(table[b:b + 1]), dev([0, c]), dev([0]))
    x = qkv.cuda()
    cu = ref.offsets(n)
    pa.cache_append(x[:, H:H + Hkv], x[:, H + Hkv:], cache, dev(table), dev(cu), dev(ctx))
    alpha = None if ecp else torch.rand(T, H, generator=gen) * 0.8 + 0.1
    held = [[t.cpu() for t in pa.cache_read(cache, dev(table[b:b + 1]), dev([0, c + m]), dev([0]), c + m)] for b, (c, m) in enumerate(zip(ctx, n))]
    return cache, table, cu, parents, x[:, :H], alpha, held


TREES = [
    # type, d, H, Hkv, page, ctx, n, k_local, period, S, ecp, deepest, roots
    ("bf16", 128, 4, 1, 32, [50], [13], 20, 16, 3, False, 6, 1),
    ("e4m3", 128, 8, 2, 64, [300, 0, 17], [26, 5, 1], 64, 100, 2, False, 6, 1),
    ("int8", 64, 3, 3, 16, [40, 1], [64, 33], 8, 3, 5, False, 20, 1),       # skips and band ends inside the tree
    ("bf16", 64, 12, 12, 128, [200], [70], 100, 0, 0, False, 5, 3),         # several roots
    ("e4m3", 64, 16, 1, 16, [33, 90], [9, 17], 12, 7, 4, False, 9, 1),      # 16 heads on one
    ("int8", 128, 7, 1, 256, [0], [40], 300, 512, 2, False, 40, 1),         # no context
    ("bf16", 128, 2, 2, 16, [70, 31], [30, 256], 10, 0, 0, True, 24, 1),    # ECP: half-segments end inside the tree
    ("int8", 64, 4, 2, 64, [129], [40], 32, 0, 0, True, 7, 2),
    ("bf16", 64, 1, 1, 16, [5] * 70, [3] * 70, 4, 2, 3, False, 3, 1),       # many sequences
    ("bf16", 128, 16, 4, 64, [500, 3], [1, 1], 64, 128, 3, False, 1, 1),    # single nodes
    ("bf16", 128, 16, 4, 64, [900, 700, 801, 64], [64, 50, 33, 64], 128, 256, 3, False, 8, 1),
    ("int8", 64, 20, 1, 16, [100, 7], [30, 5], 40, 30, 2, False, 6, 1),     # 20 heads on one
    ("e4m3", 128, 24, 1, 32, [61], [12], 33, 9, 3, False, 12, 1),
]




@pytest.mark.parametrize("more", [0, MANY])
@pytest.mark.parametrize("case", TREES, ids=lambda c: f"{c[0]}-d{c[1]}-h{c[2]}on{c[3]}-p{c[4]}-T{sum(c[6])}{'-ecp' if c[10] else ''}")
def test_extend_tree(case, more):
    kv, d, H, Hkv, page, ctx, n, kl, per, S, ecp, deep, roots = case
    checked, ctx, n = len(n), ctx + [0] * more, n + [NODES] * more
    cache, table, cu, parents, q, alpha, held = tree_case(kv, d, H, Hkv, page, ctx, n, seed=d + sum(n), deep=deep, roots=roots, extra=2, ecp=ecp)
    T, m = q.shape[0], sum(n)
    out = torch.full((T, H, d), 5.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((T, H), 5.0, device="cuda")
    args = (dev(table), dev(cu), dev(ctx), dev(sum(parents, []) + [-7, 5]), None if ecp else alpha.cuda(), kl, per, S, ECP if ecp else PI)
    got = pa.extend_tree(q, cache, *args, out=out, lse=lse)
    torch.cuda.synchronize()
    assert got[0] is out and (out[m:] == 5).all() and (lse[m:] == 5).all()
    for b in range(checked):
        if not n[b]:
            continue
        rows = slice(cu[b], cu[b + 1])
        want = sref.tree_attention(q[rows].cpu(), *held[b], None if ecp else alpha[rows], ctx[b], parents[b], kl, per, S, ECP if ecp else PI)
        ref.check_attention(f"sequence {b}", out[rows], lse[rows], want)
    again = pa.extend_tree(q, cache, *args)
    assert torch.equal(again[0][:m], out[:m]) and torch.equal(again[1][:m], lse[:m])


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
def test_a_chain_is_what_extend_attends(kv):
    """A tree without branches: the same rows as extend's."""
    n, ctx, H, Hkv = [9, 40], [100, 3], 8, 2
    cache, table, cu, _, q, alpha, held = tree_case(kv, 128, H, Hkv, 32, ctx, n, seed=5)
    parent = dev([j - 1 for m in n for j in range(m)])
    out, lse = pa.extend_tree(q, cache, dev(table), dev(cu), dev(ctx), parent, alpha.cuda(), 16, 20, 3)
    for b in range(2):
        rows = slice(cu[b], cu[b + 1])
        want = ref.attention(q[rows].cpu(), *held[b], alpha[rows], ctx[b], 16, 20, 3, PI)
        ref.check_attention(f"sequence {b}", out[rows], lse[rows], want)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("more", [0, MANY])
@pytest.mark.parametrize("n", [12, 100])
def test_rows_that_a_node_does_not_attend_do_not_matter(kv, n, more):
    """NaN in the rows of some nodes reaches their descendants only; alpha = 0 on a node without skips gives 0 and -inf."""
    H, Hkv, d, ctx = 4, 2, 64, 30
    cache, table, cu, parents, q, alpha, held = tree_case(kv, d, H, Hkv, 16, [ctx] + [0] * more, [n] + [NODES] * more, seed=n)
    alpha[3:n:7] = 0.0
    k, v = (t[ctx:].clone() for t in held[0])
    spoilt = [5, n - 1]
    for j in spoilt:
        v[j] = float("nan")
    pa.cache_append(k.cuda(), v.cuda(), cache, dev(table[:1]), dev([0, n]), dev([ctx]))
    out, lse = pa.extend_tree(q, cache, dev(table), dev(cu), dev([ctx] + [0] * more), dev(sum(parents, [])), alpha.cuda(), 300, 400, 2)
    torch.cuda.synchronize()
    out, lse, alpha = out[:n], lse[:n], alpha[:n]
    clean = np.array([not set(sref.line(parents[0], j)) & set(spoilt) for j in range(n)])
    assert clean.sum() not in (0, n)
    kh, vh = (torch.cat([h[:ctx], t]) for h, t in zip(held[0], (held[0][0][ctx:], torch.nan_to_num(v, nan=0.0))))
    want = sref.tree_attention(q[:n].cpu(), kh, vh, alpha, ctx, parents[0], 300, 400, 2, PI)
    dark = (alpha == 0).any(1).numpy()
    ref.check_attention("clean", out[clean], lse[clean], [w[clean] for w in want])
    assert torch.isnan(out[torch.from_numpy(~clean & ~dark)].float()).all()
    assert (out[torch.from_numpy(dark)] == 0).all() and torch.isneginf(lse[torch.from_numpy(dark)]).all()


@pytest.mark.parametrize("more", [0, MANY])
def test_pages_that_no_node_attends_may_be_gone(more):
    """Entries below every band, between the skips' keys and before the deepest nodes' bands name no page: nothing is recorded."""
    ctx, n, kl, per, S, page = 400, 70, 40, 100, 3, 16
    cache, table, cu, parents, q, alpha, held = tree_case("bf16", 64, 8, 2, page, [ctx] + [0] * more, [n] + [NODES] * more, seed=2)
    keep = set()
    for j, deep in enumerate(sref.depths(parents[0])):
        i = ctx + deep
        keep |= {p // page for p in list(range(max(0, i - kl), ctx)) + [i - m * per for m in range(1, S + 1) if i >= m * per]}
    gone = table.copy()
    for p in range(ctx // page):
        if p not in keep:
            gone[0, p] = -1
    assert (gone[0] != table[0]).sum() >= 10
    args = (dev(cu), dev([ctx] + [0] * more), dev(sum(parents, [])), alpha.cuda(), kl, per, S)
    want = pa.extend_tree(q, cache, dev(table), *args)
    got = pa.extend_tree(q, cache, dev(gone), *args)
    assert pa.status() == 0
    assert torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1][:n], want[1][:n])
    ref.check_attention("tree", got[0][:n], got[1][:n], sref.tree_attention(q[:n].cpu(), *held[0], alpha[:n], ctx, parents[0], kl, per, S, PI))


# ------------------------------------------------------------------ verification

def probabilities(T, V, gen, spread=2.0):
    return torch.softmax(spread * torch.randn(T, V, generator=gen), -1)


VERIFY = [
    # nodes per sequence, V, draft given, how far the draft is from the target
    ([1], 7, True, 1.0), ([6], 1000, True, 1.0), ([5, 0, 17, 1], 333, True, 3.0), ([40, 9, 33], 50021, True, 1.0),
    ([64] * 9, 2050, False, 1.0), ([12], 130001, True, 2.0), ([256, 3], 4097, True, 1.0), ([31, 7], 129, False, 0.5),
    ([20] * 40, 33, True, 2.0), ([20] * 40, 33, False, 2.0), ([9] * 5, 1, True, 0.0), ([4, 5], 8193, False, 1.0), ([8] * 300, 517, True, 1.5),
]


def verify_case(n, V, drawn, noise, seed, spread=2.0):
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    parents = [sref.random_tree(m, rng, deep=5) for m in n]
    T, cu = max(sum(n), 1), ref.offsets(n)
    x = spread * torch.randn(T, V, generator=gen)
    draft, target = torch.softmax(x, -1), torch.softmax(x + noise * torch.randn(T, V, generator=gen), -1)
    tokens = np.zeros(T, dtype=np.int32)
    for b, par in enumerate(parents):
        for j, p in enumerate(par):
            if p < 0:
                tokens[cu[b] + j] = -5  # not read
            elif drawn:
                tokens[cu[b] + j] = int(torch.multinomial(draft[cu[b] + p], 1, generator=gen))
            else:  # the likeliest ones, now and then the same one twice
                rank = sum(y == p for y in par[:j])
                tokens[cu[b] + j] = int(draft[cu[b] + p].topk(min(V, rank // 2 + 1)).indices[-1])
    u, u_next = torch.rand(T, generator=gen), torch.rand(len(n), generator=gen)
    return parents, cu, target, draft if drawn else None, tokens, u, u_next


def run_verify(parents, cu, target, draft, tokens, u, u_next, **kw):
    d = [None if t is None else t.cuda() for t in (target, draft)]
    flat = sum(parents, [])
    got = pa.verify_tree(*d, dev(tokens), dev(cu), dev(flat + [-1] * (len(tokens) - len(flat))), u.cuda(), u_next.cuda(), **kw)
    torch.cuda.synchronize()
    return [t.cpu().tolist() for t in got]


def check_verify(parents, cu, target, draft, tokens, u, u_next, got):
    path, count, nxt = got
    for b, par in enumerate(parents):
        rows = slice(cu[b], cu[b + 1])
        if not par:
            assert count[b] == 0 and nxt[b] == -1
            continue
        want, token = sref.verify(target[rows].numpy(), None if draft is None else draft[rows].numpy(), tokens[rows], par, u[rows], u_next[b])
        assert path[rows] == want + [-1] * (len(par) - len(want)), (b, path[rows], want)
        assert count[b] == len(want) and nxt[b] == token, (b, nxt[b], token)


@pytest.mark.parametrize("case", VERIFY, ids=lambda c: f"B{len(c[0])}-n{max(c[0])}-V{c[1]}{'' if c[2] else '-chosen'}")
def test_verify_tree(case):
    for seed in range(3):
        s = verify_case(*case, seed=seed)
        check_verify(*s, run_verify(*s))


@pytest.mark.parametrize("case", [([4, 9, 1], 150001, True, 1.0), ([9, 4], 150001, False, 1.0), ([2] * 160, 40001, True, 1.5)],
                         ids=["cluster", "cluster-chosen", "one"])
def test_verify_tree_whose_search_takes_a_warp_several_rounds(case):
    """More than 256 tokens of the vocabulary to a warp in the last step of the search, over a cluster of CTAs and over one."""
    s = list(verify_case(*case, seed=4, spread=0.5))
    for u_next in (None, torch.zeros(len(case[0])), torch.full((len(case[0]),), 1 - 2.0 ** -24)):
        if u_next is not None:
            s[6] = u_next
        check_verify(*s, run_verify(*s))


def test_verified_tokens_are_distributed_as_the_target():
    """A token drawn from q and its random numbers on a grid: the first new token's frequencies are p."""
    p, q, g = torch.tensor([0.1, 0.5, 0.0, 0.3, 0.1]), torch.tensor([0.4, 0.1, 0.2, 0.2, 0.1]), 50
    grid = (torch.arange(g) + 0.5) / g
    for draft in (True, False):
        first = np.zeros(5)
        for v in range(5):
            n = g * g
            parents, cu = [[-1, 0]] * n, ref.offsets([2] * n)
            u, u_next = torch.zeros(2 * n), grid.repeat(g)
            u[1::2] = grid.repeat_interleave(g)
            tokens = np.tile([0, v], n).astype(np.int32)
            rows = p.repeat(2 * n, 1)
            path, count, nxt = run_verify(parents, cu, rows, q.repeat(2 * n, 1) if draft else None, tokens, u, u_next)
            for b in range(n):
                first[v if count[b] == 2 else nxt[b]] += float(q[v]) / n
        assert np.abs(first - p.numpy()).max() <= 2.0 / g  # a grid's step for each of the two numbers


def test_verify_at_the_edges():
    """Probabilities that are zero, outside [0, 1] or not finite; random numbers at the ends; no weight left; strided rows."""
    V = 40
    gen = torch.Generator().manual_seed(1)
    big = probabilities(6, V + 3, gen)
    target = big[:, :V]
    assert target.stride(0) == V + 3
    target = torch.where(torch.rand(6, V, generator=gen) < 0.3, torch.zeros(()), target)
    target[2, 4], target[2, 5], target[2, 6] = float("nan"), float("inf"), -1.0
    target[5] = 0.0
    draft = probabilities(6, V, gen)
    draft[0] = target[0]      # a child is accepted whatever its number; nothing is left of p after
    draft[2, 7] = float("nan")
    parents, cu = [[-1, 0, 0], [-1], [-1], [-1]], np.array([0, 3, 4, 5, 6], dtype=np.int32)
    for end in (0.0, 1.0 - 2.0 ** -24):
        tokens = np.array([0, int(target[0].argmax()), 1, 0, 0, 0], dtype=np.int32)
        u, u_next = torch.full((6,), end), torch.full((4,), end)
        for d in (draft, None):
            s = (parents, cu, target, d, tokens, u, u_next)
            check_verify(*s, run_verify(*s))
    wide = big.cuda()
    s = (parents, cu, target, None, tokens, u, u_next)
    wide[:, :V] = target.cuda()
    got = pa.verify_tree(wide[:, :V], None, dev(tokens), dev(cu), dev(sum(parents, [])), u.cuda(), u_next.cuda())
    check_verify(*s, [t.cpu().tolist() for t in got])
    # numbers outside [0, 1): the nearest inside
    for x, y in ((float("nan"), 0.0), (-3.0, 0.0), (7.0, 1.0 - 2.0 ** -24), (float("inf"), 1.0 - 2.0 ** -24)):
        a = run_verify(parents, cu, target, draft, tokens, torch.full((6,), x), torch.full((4,), x))
        b = run_verify(parents, cu, target, draft, tokens, torch.full((6,), y), torch.full((4,), y))
        assert a == b


# ------------------------------------------------------------------ kept paths

KEEP = [
    # type, d, Hkv, page, ctx, n, layers
    ("bf16", 128, 4, 32, [30, 0, 5], [20, 1, 7], 3), ("int8", 64, 3, 16, [15, 100], [40, 9], 2), ("e4m3", 128, 2, 64, [63], [70], 1),
    ("bf16", 64, 12, 16, [7] * 30, [12] * 30, 1), ("int8", 128, 1, 256, [250], [300], 66), ("e4m3", 64, 16, 128, [1, 2], [0, 33], 5),
]


@pytest.mark.parametrize("case", KEEP, ids=lambda c: f"{c[0]}-d{c[1]}-h{c[2]}-p{c[3]}-L{c[6]}")
def test_cache_keep(case):
    kv, d, Hkv, page, ctx, n, layers = case
    rng = np.random.default_rng(page + d)
    table, pages = ref.make_table(ctx, n, page, rng)
    caches = []
    for _ in range(layers):
        c = pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv])
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.view(torch.uint8).random_(0, 256)
        caches.append(c)
    path, count = [], []
    for m in n:
        c = int(rng.integers(0, m + 1))
        path += sorted(rng.choice(m, c, replace=False).tolist()) + [-1] * (m - c)
        count.append(c)
    cu = ref.offsets(n)
    before = [[None if t is None else ref.bits(t).copy() for t in (c.k, c.v, c.k_scale, c.v_scale)] for c in caches]
    pa.cache_keep(pa.CacheLayers(caches) if layers > 1 else caches[0], dev(table), dev(cu), dev(ctx), dev(path + [55]), dev(count))
    torch.cuda.synchronize()
    for c, old in zip(caches, before):
        for t, x in zip((c.k, c.v, c.k_scale, c.v_scale), old):
            if t is None:
                continue
            want = x.copy()
            for b in range(len(n)):
                for j in range(count[b]):
                    s, p = ctx[b] + path[cu[b] + j], ctx[b] + j
                    want[table[b, p // page], :, p % page] = x[table[b, s // page], :, s % page]
            assert np.array_equal(ref.bits(t), want)


# ------------------------------------------------------------------ a step, and what is left out

@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
def test_a_step_leaves_the_cache_as_if_the_path_had_been_appended(kv):
    """Trees through append, attention, verification and keeping, twice, eagerly and as a replayed graph on another stream; then the
    caches of all layers hold the accepted tokens' rows, bit for bit."""
    B, H, Hkv, d, page, V, layers = 3, 4, 2, 64, 16, 300, 2
    n, ctx0 = [9, 5, 14], [20, 3, 31]
    rng, gen = np.random.default_rng(8), torch.Generator().manual_seed(8)
    table, pages = ref.make_table(ctx0, [60] * B, page, rng)
    parents = [sref.random_tree(m, rng) for m in n]
    cu, T = ref.offsets(n), sum(n)
    r = rope(64, False, "yarn")
    tab, cud, par = dev(table), dev(cu), dev(sum(parents, []))
    alpha = torch.full((T, H), 0.5, device="cuda")

    class Run:
        def __init__(self):
            self.caches = [pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv]) for _ in range(layers)]
            self.all = pa.CacheLayers(self.caches)
            self.ctx = dev(ctx0).clone()
            self.x = torch.zeros(layers, T, H + 2 * Hkv, d, device="cuda", dtype=torch.bfloat16)
            self.target, self.draft = torch.zeros(T, V, device="cuda"), torch.zeros(T, V, device="cuda")
            self.tokens = torch.zeros(T, device="cuda", dtype=torch.int32)
            self.u, self.u_next = torch.zeros(T, device="cuda"), torch.zeros(B, device="cuda")

        def step(self):
            outs = []
            for c, x in zip(self.caches, self.x):
                q = pa.rotary_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], r, c, tab, cud, self.ctx, par)
                outs.append(pa.extend_tree(q, c, tab, cud, self.ctx, par, alpha, 24, 30, 2)[0])
            self.outs = outs
            self.path, self.count, self.next = pa.verify_tree(self.target, self.draft, self.tokens, cud, par, self.u, self.u_next)
            pa.cache_keep(self.all, tab, cud, self.ctx, self.path, self.count)
            self.ctx.add_(self.count)

    eager, graphed = Run(), Run()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graphed.step()  # warm-up on zeros
        side.synchronize()
        graphed.ctx.copy_(dev(ctx0))
        for c in graphed.caches:
            for t in (c.k, c.v, c.k_scale, c.v_scale):
                if t is not None:
                    t.view(torch.uint8).zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            graphed.step()
        graphed.ctx.copy_(dev(ctx0))
    side.synchronize()
    plain = [pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv]) for _ in range(layers)]
    ctx = list(ctx0)
    for _ in range(2):
        s = verify_case(n, V, True, 0.3, seed=int(rng.integers(1 << 30)))
        target, draft = s[2], s[3]
        tokens = np.array([int(torch.multinomial(draft[cu[b] + max(p, 0)], 1, generator=gen)) for b in range(B) for p in parents[b]], dtype=np.int32)
        x = torch.randn(layers, T, H + 2 * Hkv, d, generator=gen).to(torch.bfloat16)
        for run in (eager, graphed):
            for at, value in ((run.x, x), (run.target, target), (run.draft, draft), (run.tokens, torch.from_numpy(tokens)), (run.u, s[5]),
                              (run.u_next, s[6])):
                at.copy_(value)
        eager.step()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        assert torch.equal(eager.path, graphed.path) and torch.equal(eager.next, graphed.next)
        for a, b in zip(eager.outs, graphed.outs):
            assert torch.equal(a, b)
        path, count = eager.path.tolist(), eager.count.tolist()
        for b in range(B):
            keep = path[cu[b]:cu[b] + count[b]]
            for c, rows in zip(plain, x):
                y = rows[cu[b]:][keep].cuda()
                pa.rotary_append(y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:], r, c, tab[b:b + 1], dev([0, len(keep)]), dev([ctx[b]]))
            ctx[b] += count[b]
        assert eager.ctx.tolist() == ctx
    assert sum(ctx) > sum(ctx0) + 2 * B  # some children were accepted
    for a, b, c in zip(eager.caches, graphed.caches, plain):
        for i in range(B):
            m = ctx[i] - ctx0[i]
            k = [pa.cache_read(z, tab[i:i + 1], dev([0, m]), dev([ctx0[i]]), m) for z in (a, b, c)]
            assert torch.equal(k[0][0], k[2][0]) and torch.equal(k[0][1], k[2][1]) and torch.equal(k[1][0], k[2][0])


def test_what_is_out_of_range_is_left_out():
    """A bad offset, parent, token, path or page: status says so, the sequence's outputs and rows stay, the others are right."""
    kv, d, H, Hkv, page, ctx, n = "bf16", 64, 4, 2, 16, [20, 33], [8, 9]
    cache, table, cu, parents, q, alpha, held = tree_case(kv, d, H, Hkv, page, ctx, n, seed=4)
    r, flat = rope(64, False), sum(parents, [])
    T = sum(n)

    def attend(table=table, cu=cu, ctx=ctx, parent=flat):
        out, lse = torch.full((T, H, d), 5.0, device="cuda", dtype=torch.bfloat16), torch.full((T, H), 5.0, device="cuda")
        pa.extend_tree(q, cache, dev(table), dev(cu), dev(ctx), dev(parent), alpha.cuda(), 300, 10, 2, out=out, lse=lse)
        return out

    def append(table=table, cu=cu, ctx=ctx, parent=flat):
        out, c = torch.full((T, H, d), 5.0, device="cuda", dtype=torch.bfloat16), pa.PagedCache.empty(cache.k.shape[0], Hkv, page, d)
        x = torch.ones(T, Hkv, d, device="cuda", dtype=torch.bfloat16)
        pa.rotary_append(q, x, x, r, c, dev(table), dev(cu), dev(ctx), dev(parent), out)
        assert int((c.v != 0).sum()) == int((out[:, 0, 0] != 5).sum()) * Hkv * d
        return out

    good = {f: f() for f in (attend, append)}
    assert pa.status() == 0
    bad_parent = [flat[:8] + [-1, 0, 1, 3] + flat[12:], flat[:8] + [-2] + flat[9:], flat[:16] + [2 ** 31 - 1]]
    for f in (attend, append):
        for kw in [dict(parent=p) for p in bad_parent] + [dict(ctx=[20, 2 ** 31 - 1]), dict(ctx=[20, -1]), dict(cu=[0, 8, 200])]:
            out = f(**kw)
            assert pa.status() == ERR_INDEX
            assert torch.equal(out[:8], good[f][:8]) and (out[8:] == 5).all()
    t = table.copy()
    t[1, 33 // page] = 10 ** 6
    out = append(table=t)  # positions 33 .. 41 lie on one page
    assert pa.status() == ERR_INDEX and torch.equal(out[:8], good[append][:8]) and (out[8:] == 5).all()
    whole = append(ctx=[20, 28])
    out = append(table=t, ctx=[20, 28])  # of positions 28 .. 36 those from 32 on
    assert pa.status() == ERR_INDEX and torch.equal(out[:12], whole[:12]) and (out[12:] == 5).all()
    # more nodes than a tree may have
    big = 257
    c2, table2, cu2, par2, q2, alpha2, _ = tree_case(kv, d, H, Hkv, page, [3], [big], seed=9)
    out = torch.full((big, H, d), 5.0, device="cuda", dtype=torch.bfloat16)
    pa.extend_tree(q2, c2, dev(table2), dev(cu2), dev([3]), dev(par2[0]), alpha2.cuda(), 30, 10, 2, out=out)
    assert pa.status() == ERR_INDEX and (out == 5).all()
    # verification
    s = verify_case([4, 5], 50, True, 1.0, seed=2)
    want = run_verify(*s)
    for what in range(3):
        parents2, cu3, tokens = [list(p) for p in s[0]], s[1].copy(), s[4].copy()
        if what == 0:
            parents2[1][3] = 3
        elif what == 1:
            tokens[6] = 50
        else:
            cu3[2] = 1000
        path = torch.full((9,), 77, device="cuda", dtype=torch.int32)
        got = run_verify(parents2, cu3, s[2], s[3], tokens, s[5], s[6], path=path)
        assert pa.status() == ERR_INDEX
        assert got[0][:4] == want[0][:4] and got[0][4:] == [77] * 5 and got[1] == [want[1][0], 0] and got[2] == [want[2][0], -1]
    # paths
    for path, count in (([0, 2, 1], 3), ([0, 1, 9], 3), ([-1, 0, 1], 2), ([0, 1, 2], 10), ([0, 1, 2], -1), ([1, 1, 2], 2)):
        before = cache.k.clone()
        pa.cache_keep(cache, dev(table), dev(cu), dev(ctx), dev([0, 1] + [-1] * 6 + path + [-1] * 6), dev([2, count]))
        assert pa.status() == ERR_INDEX and torch.equal(cache.k.view(torch.int16), before.view(torch.int16))


def test_empty_batches():
    """No tokens at all: nothing is launched, outputs have no rows."""
    cache = pa.PagedCache.empty(2, 2, 16, 64)
    e = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    r, table, cu, ctx = rope(64, False), dev([[0]]), dev([0, 0]), dev([0])
    none = torch.empty(0, device="cuda", dtype=torch.int32)
    assert pa.rotary_append(e, k, k, r, cache, table, cu, ctx).shape == (0, 4, 64)
    out, lse = pa.extend_tree(e, cache, table, cu, ctx, none, torch.empty(0, 4, device="cuda"), 8, 0, 0)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    pa.cache_keep(cache, table, cu, ctx, none, dev([0]))
    q, kk = pa.rotary(torch.empty(1, 4, 0, 64, device="cuda"), torch.empty(1, 2, 0, 64, device="cuda"), r)
    assert q.shape == (1, 4, 0, 64) and kk.shape == (1, 2, 0, 64)


@pytest.mark.parametrize("B,kv", [(400, "bf16"), (1300, "int8"), (1300, "bf16")])
def test_many_trees(B, kv):
    """Hundreds of trees, some empty, on the tensor-core kernel: their blocks are counted by every CTA, or (over 1152) searched."""
    rng = np.random.default_rng(B)
    d, H, Hkv, page = 64, 8, 2, 16
    n = [int(x) if x > 3 else 0 for x in rng.integers(0, 70, B)]
    n[-1], n[B // 2] = 33, 256
    cache, table, cu, parents, q, alpha, _ = tree_case(kv, d, H, Hkv, page, [0] * B, n, seed=B, extra=3)
    T = q.shape[0]
    out, lse = torch.full((T, H, d), 5.0, device="cuda", dtype=torch.bfloat16), torch.full((T, H), 5.0, device="cuda")
    ctx = np.zeros(B, dtype=np.int32)
    pa.extend_tree(q, cache, dev(table), dev(cu), dev(ctx), dev(sum(parents, []) + [-1] * 3), alpha.cuda(), 9, 4, 3, out=out, lse=lse)
    torch.cuda.synchronize()
    assert pa.status() == 0 and (out[-3:] == 5).all() and (lse[-3:] == 5).all() and not (lse[:-3] == 5).any()
    for b in sorted({0, B - 1, B // 2, *rng.integers(0, B, 25).tolist()}):
        if not n[b]:
            continue
        rows = slice(cu[b], cu[b + 1])
        k, v = (t.cpu() for t in pa.cache_read(cache, dev(table[b:b + 1]), dev([0, n[b]]), dev([0]), n[b]))
        want = sref.tree_attention(q[rows].cpu(), k, v, alpha[rows], 0, parents[b], 9, 4, 3, PI)
        ref.check_attention(f"sequence {b}", out[rows], lse[rows], want)


def test_offsets_that_decrease_are_reported():
    """Nothing outside the buffers is touched, and status says so, whichever kernel it is."""
    cache, table, cu, parents, q, alpha, _ = tree_case("bf16", 64, 8, 2, 16, [0] * 40, [40] * 40, seed=3)
    bad = cu.copy()
    bad[20] = 100
    par = dev(sum(parents, []))
    pa.extend_tree(q, cache, dev(table), dev(bad), dev([0] * 40), par, alpha.cuda(), 9, 4, 3)
    assert pa.status() == ERR_INDEX
    x = torch.ones(q.shape[0], 2, 64, device="cuda", dtype=torch.bfloat16)
    pa.rotary_append(q, x, x, rope(64, False), cache, dev(table), dev(bad), dev([0] * 40), par)
    assert pa.status() == ERR_INDEX
    pa.extend_tree(q[:8], cache, dev(table[:2]), dev([0, 6, 3]), dev([0, 0]), dev([-1] * 8), alpha[:8].cuda(), 9, 4, 3)
    assert pa.status() == ERR_INDEX


def test_two_streams_and_threads():
    """Calls of several threads on streams of their own, not waiting for one another: each result is the lone call's."""
    import threading
    cases = []
    for seed in range(4):
        cache, table, cu, parents, q, alpha, _ = tree_case("e4m3", 128, 8, 2, 32, [70, 33], [20, 60], seed=seed)
        s = verify_case([9, 30], 5000, True, 1.0, seed=seed)
        args = (q, cache, dev(table), dev(cu), dev([70, 33]), dev(sum(parents, [])), alpha.cuda(), 24, 30, 2)
        v = (s[2].cuda(), s[3].cuda(), dev(s[4]), dev(s[1]), dev(sum(s[0], [])), s[5].cuda(), s[6].cuda())
        cases.append((args, v, pa.extend_tree(*args), pa.verify_tree(*v)))
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        st = torch.cuda.Stream()
        for _ in range(20):
            got[i] = (pa.extend_tree(*cases[i][0], stream=st), pa.verify_tree(*cases[i][1], stream=st))
        st.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (_, _, tree, verified), (a, b) in zip(cases, got):
        assert all(torch.equal(x, y) for x, y in zip(tree + verified, a + b))


def test_a_single_node_is_a_decoded_token():
    """One node per sequence, as a step without drafts has it: rotary_append and extend_tree against decode_paged's row."""
    B, H, Hkv, d, page = 5, 8, 2, 128, 32
    ctx = [100, 31, 0, 64, 7]
    cache, table, cu, parents, q, alpha, held = tree_case("bf16", d, H, Hkv, page, ctx, [1] * B, seed=6)
    out, lse = pa.extend_tree(q, cache, dev(table), dev(cu), dev(ctx), dev([-1] * B), alpha.cuda(), 20, 24, 3)
    one, l1 = pa.decode_paged(q, cache, dev(table), dev([c + 1 for c in ctx]), alpha.cuda(), 20, 24, 3)
    for b in range(B):
        want = ref.attention(q[b:b + 1].cpu(), *held[b], alpha[b:b + 1], ctx[b], 20, 24, 3, PI)
        ref.check_attention("node", out[b:b + 1], lse[b:b + 1], want)
        ref.check_attention("token", one[b:b + 1], l1[b:b + 1], want)
