"""GPU tests of rotary positions and of the speculative step at the ends of their ranges: sums over long rows, weights that are nearly
nothing, far positions, many trees, a rotary that goes while a stream still reads it."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_ref as ref
import step_ref as sref
import structured_sparse_long_gb300 as pa
import test_gpu_step as steps
from structured_sparse_long_gb300 import build as pbuild
from structured_sparse_long_gb300 import paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    pbuild.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    pa.load()
    yield
    assert pa.status() == 0


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


# ------------------------------------------------------------------ rotary

PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def turned(x, pos, r, sign):
    """x [n, d] turned by pos [n], and the sum of a pair's magnitudes: as step_ref.rotate, but what is left of a turn is found in fractions."""
    x = x.astype(np.float64)
    y, size = x.copy(), np.zeros_like(x)
    for t, f in enumerate(r.freqs):
        a, b = (2 * t, 2 * t + 1) if r.interleaved else (t, t + r.rot // 2)
        w = np.array([sign * 2 * math.pi * float(Fraction(f) * p / (2 * PI) % 1) for p in pos])
        y[:, a] = r.scale * (x[:, a] * np.cos(w) - x[:, b] * np.sin(w))
        y[:, b] = r.scale * (x[:, a] * np.sin(w) + x[:, b] * np.cos(w))
        size[:, a] = size[:, b] = abs(r.scale) * (np.abs(x[:, a]) + np.abs(x[:, b]))
    return y, size


ENDS = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1 - 2 ** 31, 2 ** 30 + 1, -2 ** 30 - 1, 2 ** 24 + 1, -2 ** 24 - 1, 2 ** 21 + 1, 2 ** 16 - 1, -1, 0,
        1234567891, -1987654321]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_at_both_ends_of_the_positions(inter, back):
    """Given positions, and counted ones up to 2^31 - 1.  A step's rounding is 2^-65 turns per position, 2^-34 of a turn here: nothing beside
    the slack."""
    d, H, n = 64, 3, len(ENDS)
    gen = torch.Generator().manual_seed(7)
    r = pa.Rotary(d, 10000.0, interleaved=inter, scaling="linear", factor=0.7)  # the fastest pair above a radian per position
    x = torch.randn(1, H, n, d, generator=gen)
    call = pa.rotary_bwd if back else pa.rotary
    for pos, start in ((ENDS, 0), (None, 2 ** 31 - n)):
        y, _ = call(x.cuda(), None, r, start, None if pos is None else dev([pos]))
        at = pos or list(range(start, 2 ** 31))
        for h in range(H):
            want, size = turned(x[0, h].numpy(), at, r, -1 if back else 1)
            sref.check_rotated(f"head {h}", y[0, h].cpu().numpy().astype(np.float64), want, size, torch.finfo(torch.float32).eps)


def test_a_rotary_that_goes_while_another_stream_still_reads_it():
    """Its steps' memory is not handed out again before the calls enqueued with it are done."""
    x = torch.randn(1, 2, 50, 64, device="cuda")
    want, _ = pa.rotary(x, None, pa.Rotary(64), 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got, _ = pa.rotary(x, None, pa.Rotary(64), 3, stream=side)
    others = [torch.full((32,), 1 << 60, dtype=torch.int64, device="cuda") for _ in range(100)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(others) == 100


def test_a_rotary_whose_first_call_on_a_stream_is_captured():
    """The stream is recorded during the capture; replays read the steps, and the object goes after the graph without a trace."""
    x = torch.randn(1, 2, 50, 64, device="cuda")
    want, _ = pa.rotary(x, None, pa.Rotary(64), 3)
    r, side, out = pa.Rotary(64), torch.cuda.Stream(), torch.zeros_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pa.rotary(x, None, r, 3, q_out=out)
    out.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del g, r
    y, _ = pa.rotary(x, None, pa.Rotary(64), 3)
    assert torch.equal(y, want)


# ------------------------------------------------------------------ trees

def test_more_trees_than_a_launch_of_the_short_kernel_has_places():
    """70000 single nodes of eight heads on one: a CTA takes one each, and a launch has 65535."""
    B, H, d, page, ctx = 70000, 8, 64, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = pa.PagedCache.empty(B, 1, page, d)
    for t in (cache.k, cache.v):
        t[:, :, :ctx + 1] = torch.randn(B, 1, ctx + 1, d, device="cuda", generator=gen).bfloat16()
    table = torch.randperm(B, device="cuda", generator=gen, dtype=torch.int32)[:, None].contiguous()
    q = torch.randn(B, H, d, device="cuda", generator=gen).bfloat16()
    alpha = torch.rand(B, H, device="cuda", generator=gen) * 0.8 + 0.1
    cu = torch.arange(B + 1, device="cuda", dtype=torch.int32)
    args = (cache, table, cu, torch.full((B,), ctx, device="cuda", dtype=torch.int32), torch.full((B,), -1, device="cuda", dtype=torch.int32), alpha)
    out, lse = pa.extend_tree(q, *args, 2, 3, 1)  # the band's keys 1, 2 and 3, and key 0 as a skip
    k, v = (t[table[:, 0].long(), 0, :ctx + 1].double() for t in (cache.k, cache.v))
    off = torch.stack([torch.log(1 - alpha.double())] + [torch.log(alpha.double())] * 3, -1)
    z = torch.einsum("bhd,bkd->bhk", q.double(), k) / math.sqrt(d) + off
    p = torch.softmax(z, -1)
    want = (torch.einsum("bhk,bkd->bhd", p, v), torch.logsumexp(z, -1), torch.einsum("bhk,bkd->bhd", p, v.abs()))
    ref.check_attention("trees", out, lse, [w.cpu().numpy() for w in want])
    assert pa.status() == 0
    bad = cu.clone()
    bad[68001] = 5  # of the second launch's sequences one whose offsets decrease
    pa.extend_tree(q, cache, table, bad, *args[3:], 2, 3, 1)
    assert pa.status() == -8


def tree_kernel(kv, d, H, Hkv, page, n, width, kl, per, S, ecp=False, extra=0):
    """0: the short chunks' kernel, 1: the tensor cores'."""
    kind, a16 = list(ref.DTYPE).index(kv), 0x10000
    c = paged._CacheStruct(a16, a16, a16 if kind else None, a16 if kind else None, kind, 1, Hkv, page, d)
    return paged._load().pi_attn_debug_tree_kernel(ctypes.byref(c), len(n), sum(n) + extra, width, H, kl, per, S, pa.MODE_ECP if ecp else pa.MODE_PI)


def test_the_cases_of_trees_reach_the_kernel_that_they_are_about():
    """The tests of tree attention ask for the tensor cores' kernel by many further trees, and have the short one without (but for more than 16
    heads on one, which it cannot take, and a few large trees)."""
    seen = []
    for case in steps.TREES:
        kv, d, H, Hkv, page, ctx, n, kl, per, S, ecp = case[:11]
        for more in (0, steps.MANY):
            m = n + [steps.NODES] * more
            width = max(-(-(c + x) // page) for c, x in zip(ctx + [0] * more, m)) + 1
            got = tree_kernel(kv, d, H, Hkv, page, m, width, kl, per, S, ecp, 2)
            assert got == 1 if more or H // Hkv > 16 else got in (0, 1), case
            seen.append((bool(more), got, kv))
    assert {x[2] for x in seen if x[1] == 0} == {x[2] for x in seen if x[1] == 1} == set(ref.DTYPE)
    assert sum(x[:2] == (False, 0) for x in seen) >= 9
    for n in (12, 100):
        for kv in ("bf16", "int8"):
            assert tree_kernel(kv, 64, 4, 2, 16, [n], 10, 300, 400, 2) == 0
            assert tree_kernel(kv, 64, 4, 2, 16, [n] + [steps.NODES] * steps.MANY, 18, 300, 400, 2) == 1
    for B, kv in ((400, "bf16"), (1300, "int8"), (1300, "bf16")):
        assert tree_kernel(kv, 64, 8, 2, 16, [34] * B, 17, 9, 4, 3) == 1
    assert tree_kernel("bf16", 64, 8, 1, 16, [1] * 70000, 1, 2, 3, 1) == 0
    for kv in ("bf16", "e4m3"):
        assert tree_kernel(kv, 128, 16, 4, 256, [20], 8388352, 300, 4096, 3) == 0
        assert tree_kernel(kv, 128, 16, 4, 256, [256] * 4, 8388352, 300, 4096, 3) == 1


@pytest.mark.parametrize("more", [0, steps.MANY])
@pytest.mark.parametrize("kv,d,H,Hkv,ecp", [("bf16", 128, 4, 1, False), ("e4m3", 128, 8, 2, False), ("int8", 64, 3, 3, False), ("bf16", 64, 16, 1, True)])
def test_weights_of_few_keys_are_not_rounded_to_bf16(kv, d, H, Hkv, ecp, more):
    """Rows of up to nine keys, where a rounded weight does not drown in the others.  Outputs are rounded once (half a step, 2^-8), weights held to
    2^-15, and a score's d products are summed in 32 bits (2^-12 of the weights, as in paged_ref.check_attention)."""
    ctx, n, kl, per, S = [3, 20, 0], [6, 9, 12], 4 if ecp else 5, 7, 0 if ecp else 3
    cache, table, cu, parents, q, alpha, held = steps.tree_case(kv, d, H, Hkv, 16, ctx + [0] * more, n + [steps.NODES] * more, seed=d + H, ecp=ecp)
    assert tree_kernel(kv, d, H, Hkv, 16, n + [steps.NODES] * more, table.shape[1], kl, per, S, ecp) == bool(more)
    mode = pa.MODE_ECP if ecp else pa.MODE_PI
    out, lse = pa.extend_tree(q, cache, dev(table), dev(cu), dev(ctx + [0] * more), dev(sum(parents, [])), None if ecp else alpha.cuda(), kl, per, S, mode)
    for b in range(3):
        rows = slice(cu[b], cu[b + 1])
        want, _, size = sref.tree_attention(q[rows].cpu(), *held[b], None if ecp else alpha[rows], ctx[b], parents[b], kl, per, S, mode)
        off = np.abs(out[rows].float().cpu().numpy().astype(np.float64) - want)
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -15 + 2.0 ** -12) * size + 1e-30
        assert (off <= bound).all(), f"sequence {b}: off by {(off / bound).max():.2f} of its bound"


@pytest.mark.parametrize("more", [0, steps.MANY])
def test_infinite_values_reach_those_that_attend_them(more):
    """An infinity among a node's values: that element of its own row and its descendants' is the infinity (not a NaN, whichever term of a weight
    is zero), all other elements are finite and as without it: equal but for the order of sums (rows that share a tile with it are computed again), so
    off by half a step of each output, 2^-8 twice, and 2^-12 of sums of weighted values below 4."""
    H, Hkv, d, ctx, n = 8, 2, 64, 20, 30
    cache, table, cu, parents, q, alpha, held = steps.tree_case("bf16", d, H, Hkv, 16, [ctx] + [0] * more, [n] + [steps.NODES] * more, seed=3)
    args = (cache, dev(table), dev(cu), dev([ctx] + [0] * more), dev(sum(parents, [])), alpha.cuda(), 300, 400, 2)
    want, want_lse = (t[:n] for t in pa.extend_tree(q, *args))
    k, v = (t[ctx:].clone() for t in held[0])
    v[4, 0, 7], v[4, 1, 60] = float("inf"), -float("inf")
    pa.cache_append(k.cuda(), v.cuda(), cache, dev(table[:1]), dev([0, n]), dev([ctx]))
    out, lse = (t[:n] for t in pa.extend_tree(q, *args))
    below = torch.tensor([4 in sref.line(parents[0], j) for j in range(n)], device="cuda")
    assert 1 < int(below.sum()) < n
    assert (out[below, :4, 7] == float("inf")).all() and (out[below, 4:, 60] == -float("inf")).all()
    other = torch.ones_like(out, dtype=torch.bool)
    other[below, :4, 7] = other[below, 4:, 60] = False
    off = (out.float() - want.float()).abs()[other]
    assert torch.isfinite(out[other]).all() and (off <= 2.0 ** -7 * want.float().abs()[other] + 2.0 ** -10).all()
    assert torch.equal(lse, want_lse)


@pytest.mark.parametrize("trees", [1, 4])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_tree_at_the_last_positions(kv, trees):
    """The last rows that a page table reaches, 2^31 - 65536: appended and attended as the same tree is a whole number of pages earlier,
    bit for bit (the frequencies are 0)."""
    n, H, Hkv, d, page = 256 if trees > 1 else 20, 16, 4, 128, 256
    width = 0x7fff0000 // page
    ctx, kl, per, S = width * page - n, 300, 4096, 3
    near = 64 * page - n
    rng, gen = np.random.default_rng(trees), torch.Generator(device="cuda").manual_seed(trees)
    parents = sum((sref.random_tree(n, rng) for _ in range(trees)), [])
    T = trees * n
    r = pa.Rotary(d, freqs=[0.0] * (d // 2))
    x = torch.randn(T, H + 2 * Hkv, d, device="cuda", generator=gen).bfloat16()
    alpha = torch.rand(T, H, device="cuda", generator=gen) * 0.8 + 0.1
    results = []
    for c, w in ((near, 64), (ctx, width)):
        cache = pa.PagedCache.empty(64 * trees, Hkv, page, d, ref.DTYPE[kv])
        table = torch.full((trees, w), -1, device="cuda", dtype=torch.int32)
        table[:, w - 64:] = torch.arange(64 * trees, device="cuda", dtype=torch.int32).view(trees, 64)
        fill = torch.Generator(device="cuda").manual_seed(5)
        old = torch.randn(2, trees * 63 * page, Hkv, d, device="cuda", generator=fill).bfloat16()
        rows = 63 * page  # (the last page: the tree's, behind what is filled here)
        start = dev([(w - 64) * page] * trees)
        pa.cache_append(old[0], old[1], cache, table, dev(np.arange(trees + 1) * rows), start)
        cu, at, par = dev(np.arange(trees + 1) * n), dev([c] * trees), dev(parents)
        q = pa.rotary_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], r, cache, table, cu, at, par)
        assert torch.equal(q, x[:, :H])
        results.append(pa.extend_tree(q, cache, table, cu, at, par, alpha, kl, per, S))
    assert pa.status() == 0
    (a, la), (b, lb) = results
    assert torch.isfinite(a.float()).all() and torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_a_step_on_the_last_pages_of_a_large_pool(kv):
    """Pages from 2^32 elements on (8.6 GB of bf16 keys): a step there leaves what it leaves on the first pages, bit for bit."""
    H, Hkv, d, page, n, ctx = 8, 4, 128, 256, 40, 300
    pages = (1 << 25) // (Hkv * page) + 4  # 2^25 rows of 128 and four pages more
    rng, gen = np.random.default_rng(2), torch.Generator(device="cuda").manual_seed(2)
    parent = dev(sref.random_tree(n, rng))
    r = pa.Rotary(d, 10000.0)
    x = torch.randn(n, H + 2 * Hkv, d, device="cuda", generator=gen).bfloat16()
    old = torch.randn(2, ctx, Hkv, d, device="cuda", generator=gen).bfloat16()
    alpha = torch.rand(n, H, device="cuda", generator=gen) * 0.8 + 0.1
    path, count = dev([0] + sorted(rng.choice(np.arange(1, n), 9, replace=False).tolist()) + [-1] * (n - 10)), dev([10])
    cache = pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv])
    assert cache.k.numel() > 1 << 32
    results = []
    for first in (0, pages - 4):
        table, cu, at = dev([[first + 2, first, first + 3, first + 1]]), dev([0, n]), dev([ctx])
        pa.cache_append(old[0], old[1], cache, table, dev([0, ctx]), dev([0]))
        q = pa.rotary_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], r, cache, table, cu, at, parent)
        out, lse = pa.extend_tree(q, cache, table, cu, at, parent, alpha, 64, 100, 2)
        pa.cache_keep(cache, table, cu, at, path, count)
        results.append((q, out, lse, *pa.cache_read(cache, table, dev([0, ctx + n]), dev([0]), ctx + n)))
    assert pa.status() == 0 and all(torch.equal(a, b) for a, b in zip(*results))
    assert not torch.equal(results[0][3][ctx + 1:ctx + 10], torch.zeros_like(results[0][3][ctx + 1:ctx + 10]))


# ------------------------------------------------------------------ verification

@pytest.mark.parametrize("drawn", [False, True])
def test_a_sum_over_a_long_row_finds_its_token(drawn):
    """2^25 tokens to one CTA (there are that many sequences, all but one without tokens).  Half of the tokens have a probability whose running
    sums round, the others a power of two, and the next token lies among those; every exact sum here is a multiple of 2^-25 below
    2^25, so 64 bits hold it.  The kernel's sums are within 2^-42 + V 2^-54 of the whole, 0.08 tokens of 0.5 here, the running one and the whole one
    that the number multiplies: 0.16 tokens, so borders nearer than 0.2 are left out."""
    V, B, c = 1 << 25, 160, float(np.float32(0.743142128))
    half = V // 2
    target = torch.full((2 if drawn else 1, V), 0.5, device="cuda")
    target[:, :half] = c
    T, tokens, parent, draft = 1, [0], [-1], None
    if drawn:  # a drafted token that is refused (r q = 0.9 > p = 0.5) takes its own weight alone: q is 0 elsewhere
        T, tokens, parent = 2, [0, V - 1], [-1, 0]
        draft = torch.zeros(2, V, device="cuda")
        draft[0, V - 1] = 1.0
    whole = c * half + 0.5 * (half - drawn)
    cu = dev([0] + [T] * B)
    u = torch.full((T,), 0.9, device="cuda")
    seen = 0
    for want_u in np.linspace(0.6, 0.99, 80):
        u_next = np.float32(want_u)
        x = (float(u_next) * whole - c * half) / 0.5
        if not 0.2 < x % 1 < 0.8:
            continue
        seen += 1
        un = torch.full((B,), float(u_next), device="cuda")
        path, count, token = pa.verify_tree(target, draft, dev(tokens), cu, dev(parent), u, un)
        assert int(token[0]) == half + int(x) and int(count[0]) == 1
    assert seen > 30


def test_weights_that_are_nearly_nothing():
    """After two refusals p is a q but for its rounding: weights of 2^-26 of p, some positive and some not, which the low part of a decides.  The
    next token against exact fractions; the kernel's weights are within 2^-46 of p, 2^-20 of one another's sum."""
    rng, B, V = np.random.default_rng(1), 400, 9
    target, draft = np.zeros((3 * B, V), dtype=np.float32), np.zeros((3 * B, V), dtype=np.float32)
    u_next, want = np.zeros(B, dtype=np.float32), []
    for b in range(B):
        while True:
            q = rng.random(V - 1) + 0.1
            q = (q / q.sum()).astype(np.float32)
            p = (np.float64(1.0 + rng.random() * 0.8) * q).astype(np.float32)
            a = 1 + sum(Fraction(float(x)) - Fraction(float(y)) for x, y in zip(p, q))
            w = [max(Fraction(float(x)) - a * Fraction(float(y)), 0) for x, y in zip(p, q)]
            r = np.float32(rng.random())
            goal, upto, at = Fraction(float(r)) * sum(w), Fraction(0), None
            near = []
            for v, x in enumerate(w):
                upto += x
                near.append(abs(float(upto - goal)))
                if at is None and upto > goal:
                    at = v
            if at is not None and min(near) > 2.0 ** -40 and max(float(x) for x in p) <= 1:
                break
        # the last token is refused whenever it is drawn: p is 0 there
        target[3 * b, :V - 1], draft[3 * b, :V - 1], draft[3 * b, V - 1] = p, q, 0.5
        u_next[b] = r
        want.append(at)
    tokens, parent = np.tile([0, V - 1, V - 1], B), np.tile([-1, 0, 0], B)
    got = pa.verify_tree(torch.from_numpy(target).cuda(), torch.from_numpy(draft).cuda(), dev(tokens), dev(3 * np.arange(B + 1)), dev(parent),
                         torch.full((3 * B,), 0.5, device="cuda"), torch.from_numpy(u_next).cuda())
    assert got[1].tolist() == [1] * B and got[2].tolist() == want
