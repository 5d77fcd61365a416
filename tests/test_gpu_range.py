"""GPU: the forwards' range.  A row's output is a mean of the values it attends, so it is finite whenever they are, for values
up to fp32's largest over the row's number of keys; its unnormalised sum must not overflow on the way.

The kernels keep a softmax reference that may lag behind the row's largest logit.  Here a row's first keys score 0 and later
ones 11 (log2 units), which a lagging reference turns into weights of 2^11 before the division: 150 keys of those, or seven
under the skips, times the values used here are past 2^128, while the weights relative to the row's largest logit are at most one
each."""
import numpy as np
import pytest
import torch

import oracle
import paged_ref as ref
import structured_sparse_long_gb300 as pa
from structured_sparse_long_gb300 import build as pbuild

pytestmark = pytest.mark.gpu

PI, ECP, BIDIR = pa.MODE_PI, pa.MODE_ECP, pa.MODE_PI_BIDIR


@pytest.fixture(scope="module", autouse=True)
def built():
    pbuild.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    pa.load()
    yield
    assert pa.status() == 0


CASES = [
    # k_local, period, S, mode, size of the values, hot(j): keys with the large logits
    ("band", 300, 1, 0, PI, 2.0 ** 112, lambda j: (j // 150) % 2 == 1),
    ("band-larger", 300, 1, 0, PI, 2.0 ** 117, lambda j: (j // 150) % 2 == 1),
    ("skips", 40, 64, 6, PI, 2.0 ** 116, lambda j: j % 64 >= 60),
    ("ecp", 200, 0, 0, ECP, 2.0 ** 112, lambda j: (j // 150) % 2 == 1),
    ("both-ways", 200, 256, 1, BIDIR, 2.0 ** 112, lambda j: (j // 150) % 2 == 1),
]


def inputs(d, N, H, Hkv, size, hot, seed):
    """Queries of +-1 and keys along them: a hot key's logit is 11 log2 units (d / sqrt(d) * key * log2(e)), a cold one's about 0."""
    gen = torch.Generator().manual_seed(seed)
    sign = torch.where(torch.rand(d, generator=gen) < 0.5, -1.0, 1.0)
    q = sign.expand(1, H, N, d).contiguous()
    key = torch.where(hot(torch.arange(N)), 11 / 1.4427 / d ** 0.5, 0.0)
    k = key[:, None] * sign + 0.01 * torch.randn(1, Hkv, N, d, generator=gen)
    v = size * torch.randn(1, Hkv, N, d, generator=gen)
    return [x.to(torch.bfloat16) for x in (q, k, v)]


def check(name, out, lse, q, k, v, alpha, kl, per, S, mode, rows=slice(None)):
    ro, rl = oracle.fwd(q, k, v, alpha, kl, per, S, mode)
    size, _ = oracle.fwd(q, k, v.abs(), alpha, kl, per, S, mode)
    ref.check_attention(name, out, lse, (ro[:, :, rows], rl[:, :, rows], size[:, :, rows]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_large_values_stay_finite(case, d):
    name, kl, per, S, mode, size, hot = case
    N, H, Hkv = 700, 4, 2
    q, k, v = inputs(d, N, H, Hkv, size, hot, seed=d)
    alpha = None if mode == ECP else torch.full((1, H, N), 0.5)
    dv = [x.cuda() for x in (q, k, v)]
    da = None if alpha is None else alpha.cuda()
    out, lse = pa.fwd(*dv, da, kl, per, S, mode)
    check(name, out, lse, q, k, v, alpha, kl, per, S, mode)
    if mode != BIDIR:
        first = 384
        out, lse = pa.fwd_shard(dv[0][:, :, first:].contiguous(), dv[1], dv[2], None if da is None else da[:, :, first:].contiguous(), first,
                                kl, per, S, mode)
        check(name + " shard", out, lse, q, k, v, alpha, kl, per, S, mode, slice(first, None))
    if mode == PI:  # weights of zero: the gate is sigmoid(0)
        gate = (torch.zeros(H, 8, d, dtype=torch.bfloat16).cuda(), *(torch.zeros(s).cuda() for s in ((H, 8), (H, 8), (H,))))
        out, lse, _ = pa.fwd_gated(*dv, gate, kl, per, S, mode)
        check(name + " gated", out, lse, q, k, v, alpha, kl, per, S, mode)


@pytest.mark.parametrize("case", CASES[:4], ids=[c[0] for c in CASES[:4]])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_large_values_over_pages(case, kv):
    """The same rows as a chunk over a paged cache, and its last as a single token."""
    name, kl, per, S, mode, size, hot = case
    d, N, H, Hkv, page, ctx = 128, 700, 16, 4, 32, 60
    q, k, v = (x[0].transpose(0, 1).contiguous() for x in inputs(d, N, H, Hkv, size, hot, seed=5))
    pages = -(-N // page)
    cache = pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv])
    table, n = torch.arange(pages, dtype=torch.int32).cuda()[None], N - ctx
    at = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    pa.cache_append(k.cuda(), v.cuda(), cache, table, at(0, N), at(0))
    held = [x.cpu() for x in pa.cache_read(cache, table, at(0, N), at(0), N)]
    alpha = None if mode == ECP else torch.full((n, H), 0.5)
    da = None if alpha is None else alpha.cuda()
    out, lse = pa.extend(q[ctx:].cuda(), cache, table, at(0, n), at(ctx), da, kl, per, S, mode)
    want = ref.attention(q[ctx:], *held, alpha, ctx, kl, per, S, mode)
    ref.check_attention(name, out, lse, want)
    out, lse = pa.decode_paged(q[-1:].cuda(), cache, table, at(N), None if da is None else da[-1:], kl, per, S, mode)
    ref.check_attention(name + " token", out, lse, [x[-1:] for x in want])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slope", [0.2, 0.37, 1.0, -0.4])
@pytest.mark.parametrize("k_local,mode", [(250, PI), (96, ECP), (200, BIDIR)])
def test_logits_that_rise_along_the_keys(d, slope, k_local, mode):
    """Logits that rise (or fall) by `slope` log2 units per key over runs of 300 keys: the reference moves within tiles, between them,
    in tiles with and without masks.

    A logit z is a sum of d products of one sign in 32 bits, off by at most d 2^-24 |z|, and |z| <= 300 |slope| ln 2 and a bit;
    a weight is off by as much, relative, lse by as much, and the output by twice that of sum p |v|, beside the roundings of
    paged_ref.check_attention."""
    N, H, Hkv, S, per = 700, 4, 2, (0 if mode == ECP else 2), 256
    q, _, v = inputs(d, N, H, Hkv, 1.0, lambda j: j < 0, seed=9)
    gen = torch.Generator().manual_seed(1)
    rise = slope * (torch.arange(N) % 300) / 1.4427 / d ** 0.5
    k = (rise[:, None] * q[0, 0, 0].float() + 0.01 * torch.randn(1, Hkv, N, d, generator=gen)).to(torch.bfloat16)
    alpha = None if mode == ECP else torch.full((1, H, N), 0.5)
    out, lse = pa.fwd(q.cuda(), k.cuda(), v.cuda(), None if alpha is None else alpha.cuda(), k_local, per, S, mode)
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    ro, rl = oracle.fwd(q, k, v, alpha, k_local, per, S, mode)
    size, _ = oracle.fwd(q, k, v.abs(), alpha, k_local, per, S, mode)
    eps = d * 2.0 ** -24 * (300 * abs(slope) * 0.6932 + 8)
    assert (np.abs(out - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -12 + 2 * eps) * size).all()
    assert (np.abs(lse - rl) <= 2.0 ** -12 + eps + 2.0 ** -22 * np.abs(rl)).all()
