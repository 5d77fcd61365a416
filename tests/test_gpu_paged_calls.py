"""GPU: calls of the paged cache that its documentation allows, at their edges."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import structured_sparse_long_gb300 as pa
from structured_sparse_long_gb300 import build as pbuild

pytestmark = pytest.mark.gpu

PI = pa.MODE_PI


@pytest.fixture(scope="module", autouse=True)
def built():
    pbuild.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    pa.load()
    yield
    assert pa.status() == 0


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Sequence:
    """One sequence of N rows in shuffled pages, and queries for its last n positions."""

    def __init__(self, N, n, H, Hkv, d, page, kv, seed, spoil=()):
        gen = torch.Generator().manual_seed(seed)
        self.N, self.n, self.ctx = N, n, N - n
        self.q, k, v = (torch.randn(m, h, d, generator=gen).to(torch.bfloat16) for m, h in ((n, H), (N, Hkv), (N, Hkv)))
        for pos, value in spoil:  # values that are not finite
            v[pos] = value
        pages = -(-N // page)
        self.cache = pa.PagedCache.empty(pages, Hkv, page, d, ref.DTYPE[kv])
        self.table = torch.randperm(pages, generator=gen).int().cuda()[None]
        pa.cache_append(k.cuda(), v.cuda(), self.cache, self.table, ints(0, N), ints(0))
        self.k, self.v = (x.cpu() for x in pa.cache_read(self.cache, self.table, ints(0, N), ints(0), N))

    def extend(self, alpha, *args, **kw):
        return pa.extend(self.q.cuda(), self.cache, self.table, ints(0, self.n), ints(self.ctx), alpha.cuda(), *args, **kw)

    def check(self, got, alpha, *args):
        ref.check_attention("rows", *got, ref.attention(self.q, self.k, self.v, alpha, self.ctx, *args, PI))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_a_workspace_of_the_size_asked_for(kv):
    """Zero bytes (short chunks: an empty tensor) and more (long ones)."""
    for n, H, Hkv in ((3, 8, 2), (300, 20, 1)):  # (20 heads on one: always the long chunks' kernels)
        s = Sequence(n + 50, n, H, Hkv, 64, 16, kv, seed=n)
        a = torch.full((n, H), 0.5)
        need = pa.extend_workspace_size(s.cache, 1, n, s.table.shape[1], H, 40, 64, 2)
        assert (need == 0) == (n == 3)
        got = s.extend(a, 40, 64, 2, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        s.check(got, a, 40, 64, 2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("n", [2, 600])
def test_rows_without_a_finite_logit_are_zero(kv, n):
    """alpha = 0 leaves a row its skips alone, and the first rows none at all: out 0 and lse -inf there, whatever the band's values
    are, infinities and NaN among them; the other rows are the oracle's."""
    H, Hkv, d, kl, per, S = 16, 4, 128, 30, 500, 1  # skips from position 500 on
    N = max(n, 40)
    spoil = [(N - n, float("nan")), (N - 1, float("inf"))] + ([(x, float("nan")) for x in (100, 260, 390)] if n > 2 else [])
    s = Sequence(N, n, H, Hkv, d, 64, kv, seed=n, spoil=spoil)
    alpha = torch.rand(n, H, generator=torch.Generator().manual_seed(1)) * 0.5 + 0.25
    empty = torch.zeros(n, H, dtype=torch.bool)
    empty[::3, 1::2] = True
    empty[:, 5] = empty[-1] = True
    alpha[empty] = 0.0
    pos = torch.arange(N - n, N)
    empty &= (pos < per)[:, None]
    assert empty.any()
    assert (pa.extend_workspace_size(s.cache, 1, n, s.table.shape[1], H, kl, per, S) == 0) == (n == 2)  # both kernels
    got = s.extend(alpha, kl, per, S)
    torch.cuda.synchronize()
    out, lse = got[0].float().cpu(), got[1].cpu()
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    if n > 2:  # rows that attend none of the spoilt values
        clean = torch.tensor([all(not (p - kl <= x <= p or (p - per == x)) for x, _ in spoil) for p in pos.tolist()])
        ro, rl, size = ref.attention(s.q, s.k, torch.nan_to_num(s.v, nan=0.0, posinf=0.0, neginf=0.0), alpha, s.ctx, kl, per, S, PI)
        rows = clean.numpy()
        ref.check_attention("clean rows", got[0][clean.cuda()], got[1][clean.cuda()], (ro[rows], rl[rows], size[rows]))
    # the same row as a single token
    one, ls = pa.decode_paged(s.q[:1].cuda(), s.cache, s.table, ints(s.ctx + 1), torch.zeros(1, H, device="cuda"), kl, per, S)
    torch.cuda.synchronize()
    assert (one == 0).all() and torch.isneginf(ls).all()


@pytest.mark.parametrize("S", [4, 64, 2 ** 31 - 1])
def test_more_skips_than_the_table_reaches(S):
    """Whatever S is beyond the skips that lie before a token, the results are the same."""
    s = Sequence(900, 3, 8, 2, 128, 64, "bf16", seed=3)
    a = torch.full((3, 8), 0.4)
    got = s.extend(a, 64, 200, S)
    s.check(got, a, 64, 200, 4)
    one = pa.decode_paged(s.q[-1:].cuda(), s.cache, s.table, ints(900), a[-1:].cuda(), 64, 200, S)
    want = ref.attention(s.q, s.k, s.v, a, s.ctx, 64, 200, 4, PI)
    ref.check_attention("token", *one, [x[-1:] for x in want])
