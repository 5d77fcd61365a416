"""GPU tests of rotary positions and of the speculative step at the ends of their ranges: sums over long rows, weights that are nearly
nothing."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import structured_sparse_long_gb300 as pa
from structured_sparse_long_gb300 import build as pbuild

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


# ------------------------------------------------------------------ verification

@pytest.mark.parametrize("drawn", [False, True])
def test_a_sum_over_a_long_row_finds_its_token(drawn):
    """2^25 tokens to one CTA (there are that many sequences, all but one without tokens).  Half of the tokens have a probability whose running
    sums round, the others a power of two, and the next token lies among those; every exact sum here is a multiple of 2^-25 below
    2^25, so 64 bits hold it.  The kernel's sums are within 2^-43 + V 2^-54 of the whole, 0.04 tokens of 0.5 here."""
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
    for want_u in np.linspace(0.6, 0.99, 40):
        u_next = np.float32(want_u)
        x = (float(u_next) * whole - c * half) / 0.5
        if not 0.1 < x % 1 < 0.9:
            continue
        seen += 1
        un = torch.full((B,), float(u_next), device="cuda")
        path, count, token = pa.verify_tree(target, draft, dev(tokens), cu, dev(parent), u, un)
        assert int(token[0]) == half + int(x) and int(count[0]) == 1
    assert seen > 20


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
