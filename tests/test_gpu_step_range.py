"""GPU tests of rotary positions and of the speculative step at the ends of their ranges: sums over long rows."""
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
