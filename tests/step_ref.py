"""64-bit references of rotary positions and of a speculative serving step (numpy; shares no code with the kernels)."""
import math

import numpy as np
import torch

import paged_ref as ref


def rotate(x, pos, rope, sign=1):
    """x [..., d] (any float type) turned by pos [...], and the sum of a pair's magnitudes for every element."""
    x = np.asarray(x, dtype=np.float64)
    y, size = x.copy(), np.zeros_like(x)
    half = rope.rot // 2
    for t, f in enumerate(rope.freqs):
        a, b = (2 * t, 2 * t + 1) if rope.interleaved else (t, t + half)
        w = sign * np.asarray(pos, dtype=np.float64) * f
        y[..., a] = rope.scale * (x[..., a] * np.cos(w) - x[..., b] * np.sin(w))
        y[..., b] = rope.scale * (x[..., a] * np.sin(w) + x[..., b] * np.cos(w))
        size[..., a] = size[..., b] = abs(rope.scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


# An angle is off by 2^-24 of a half turn (its fp32 form), i.e. pi 2^-24; sine and cosine by an ulp, 2^-23; the scale's product, the two
# of a pair and their sum round by 2^-24 each: below 2^-20 of the pair's magnitudes in all.  (The reference's own angles, position times
# frequency in 64 bits, are off by 2^-53 of up to 2^21 radians at the positions used.)
SLACK = 2.0 ** -20


def check_rotated(name, got, want, size, eps):
    """got rounded once from 32 bits (half a step: eps / 2 of the value)."""
    off = np.abs(np.asarray(got, dtype=np.float64) - want)
    bound = eps / 2 * np.abs(want) + (1 + eps) * SLACK * size + 1e-37
    assert (off <= bound).all(), f"{name}: off by {(off / bound).max():.3f} of its bound at {np.unravel_index((off / bound).argmax(), off.shape)}"


def check_quantised(name, codes, scales, want, size, kv):
    """8-bit rows of elements known to SLACK * size: the scales the smallest that may be, each code the nearest."""
    b = lambda x: x.reshape(*x.shape[:-1], -1, 32)  # noqa: E731
    top, slack = np.abs(b(want)).max(-1), SLACK * b(size).max(-1)
    e = scales.astype(np.float64) - 127
    assert (top - slack <= ref.QMAX[kv] * 2.0 ** e).all(), f"{name}: a scale too small"
    assert ((top + slack > ref.QMAX[kv] * 2.0 ** (e - 1)) | (e == -120)).all(), f"{name}: a scale too large"
    got = ref.decode(codes, scales, kv)
    unit = np.repeat(2.0 ** e, 32, -1)
    if kv == "int8":
        half = 0.5 * unit
    else:  # half a step: 2^-4 of the value's power of two, at least of 2^-6 scaled
        half = 2.0 ** -4 * np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(want), 1e-300))), 2.0 ** -6 * unit)
    off = np.abs(got - want)
    assert (off <= (1 + 2.0 ** -19) * half + SLACK * size).all(), f"{name}: a code off by {(off / half).max():.3f} half steps"


def depths(parent):
    out = []
    for p in parent:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def line(parent, j):
    """Node j's ancestors and itself, from the root down."""
    out = []
    while j >= 0:
        out.append(j)
        j = parent[j]
    return out[::-1]


def random_tree(n, rng, deep=6, roots=1):
    """Parents of n nodes, paths of at most `deep` nodes where that is possible."""
    parent = []
    for j in range(n):
        d = depths(parent)
        free = [x for x in range(j) if d[x] + 1 < deep] or list(range(j))
        parent.append(-1 if j < roots else int(rng.choice(free)))
    return parent


def tree_attention(q, k, v, alpha, ctx, parent, k_local, period, S, mode):
    """Rows of a tree whose node j has row ctx + j of k, v [ctx + n, Hkv, d]: each is the last row of its own text."""
    rows = []
    for j in range(len(parent)):
        at = list(range(ctx)) + [ctx + x for x in line(parent, j)]
        rows.append(ref.attention(q[j:j + 1], k[at], v[at], None if alpha is None else alpha[j:j + 1], len(at) - 1, k_local, period, S, mode))
    return tuple(np.concatenate([r[i] for r in rows]) for i in range(3))


def verify(target, draft, tokens, parent, u, u_next):
    """One sequence: (path, next token), by the residual distributions themselves."""
    def clean(row):
        row = np.asarray(row, dtype=np.float64)
        return np.clip(np.nan_to_num(row, nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)

    x, path = 0, [0]
    while True:
        p = clean(target[x])
        left, mass, took = p.copy(), 1.0, None  # the residual times `mass`
        for c in [j for j in range(len(parent)) if parent[j] == x]:
            t, r = int(tokens[c]), float(u[c])
            if draft is not None:
                q = clean(draft[x])
                if r * q[t] * mass < left[t]:
                    took = c
                    break
                left = np.maximum(left / mass - q, 0.0) if mass > 0 else left * 0
                mass = math.fsum(left)
            else:
                if r * mass < left[t]:
                    took = c
                    break
                mass -= left[t]
                left[t] = 0.0
        if took is None:
            break
        x = took
        path.append(x)
    if not left.sum() > 0:
        left = p
    if not left.sum() > 0:
        return path, -1
    goal = float(u_next) * math.fsum(left)
    upto = np.cumsum(left)
    past = np.nonzero(upto > goal)[0]
    return path, int(past[0]) if len(past) else int(np.nonzero(left)[0][-1])
