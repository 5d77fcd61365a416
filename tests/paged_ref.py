"""64-bit reference of the paged cache's formats and batches (numpy; shares no code with the kernels)."""
import numpy as np
import torch

import oracle

QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def e4m3_grid():
    """Value of every e4m3 code without sign, 0x00 .. 0x7e."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def encode(x, kv):
    """x [..., d] (bf16 values) -> (codes [..., d] uint8 bits, scale bytes [..., d / 32]).

    The scale is searched upwards from the smallest one, and an e4m3 code among all its neighbours:
    nothing here follows the kernel's bit arithmetic."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    finite = np.isfinite(b).all(-1)
    b = np.where(finite[..., None], b, 0.0)
    amax = np.abs(b).max(-1)
    e = np.full(amax.shape, -120)
    for cand in range(-119, 128):
        e = np.where(amax > QMAX[kv] * 2.0 ** (cand - 1), cand, e)
    y = b * np.exp2(-e.astype(np.float64))[..., None]
    if kv == "int8":
        codes = np.rint(y).astype(np.int64) & 0xFF
    else:
        grid = e4m3_grid()
        mid = (grid[1:] + grid[:-1]) / 2
        a = np.abs(y)
        lo = np.searchsorted(mid, a, side="left")   # a tie goes down ...
        hi = np.searchsorted(mid, a, side="right")  # ... or up:
        codes = np.where(lo % 2 == 0, lo, hi)       # to the even code
        codes = codes | (np.signbit(y).astype(np.int64) << 7)
    codes = np.where(finite[..., None], codes, 0)
    return codes.reshape(x.shape).astype(np.uint8), np.where(finite, e + 127, 255).astype(np.uint8)


def decode(codes, scales, kv):
    """Values of codes [..., d] (uint8 bits) with scale bytes [..., d / 32], float64; infinity from 2^128 on, which
    a code that was rounded up can stand for (255 * 2^120, bf16's largest number, is 256 * 2^120 in e4m3 and
    64 * 2^122 in int8) and neither bf16 nor fp32 holds."""
    c = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    if kv == "int8":
        v = c.view(np.int8).astype(np.float64)
    else:
        grid = np.append(e4m3_grid(), np.nan)
        v = grid[c & 0x7F] * np.where(c & 0x80, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    x = (v * s[..., None]).reshape(codes.shape)
    return np.where(np.abs(x) >= 2.0 ** 128, np.copysign(np.inf, x), x)


def bits(t):
    """A page tensor's raw contents as numpy integers."""
    t = t.detach().cpu().contiguous()
    return t.view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.view(torch.uint8).numpy()


def make_table(ctx, n, page, rng, extra=2, width_extra=1):
    """A page table of shuffled pages for sequences of ctx + n rows, and the number of pages."""
    used = [-(-(c + m) // page) for c, m in zip(ctx, n)]
    pages = sum(used) + extra
    order = rng.permutation(pages)
    table = np.full((len(ctx), max(max(used), 1) + width_extra), -1, dtype=np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    return table, pages


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def attended_pages(first, last, page, k_local, period, S, ecp):
    """Pages of one sequence that hold a key of some query at positions first .. last."""
    keep = set()
    for i in range(first, last + 1):
        if ecp:
            keys = range(max(0, (i // k_local - 1) * k_local), i + 1)
        else:
            keys = list(range(max(0, i - k_local), i + 1)) + [i - m * period for m in range(1, S + 1)
                                                               if m * period > k_local and i >= m * period]
        keep |= {j // page for j in keys}
    return keep


def attention(q, k, v, alpha, first, k_local, period, S, mode):
    """Rows first .. N-1 of the oracle's forward for one sequence, and sum_j p_ij |v_j| (the size that
    rounding P to bf16 acts on).  q [n, H, d], k, v [N, Hkv, d], alpha [n, H] or None."""
    n, H, d = q.shape
    N = k.shape[0]

    def whole(x, fill):
        y = torch.full((1, H, N) + x.shape[2:], fill, dtype=x.dtype)
        y[0, :, first:] = x.transpose(0, 1)
        return y
    qf, kf, vf = whole(q, 0.0), k.transpose(0, 1)[None].contiguous(), v.transpose(0, 1)[None].contiguous()
    af = None if alpha is None else whole(alpha, 0.5)
    out, lse = oracle.fwd(qf, kf, vf, af, k_local, period, S, mode, rows=(first, N))
    size, _ = oracle.fwd(qf, kf, vf.abs(), af, k_local, period, S, mode, rows=(first, N))
    return out[0].transpose(1, 0, 2), lse[0].T, size[0].transpose(1, 0, 2)


def check_attention(name, out, lse, ref):
    """The kernels round P to bf16 (half a step: 2^-8 of each p, so 2^-8 of sum p |v|), the output to bf16
    (2^-8 of it), and sum a score's d products in 32 bits: with |q . k| / sqrt(d) and sum |q k| / sqrt(d) of
    order 10, d 2^-24 of that is below 2^-13, which moves each p by as much and lse by twice that at most."""
    ro, rl, size = ref
    out, lse = out.detach().float().cpu().numpy().astype(np.float64), lse.detach().cpu().numpy().astype(np.float64)
    bound = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -12) * size + 1e-30
    off = np.abs(out - ro)
    assert np.isfinite(out).all() and (off <= bound).all(), (
        f"{name}: out off by {(off / bound).max():.3f} of its bound at {np.unravel_index((off / bound).argmax(), off.shape)}")
    fin = np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse), ~fin), f"{name}: rows without a key differ"
    off = np.abs(lse[fin] - rl[fin])
    bound = 2.0 ** -12 + 2.0 ** -22 * np.abs(rl[fin])
    assert (off <= bound).all(), f"{name}: lse off by {off.max():.3e}"
