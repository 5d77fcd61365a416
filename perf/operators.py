"""Measured cases of the paged key/value cache operators.

Four operators of a serving step, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and, with ``own`` set, through this package's entry points:

  append  the new tokens' K and V rows written into their sequences' cache pages, quantised to
          8 bits on the way where the cache holds 8 bits
  read    rows of the cache read back into packed bf16 tensors (a prefix handed to another worker)
  extend  pi-Attention / ECP attention of a chunk of new tokens per sequence over the paged cache
  decode  the same for one new token per sequence

A batch is B sequences.  Sequence b has ctx[b] rows in the cache before the call and n[b] new ones;
the new tokens are packed, those of sequence b at cu[b] .. cu[b+1]-1, and take positions ctx[b] ...
Position p of sequence b lives in row p % page of page table[b, p // page].  Pages are
[pages, Hkv, page, d].  An 8-bit cache holds, per row and block of 32 elements, codes (e4m3 or int8)
and one scale byte s that stands for 2^(s - 127): the smallest power of two that brings the block's
largest magnitude to at most 448 (e4m3) or 127 (int8), not below 2^-120.  Powers of two scale
without rounding, so a code is the block's element rounded once, to nearest even.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases

def _case(name, op, kv, B, n, ctx, H, Hkv, d, page, k_local=256, period=1024, S=4, ecp=False, ragged=False, shape=0):
    return {"name": name, "op": op, "kv": kv, "B": B, "n": n, "ctx": ctx, "H": H, "Hkv": Hkv, "d": d, "page": page,
            "k_local": k_local, "period": period, "S": S, "ecp": ecp, "ragged": ragged, "shape": shape}


def listed():
    return [
        # a decode step's write: one token of each of 64 sequences, where only latency counts
        _case("append-token-e4m3", "append", "e4m3", 64, 1, 4095, 16, 4, 128, 64, ragged=True, shape=1),
        # a whole 64k prompt of the long-context GQA layer written at once
        _case("append-prompt-int8", "append", "int8", 1, 65536, 0, 16, 4, 128, 64),
        # four prompts of the language-model layer into an unquantised cache of small pages
        _case("append-lm-bf16", "append", "bf16", 4, 4096, 37, 12, 12, 64, 16),
        # a long prefix handed over in bf16
        _case("read-context-e4m3", "read", "e4m3", 1, 65536, 0, 16, 4, 128, 64),
        # ragged prefixes that start and end inside pages
        _case("read-ragged-int8", "read", "int8", 7, 1500, 900, 16, 16, 64, 16, ragged=True, shape=2),
        # five drafted tokens of 16 sequences checked at once: latency
        _case("extend-draft-bf16", "extend", "bf16", 16, 5, 16000, 16, 4, 128, 32, ragged=True, shape=3),
        # a long chunk of a 64k prompt: the long-context layer's ordinary prefill
        _case("extend-long-bf16", "extend", "bf16", 1, 16384, 49152, 16, 4, 128, 64),
        # continuous batching: chunks of many lengths at odd contexts over an 8-bit cache
        _case("extend-mixed-e4m3", "extend", "e4m3", 12, 2000, 16000, 16, 4, 128, 64, ragged=True, shape=4),
        # paired-segment attention, every query head with its own cache head
        _case("extend-ecp-int8", "extend", "int8", 2, 2048, 6144, 16, 16, 64, 128, k_local=512, period=0, S=0, ecp=True),
        # the benchmarked decode step of the long-context layer, 64 sequences
        _case("decode-batch-bf16", "decode", "bf16", 64, 1, 16383, 16, 4, 128, 64),
        # one user's next token at 64k: latency
        _case("decode-one-e4m3", "decode", "e4m3", 1, 1, 65535, 16, 4, 128, 64),
        # the language-model layer, ragged contexts, small pages
        _case("decode-lm-int8", "decode", "int8", 32, 1, 4095, 12, 12, 64, 16, k_local=128, period=256, S=1, ragged=True,
              shape=5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "extend", "extend", "decode", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12, 16] if d == 64 else [1, 2, 4, 8])
    H = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if Hkv * g <= 16])
    page = rng.choice([16, 32, 64, 128, 256])
    ecp = op in ("extend", "decode") and rng.random() < 0.25
    k_local = rng.choice([96, 128, 200, 256, 512]) if ecp else _spread(rng, 8, 512)
    period = 0 if ecp else _spread(rng, 32, 2048)
    S = 0 if ecp else rng.randint(0, 5)
    if op == "decode":
        B, n = _spread(rng, 1, 64), 1
    elif op == "extend":
        n = _spread(rng, 1, 4096)
        B = rng.randint(1, max(1, min(24, 6000 // (n * max(1, Hkv // 4)))))
    else:
        n = _spread(rng, 1, 32768)
        B = rng.randint(1, max(1, min(64, 40000 // n)))
    ctx = _spread(rng, 1, 16384)
    c = _case("", op, rng.choice(["bf16", "e4m3", "int8"]), B, n, ctx, H, Hkv, d, page, k_local, period, S, ecp,
              rng.random() < 0.7, rng.randrange(1 << 30))
    del c["name"]
    return c


def _lengths(case):
    """Per sequence: rows in the cache before the call, and new rows."""
    B, n, ctx = case["B"], case["n"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * B, [n] * B
    rng = random.Random(case["shape"])
    return [rng.randint(0, ctx) for _ in range(B)], [rng.randint(1, n) for _ in range(B)]


# ------------------------------------------------------------------ inputs

def _scale_of(byte):
    """2^(byte - 127) from its bits; a byte of 255 marks a block with a non-finite element."""
    f = (byte.to(torch.int32) << 23).view(torch.float32)
    return torch.where(byte == 255, torch.full_like(f, math.nan), f)


def _quantise(x, kv):
    """x [..., d] -> codes [..., d], scale bytes [..., d / 32]."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    # 448 = 0.875 * 2^9 and 127 = 0.9921875 * 2^7
    top, up = (0.875, 9) if kv == "e4m3" else (0.9921875, 7)
    e = torch.clamp(e - up + (m > top), min=-120)
    e = torch.where(amax == 0, torch.full_like(e, -120), e)
    y = b * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)  # times 2^-e
    codes = y.to(torch.float8_e4m3fn) if kv == "e4m3" else torch.round(y).to(torch.int8)
    return codes.flatten(-2), (e + 127).to(torch.uint8)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    ctx, n = _lengths(case)
    B, H, Hkv, d, page, kv = (case[x] for x in ("B", "H", "Hkv", "d", "page", "kv"))
    T = sum(n)
    used = [-(-(c + m) // page) for c, m in zip(ctx, n)]
    width = max(used) + 1
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
    table = torch.full((B, width), -1, device=dev, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    cu = torch.tensor([sum(n[:b]) for b in range(B + 1)], device=dev, dtype=torch.int32)
    s = {**{x: case[x] for x in ("op", "kv", "H", "Hkv", "d", "page", "k_local", "period", "S", "ecp")}, "T": T,
         "table": table, "cu": cu, "ctx": torch.tensor(ctx, device=dev, dtype=torch.int32)}

    def pool():
        x = torch.randn(pages, Hkv, page, d, generator=g, device=dev, dtype=torch.float32)
        x[..., 5::48] *= 6.0  # the few large channels that keys have
        x = x.to(torch.bfloat16)
        return (x, None) if kv == "bf16" else _quantise(x, kv)

    s["k"], s["ks"] = pool()
    s["v"], s["vs"] = pool()
    # the projection's output: queries, keys and values of a token next to one another
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g, device=dev, dtype=torch.float32)
    if case["op"] == "append":
        qkv[..., 5::48] *= 6.0
    qkv = qkv.to(torch.bfloat16)
    s["q"], s["k_new"], s["v_new"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    s["alpha"] = None if case["ecp"] else torch.sigmoid(1.5 * torch.randn(T, H, generator=g, device=dev))
    s["lens"] = s["ctx"] + 1  # decode: the rows of the cache, the new token's among them
    return s


# ------------------------------------------------------------------ plain form

def _tokens(s):
    """Sequence and position of every packed token."""
    t = torch.arange(s["T"], device=s["cu"].device)
    seq = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    return seq, s["ctx"][seq] + t - s["cu"][seq]


def _rows(s, pages, scales, seq, pos):
    """Cache rows at positions pos of sequences seq, in 32 bits: [..., Hkv, d]."""
    at = s["table"][seq, pos // s["page"]].long()
    x = pages[at, :, pos % s["page"]].float()
    if scales is None:
        return x
    return (x.unflatten(-1, (-1, 32)) * _scale_of(scales[at, :, pos % s["page"]]).unsqueeze(-1)).flatten(-2)


def _plain_append(s):
    seq, pos = _tokens(s)
    at, row = s["table"][seq, pos // s["page"]].long(), pos % s["page"]
    if s["kv"] == "bf16":
        s["k"][at, :, row] = s["k_new"]
        s["v"][at, :, row] = s["v_new"]
    else:
        s["k"][at, :, row], s["ks"][at, :, row] = _quantise(s["k_new"], s["kv"])
        s["v"][at, :, row], s["vs"][at, :, row] = _quantise(s["v_new"], s["kv"])


def _plain_attention(s, seq, pos):
    T, H, Hkv, d, c = s["T"], s["H"], s["Hkv"], s["d"], s["k_local"]
    dev = pos.device
    p = pos.long()[:, None]
    if s["ecp"]:  # the row's own half-segment and the one before it
        keys = torch.clamp((p // c - 1) * c, min=0) + torch.arange(2 * c, device=dev)
        band = keys <= p
        skip = torch.zeros_like(band)
    else:  # the band, then the skips that lie outside it
        m = torch.arange(1, s["S"] + 1, device=dev) * s["period"]
        keys = torch.cat([p - torch.arange(c + 1, device=dev), p - m[m > c]], 1)
        is_skip = torch.arange(keys.shape[1], device=dev) > c
        band, skip = (keys >= 0) & ~is_skip, (keys >= 0) & is_skip
    at = torch.where(band | skip, keys, torch.zeros_like(keys))
    K = _rows(s, s["k"], s["ks"], seq[:, None], at)  # [T, keys, Hkv, d]
    z = torch.matmul(s["q"].float().view(T, Hkv, H // Hkv, d), K.permute(0, 2, 3, 1)) / math.sqrt(d)
    del K
    off = torch.zeros(T, H, 1, device=dev) if s["alpha"] is None else torch.log(s["alpha"])[..., None]
    off_skip = off if s["alpha"] is None else torch.log(1 - s["alpha"])[..., None]
    z = z.view(T, H, -1)
    z = torch.where(band[:, None], z + off, torch.where(skip[:, None], z + off_skip, torch.full_like(z, -math.inf)))
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    V = _rows(s, s["v"], s["vs"], seq[:, None], at)
    out = torch.matmul((e / total).view(T, Hkv, H // Hkv, -1), V.permute(0, 2, 1, 3)).view(T, H, d)
    return out.to(torch.bfloat16), (top + torch.log(total))[..., 0]


def run(state):
    s = state
    if own:
        import structured_sparse_long_gb300 as pa
        if "cache" not in s:  # the handle of the pages, which a serving program keeps
            s["cache"] = pa.PagedCache(s["k"], s["v"], s["ks"], s["vs"])
        mode = pa.MODE_ECP if s["ecp"] else pa.MODE_PI
        if s["op"] == "append":
            pa.cache_append(s["k_new"], s["v_new"], s["cache"], s["table"], s["cu"], s["ctx"])
        elif s["op"] == "read":
            return pa.cache_read(s["cache"], s["table"], s["cu"], s["ctx"], s["T"])
        elif s["op"] == "extend":
            return pa.extend(s["q"], s["cache"], s["table"], s["cu"], s["ctx"], s["alpha"], s["k_local"], s["period"],
                             s["S"], mode)
        else:
            return pa.decode_paged(s["q"], s["cache"], s["table"], s["lens"], s["alpha"], s["k_local"], s["period"],
                                   s["S"], mode)
    elif s["op"] == "append":
        _plain_append(s)
    else:
        seq, pos = _tokens(s)
        if s["op"] == "read":
            return tuple(_rows(s, s[x], s[y], seq, pos).to(torch.bfloat16) for x, y in (("k", "ks"), ("v", "vs")))
        return _plain_attention(s, seq, pos)
    return [x for x in (s["k"], s["v"], s["ks"], s["vs"]) if x is not None]


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs_and_keys(case, ctx, n):
    """Attended (query, key) pairs and distinct keys of one sequence."""
    p0, p1, c = ctx, ctx + n, case["k_local"]
    if case["ecp"]:
        pairs = sum(p + 1 - max(0, (p // c - 1) * c) for p in range(p0, p1))
        return pairs, p1 - max(0, (p0 // c - 1) * c)
    ms = [m * case["period"] for m in range(1, case["S"] + 1) if m * case["period"] > c]
    pairs = sum(min(p, c) + 1 for p in range(p0, p1)) + sum(max(0, p1 - max(p0, m)) for m in ms)
    # windows, last first: the band's, then each skip's
    spans = sorted([(max(0, p0 - c), p1)] + [(max(0, p0 - m), p1 - m) for m in ms if p1 > m])
    keys, end = 0, 0
    for a, b in spans:
        a = max(a, end)
        keys += max(0, b - a)
        end = max(end, b)
    return pairs, keys


def work(case):
    ctx, n = _lengths(case)
    H, Hkv, d, T = case["H"], case["Hkv"], case["d"], sum(n)
    row = 2 * d if case["kv"] == "bf16" else d + d // 32  # bytes of a cache row of one head
    if case["op"] in ("append", "read"):
        return {"bytes": 2 * T * Hkv * (2 * d + row), "flops": 0}
    pairs, keys = (sum(x) for x in zip(*(_pairs_and_keys(case, c, m) for c, m in zip(ctx, n))))
    per_row = 4 * d + 4 + (0 if case["ecp"] else 4)  # q, out, lse, alpha
    return {"bytes": T * H * per_row + 2 * keys * Hkv * row, "flops": 4 * d * H * pairs}


# ------------------------------------------------------------------ 64 bits

def _exact_block(x, kv):
    """Codes (as values) and scale bytes of x [..., d], in 64 bits."""
    def power(n):  # 2^n, exact
        return ((n.long() + 1023) << 52).view(torch.float64)

    b = x.double().reshape(*x.shape[:-1], -1, 32)
    big = b.abs().amax(-1)
    e = torch.round(torch.log2(torch.clamp(big, min=2.0 ** -300) / QMAX[kv])) - 1
    e = (e + (big > QMAX[kv] * power(e))).clamp(min=-120)  # log2 is right to far less than one half
    e = e + (big > QMAX[kv] * power(e))
    y = b * power(-e)[..., None]
    if kv == "int8":
        codes = torch.round(y)
    else:
        size = y.abs().clamp(min=2.0 ** -6)
        n = torch.round(torch.log2(size)) - 1
        n = n + (size >= power(n + 1))
        step = power(n + (size >= power(n + 1)) - 3)
        codes = torch.round(y / step) * step
    return codes.reshape(x.shape), (e + 127).long()


def exact(case, seed):
    s = prepare(case, seed)
    ctx, n = _lengths(case)
    H, Hkv, d, page, c, kv = (case[x] for x in ("H", "Hkv", "d", "page", "k_local", "kv"))
    tables = s["table"].tolist()
    if case["op"] == "append":
        pages = [s["k"].double(), s["v"].double()]
        scales = [] if kv == "bf16" else [s["ks"].long(), s["vs"].long()]
        for i, name in enumerate(("k_new", "v_new")):
            codes, sc = (s[name].double(), None) if kv == "bf16" else _exact_block(s[name], kv)
            t = 0
            for b in range(case["B"]):
                p, end = ctx[b], ctx[b] + n[b]
                while p < end:
                    m = min(page - p % page, end - p)
                    at, r = tables[b][p // page], p % page
                    pages[i][at, :, r:r + m] = codes[t:t + m].transpose(0, 1)
                    if sc is not None:
                        scales[i][at, :, r:r + m] = sc[t:t + m].transpose(0, 1)
                    p, t = p + m, t + m
        if kv == "int8":
            pages = [x.round().long() for x in pages]
        return pages + scales

    def rows(name, b, lo, hi):  # [hi - lo, Hkv, d]
        at = s["table"][b, lo // page:-(-hi // page)].long()
        x = s[name][at].double()
        if kv != "bf16":
            x = x.reshape(*x.shape[:-1], -1, 32) * torch.exp2(s[name + "s"][at].double() - 127)[..., None]
            x = x.reshape(*x.shape[:-2], d)
        x = x.transpose(1, 2).reshape(-1, Hkv, d)
        return x[lo - lo // page * page:][:hi - lo]

    if case["op"] == "read":
        return tuple(torch.cat([rows(x, b, ctx[b], ctx[b] + n[b]) for b in range(case["B"])]) for x in ("k", "v"))
    outs, lses = [], []
    t = 0
    for b in range(case["B"]):
        for p0 in range(ctx[b], ctx[b] + n[b], 256):
            p1 = min(p0 + 256, ctx[b] + n[b])
            i = torch.arange(p0, p1, device="cuda")[:, None]
            lo = max(0, (p0 // c - 1) * c) if case["ecp"] else max(0, p0 - max(c, case["S"] * case["period"]))
            j = torch.arange(lo, p1, device="cuda")[None]
            gap = i - j
            if case["ecp"]:
                band, skip = (gap >= 0) & (j // c >= i // c - 1), gap < -p1
            else:
                band = (gap >= 0) & (gap <= c)
                skip = (gap > c) & (gap % max(1, case["period"]) == 0) & (gap <= case["S"] * case["period"])
            q = s["q"][t:t + p1 - p0].double().transpose(0, 1).reshape(Hkv, -1, p1 - p0, d)
            K, V = (rows(x, b, lo, p1).transpose(0, 1)[:, None] for x in ("k", "v"))
            w = torch.exp(q @ K.transpose(-1, -2) / math.sqrt(d)).reshape(H, p1 - p0, -1)
            if case["ecp"]:
                w = w * band
            else:
                a = s["alpha"][t:t + p1 - p0].double().T[..., None]
                w = w * (a * band + (1 - a) * skip)
            total = w.sum(-1, keepdim=True)
            outs.append(((w / total).reshape(Hkv, -1, p1 - p0, p1 - lo) @ V).reshape(H, p1 - p0, d).transpose(0, 1))
            lses.append(torch.log(total[..., 0]).T)
            t += p1 - p0
    return torch.cat(outs), torch.cat(lses)
