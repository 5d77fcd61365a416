"""Measured cases of rotary positions and of a speculative serving step over the paged key/value cache.

Operators, each in a plain form (elementary torch operations in 32 bits, in 64 where the angle of a far position or a sum next
to a border needs it, rounded once at the end) and, with ``own`` set, through this package's entry points:

  rotary   queries and keys of a training layer rotated by their positions on the way from the projection's layout
           [B, N, heads, d] to the attention's [B, heads, N, d], or their gradients rotated back the other way
  append   new tokens of serving sequences: queries and keys rotated, keys and values written into their cache pages
  tree     pi-Attention / ECP attention of a tree of drafted tokens per sequence over the paged cache: node j of sequence b
           lies in cache row ctx[b] + j, its position is ctx[b] plus its depth, and of the tree it attends its ancestors only
  verify   the drafted tokens checked against the target's probabilities with given random numbers: the accepted path
           and the next token of every sequence
  keep     the accepted path's cache rows moved together, in all layers

Rotary: rot <= d, pairs (t, rot / 2 + t) or, interleaved, (2t, 2t + 1); the pair's angle is position * freq[t].
Pages, tables, offsets and 8-bit rows are those of the paged cache: position p of sequence b lies in row p % page of page
table[b, p // page], pages are [pages, Hkv, page, d], an 8-bit row keeps codes and, per block of 32, a power of two as scale.
A tree's parents are node numbers of the same sequence, below the node's own; -1: the last cached token.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases

def listed():
    def rotary(name, **kw):
        return {"name": name, "op": "rotary", "back": False, "dtype": "bf16", "rot": kw["d"], "inter": False, "scaling": "none",
                "start": 0, "packed": False, **kw}

    def append(name, **kw):
        return {"name": name, "op": "append", "rot": kw["d"], "inter": False, "scaling": "none", "tree": False, "ragged": True, **kw}

    def tree(name, **kw):
        return {"name": name, "op": "tree", "k_local": 256, "period": 1024, "S": 4, "ecp": False, "roots": 1, "ragged": True, **kw}

    return [
        # a language-model layer's queries and keys before the training forward, packed documents: positions start again
        rotary("rotary-train-lm", B=4, N=4096, H=12, Hkv=12, d=64, packed=True, shape=1),
        # the long-context layer's gradients on their way back: half of each head rotated, scaled for the long context
        rotary("rotary-back-long", B=1, N=65536, H=16, Hkv=4, d=128, rot=64, inter=True, scaling="yarn", back=True, shape=2),
        # one new token of 64 sequences far into their contexts: latency
        append("append-token-bf16", kv="bf16", B=64, n=1, ctx=130000, H=16, Hkv=4, d=128, page=64, scaling="yarn", shape=3),
        # a long prompt's chunk into an 8-bit cache, and its rows read back
        append("append-prompt-int8", kv="int8", B=1, n=32768, ctx=16384, H=16, Hkv=4, d=128, page=64, ragged=False, shape=4),
        # one user's drafted tree at 64k: latency
        tree("tree-one-e4m3", kv="e4m3", B=1, n=26, ctx=65535, H=16, Hkv=4, d=128, page=64, ragged=False, shape=5),
        # a batch of large trees on the long-context layer
        tree("tree-batch-bf16", kv="bf16", B=48, n=64, ctx=32000, H=16, Hkv=4, d=128, page=64, shape=6),
        # the language-model layer: small pages, a short band, every query head with its own cache head
        tree("tree-lm-int8", kv="int8", B=16, n=32, ctx=4000, H=12, Hkv=12, d=64, page=16, k_local=128, period=256, S=1, shape=7),
        # one user's chain of five drafted tokens: latency
        {"name": "verify-chain", "op": "verify", "B": 1, "n": 6, "V": 32000, "fan": 1, "depth": 6, "drawn": True, "noise": 1.0,
         "ragged": False, "shape": 8},
        # trees of independently drawn tokens, a large vocabulary of odd size: rejections need whole rows
        {"name": "verify-batch", "op": "verify", "B": 32, "n": 32, "V": 128001, "fan": 3, "depth": 6, "drawn": True, "noise": 1.5,
         "ragged": True, "shape": 9},
        # trees of the draft's likeliest tokens
        {"name": "verify-chosen", "op": "verify", "B": 16, "n": 64, "V": 50257, "fan": 4, "depth": 6, "drawn": False, "noise": 1.0,
         "ragged": True, "shape": 10},
        # one user's accepted path in one layer: latency
        {"name": "keep-one-bf16", "op": "keep", "kv": "bf16", "layers": 1, "B": 1, "n": 26, "ctx": 65535, "most": 6, "Hkv": 4, "d": 128,
         "page": 64, "ragged": False, "shape": 11},
        # a batch's paths in all layers of a model, 8-bit cache
        {"name": "keep-batch-int8", "op": "keep", "kv": "int8", "layers": 32, "B": 64, "n": 64, "ctx": 4000, "most": 8, "Hkv": 4, "d": 128,
         "page": 64, "ragged": True, "shape": 12},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "tree", "tree", "verify", "keep"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12, 16] if d == 64 else [1, 2, 4, 8])
    H = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if Hkv * g <= 16])
    c = {"op": op, "shape": rng.randrange(1 << 30)}
    if op in ("rotary", "append"):
        c.update(H=H, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4, 16 * rng.randint(1, d // 16)]), inter=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
    if op == "rotary":
        n = _spread(rng, 3, 24000)
        return {**c, "back": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "B": rng.randint(1, max(1, min(16, 24000 // n))),
                "N": n, "start": _spread(rng, 1, 1 << 20) - 1, "packed": rng.random() < 0.5}
    c.update(ragged=rng.random() < 0.7, ctx=_spread(rng, 1, 16384))
    if op == "verify":
        B, n = _spread(rng, 1, 32), _spread(rng, 1, 64)
        V = _spread(rng, 500, 160000)
        return {**c, "B": max(1, min(B, (64 << 20) // (n * V))), "n": n, "V": V, "fan": rng.randint(1, 5), "depth": rng.randint(2, 8),
                "drawn": rng.random() < 0.6, "noise": rng.choice([0.3, 1.0, 2.0])}
    c.update(kv=rng.choice(["bf16", "e4m3", "int8"]), Hkv=Hkv, d=d, page=rng.choice([16, 32, 64, 128, 256]))
    if op == "append":
        n = _spread(rng, 1, 16384)
        return {**c, "B": rng.randint(1, max(1, min(64, 20000 // n))), "n": n, "tree": n <= 128 and rng.random() < 0.5}
    if op == "tree":
        ecp = rng.random() < 0.25
        n = _spread(rng, 1, 160)
        return {**c, "B": rng.randint(1, max(1, min(48, 2400 // n))), "n": n, "H": H, "ecp": ecp, "roots": rng.choice([1, 1, 3]),
                "k_local": rng.choice([96, 128, 200, 256]) if ecp else _spread(rng, 8, 512),
                "period": 0 if ecp else _spread(rng, 32, 2048), "S": 0 if ecp else rng.randint(0, 5)}
    n = _spread(rng, 1, 128)
    return {**c, "B": _spread(rng, 1, 64), "n": n, "layers": _spread(rng, 1, 32), "most": rng.randint(1, min(n, 12))}


def _lengths(case):
    """Per sequence: rows in the cache before the call, and new rows."""
    B, n, ctx = case["B"], case["n"], case.get("ctx", 0)
    if not case["ragged"]:
        return [ctx] * B, [n] * B
    rng = random.Random(case["shape"])
    return [rng.randint(0, ctx) for _ in range(B)], [rng.randint(1, n) for _ in range(B)]


def _trees(case, n, seed, fan=4, depth=8, roots=1):
    """Parents of every sequence's nodes: early nodes have more children, none more than `fan`, and no path is longer than
    `depth`; a node that has no place any more starts a tree of its own."""
    rng, trees = random.Random(seed), []
    for m in n:
        par, deep, kids = [-1], [1], [0]
        for j in range(1, m):
            if j < roots:
                p = -1
            else:
                free = [x for x in range(j) if kids[x] < fan and deep[x] < depth] or [-1]
                p = free[min(int(len(free) * rng.random() ** 1.5), len(free) - 1)]
                if p >= 0:
                    kids[p] += 1
            par.append(p)
            deep.append(1 if p < 0 else deep[p] + 1)
            kids.append(0)
        trees.append(par)
    return trees


# ------------------------------------------------------------------ inputs

def _rope_setting(case):
    """Base, factor and original length of a case's frequencies."""
    return {"none": (10000.0, 1.0, 0), "linear": (10000.0, 4.0, 0), "ntk": (10000.0, 8.0, 0), "yarn": (500000.0, 16.0, 8192)}[case["scaling"]]


def _frequencies(case, device):
    """freq [rot / 2] in 64 bits, and the factor that the rotated elements are multiplied by."""
    base, factor, original = _rope_setting(case)
    rot, kind = case["rot"], case["scaling"]
    t = torch.arange(rot // 2, dtype=torch.float64, device=device)
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = torch.exp(t * (-2.0 / rot * math.log(base)))
    if kind == "linear":
        f = f / factor
    if kind != "yarn":
        return f, 1.0
    keep = torch.clamp((original * f / (2 * math.pi) - 1) / (32 - 1), 0, 1)  # turns over the original length: from 1 to 32
    return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1


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

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    s = dict(case)
    if "rot" in case:
        s["freq"], s["mul"] = _frequencies(case, dev)
    if case["op"] == "rotary":
        B, N, H, Hkv, d = (case[x] for x in ("B", "N", "H", "Hkv", "d"))
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        if case["packed"]:  # several documents in a row of the batch
            rng, pos = random.Random(case["shape"]), torch.empty(B, N, dtype=torch.int32)
            for b in range(B):
                at = 0
                while at < N:
                    m = min(N - at, rng.randint(1, N))
                    pos[b, at:at + m] = torch.arange(m, dtype=torch.int32) + case["start"]
                    at += m
            s["pos"] = pos.to(dev)
        else:
            s["pos"] = None
        if case["back"]:  # from the attention's backward; dv lies in the projection's gradient already
            s["dq"], s["dk"] = randn(B, H, N, d).to(dt), randn(B, Hkv, N, d).to(dt)
            s["dqkv"] = randn(B, N, H + 2 * Hkv, d).to(dt)
        else:
            s["qkv"] = randn(B, N, H + 2 * Hkv, d).to(dt)
        return s

    ctx, n = _lengths(case)
    B, T = case["B"], sum(n)
    s["T"] = T
    s["cu"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], device=dev, dtype=torch.int32)
    s["ctx"] = torch.tensor(ctx, device=dev, dtype=torch.int32)
    if case["op"] == "verify":
        trees = _trees(case, n, case["shape"], case["fan"], case["depth"])
        V = case["V"]
        s["parent"] = torch.tensor(sum(trees, []), device=dev, dtype=torch.int32)
        draft = torch.empty(T, V, device=dev)
        target = torch.empty(T, V, device=dev)
        for t in range(0, T, 256):
            x = 2.5 * randn(min(256, T - t), V)
            draft[t:t + 256] = torch.softmax(x, -1)
            target[t:t + 256] = torch.softmax(x + case["noise"] * randn(*x.shape), -1)
        up = (s["parent"] + torch.repeat_interleave(s["cu"][:-1], torch.tensor(n, device=dev))).clamp(min=0).long()
        tokens = torch.empty(T, device=dev, dtype=torch.int32)
        if case["drawn"]:  # from the draft's probabilities, each on its own
            for t in range(0, T, 256):
                q = draft[up[t:t + 256]]
                tokens[t:t + 256] = (q / torch.empty_like(q).exponential_(generator=g)).argmax(-1)
        else:  # the likeliest ones in order
            best = torch.cat([draft[t:t + 256].topk(case["fan"] + 1, -1).indices for t in range(0, T, 256)])
            rank, kids = [], {}
            for b, par in enumerate(trees):
                for p in par:
                    kids[b, p] = kids.get((b, p), -1) + 1
                    rank.append(min(kids[b, p], case["fan"]))
            tokens[:] = best[up, torch.tensor(rank, device=dev)]
        s["target"], s["draft"], s["tokens"] = target, draft if case["drawn"] else None, tokens
        s["u"] = torch.rand(T, generator=g, device=dev)
        s["u_next"] = torch.rand(B, generator=g, device=dev)
        return s

    Hkv, d, page, kv = (case[x] for x in ("Hkv", "d", "page", "kv"))
    used = [-(-(c + m) // page) for c, m in zip(ctx, n)]
    pages, width = sum(used) + 3, max(used) + 1
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
    table = torch.full((B, width), -1, device=dev, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    layers = case.get("layers", 1)

    def pool():
        if case["op"] == "keep":  # rows are moved as they are
            k = torch.randint(0, 127, (layers, pages, Hkv, page, 2 * d if kv == "bf16" else d), generator=g, device=dev, dtype=torch.int8)
            if kv == "bf16":
                return (k.view(torch.int16) & 0x3FFF).view(torch.bfloat16), None
            return (k if kv == "int8" else k.view(torch.float8_e4m3fn),
                    torch.randint(100, 140, (layers, pages, Hkv, page, d // 32), generator=g, device=dev, dtype=torch.uint8))
        x = randn(pages, Hkv, page, d)
        x[..., 5::48] *= 6.0  # the few large channels that keys have
        return (x.to(torch.bfloat16), None) if kv == "bf16" else _quantise(x, kv)

    # only the pages that a call can reach need contents of their own: a long context's pages repeat one another
    if case["op"] == "keep":
        first = [c // page for c in ctx]
        pages = sum(u - f for u, f in zip(used, first)) + 3
        order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
        at = 0
        for b, (u, f) in enumerate(zip(used, first)):
            table[b, :f] = -1  # not touched
            table[b, f:u] = order[at:at + u - f]
            at += u - f
    s["table"] = table
    s["k"], s["ks"] = pool()
    s["v"], s["vs"] = pool()
    if case["op"] == "keep":
        rng, path, count = random.Random(case["shape"] + 1), [], []
        for m in n:
            c = rng.randint(1, min(m, case["most"]))
            keep = [0] + sorted(rng.sample(range(1, m), c - 1))
            path += keep + [-1] * (m - c)
            count.append(c)
        s["path"], s["count"] = (torch.tensor(x, device=dev, dtype=torch.int32) for x in (path, count))
        return s
    s["parent"] = None
    if case["op"] == "tree" or case["tree"]:
        trees = _trees(case, n, case["shape"], roots=case.get("roots", 1))
        s["parent"] = torch.tensor(sum(trees, []), device=dev, dtype=torch.int32)
    # the projection's output: queries, keys and values of a token next to one another
    qkv = randn(T, case["H"] + 2 * Hkv, d).to(torch.bfloat16)
    s["q"], s["k_new"], s["v_new"] = qkv[:, :case["H"]], qkv[:, case["H"]:case["H"] + Hkv], qkv[:, case["H"] + Hkv:]
    if case["op"] == "tree":
        s["alpha"] = None if case["ecp"] else torch.sigmoid(1.5 * randn(T, case["H"]))
    return s


# ------------------------------------------------------------------ plain form

def _tokens(s):
    """Sequence and place of every packed token."""
    t = torch.arange(s["T"], device=s["cu"].device)
    seq = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    return seq, t - s["cu"][seq]


def _ancestors(s, most):
    """up [T, most']: a node's 0th, 1st, ... ancestor as a packed index, -1 past the root; depth [T]."""
    seq, _ = _tokens(s)
    T = s["T"]
    step = torch.where(s["parent"] >= 0, s["parent"] + s["cu"][seq], -1).long()
    step = torch.cat([step, step.new_full((1,), -1)])  # the last entry: past the root
    up = torch.arange(T + 1, device=step.device)[:, None]
    up[T] = -1
    while up.shape[1] < most:  # ancestors 0 .. k - 1 and the step of k: twice as many
        up = torch.cat([up, up[step]], 1)
        step = step[step]
    up = up[:T]
    return up, (up >= 0).sum(1) - 1


def _rotate(x, pos, s):
    """x [..., d] in 32 bits rotated by pos (of x's leading shape, broadcast)."""
    rot = s["rot"]
    angle = torch.remainder(pos[..., None].double() * s["freq"], 2 * math.pi)
    c, w = (torch.cos(angle) * s["mul"]).float(), (torch.sin(angle) * s["mul"]).float()
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    y0, y1 = a * c - b * w, a * w + b * c
    y = torch.stack([y0, y1], -1).flatten(-2) if s["inter"] else torch.cat([y0, y1], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rotary(s):
    N, dev = s["N"], s["freq"].device
    pos = s["pos"] if s["pos"] is not None else (torch.arange(N, device=dev) + s["start"])[None]
    H, Hkv = s["H"], s["Hkv"]
    if s["back"]:
        for x, lo, hi in ((s["dq"], 0, H), (s["dk"], H, H + Hkv)):
            s["dqkv"][:, :, lo:hi] = _rotate(x, -pos[:, None], s).transpose(1, 2).to(x.dtype)
        return s["dqkv"]
    return tuple(_rotate(s["qkv"][:, :, lo:hi], pos[:, :, None], s).transpose(1, 2).to(s["qkv"].dtype).contiguous()
                 for lo, hi in ((0, H), (H, H + Hkv)))


def _rows(s, pages, scales, seq, pos):
    """Cache rows at positions pos of sequences seq, in 32 bits: [..., Hkv, d]."""
    at = s["table"][seq, pos // s["page"]].long()
    x = pages[at, :, pos % s["page"]].float()
    if scales is None:
        return x
    return (x.unflatten(-1, (-1, 32)) * _scale_of(scales[at, :, pos % s["page"]]).unsqueeze(-1)).flatten(-2)


def _plain_append(s):
    seq, place = _tokens(s)
    deep = _ancestors(s, s["n"])[1] if s["parent"] is not None else place
    pos = (s["ctx"][seq] + deep)[:, None]
    q, k = _rotate(s["q"], pos, s).to(torch.bfloat16), _rotate(s["k_new"], pos, s)
    line = s["ctx"][seq] + place
    at, row = s["table"][seq, line // s["page"]].long(), line % s["page"]
    if s["kv"] == "bf16":
        s["k"][at, :, row] = k.to(torch.bfloat16)
        s["v"][at, :, row] = s["v_new"]
        return q, s["k"], s["v"]
    s["k"][at, :, row], s["ks"][at, :, row] = _quantise(k, s["kv"])
    s["v"][at, :, row], s["vs"][at, :, row] = _quantise(s["v_new"], s["kv"])
    return (q,) + tuple(_rows(s, s[x], s[y], seq, line).to(torch.bfloat16) for x, y in (("k", "ks"), ("v", "vs")))


def _plain_tree(s):
    T, H, Hkv, d, c = s["T"], s["H"], s["Hkv"], s["d"], s["k_local"]
    seq, _ = _tokens(s)
    dev = seq.device
    up, deep = _ancestors(s, s["n"])
    ctx = s["ctx"][seq].long()[:, None]
    p = ctx + deep[:, None]
    if s["ecp"]:  # the position's own half-segment and the one before it
        keys = torch.clamp((p // c - 1) * c, min=0) + torch.arange(2 * c, device=dev)
        band = keys <= p
        skip = torch.zeros_like(band)
    else:  # the band, then the skips that lie outside it
        m = torch.arange(1, s["S"] + 1, device=dev) * s["period"]
        keys = torch.cat([p - torch.arange(c + 1, device=dev), p - m[m > c]], 1)
        is_skip = torch.arange(keys.shape[1], device=dev) > c
        band, skip = (keys >= 0) & ~is_skip, (keys >= 0) & is_skip
    # a position of the tree is the ancestor at its depth
    anc = up.gather(1, torch.clamp(p - keys, min=0, max=up.shape[1] - 1))
    line = torch.where(keys >= ctx, ctx + anc - s["cu"][seq].long()[:, None], keys)
    at = torch.where(band | skip, line, torch.zeros_like(line))
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


def _plain_verify(s):
    T, B, V = s["T"], s["B"], s["V"]
    seq, place = _tokens(s)
    cu = s["cu"].long()
    up = torch.where(s["parent"] >= 0, s["parent"] + cu[seq], -1)
    t = torch.arange(T, device=up.device)
    rank = ((up[:, None] == up[None]) & (t[None] < t[:, None])).sum(1)  # among the children of its parent
    kids = up.new_full((T + 1, s["fan"]), -1)
    kids[torch.where(up >= 0, up, T), rank.clamp(max=s["fan"] - 1)] = t
    kids[T] = -1
    cur, count = cu[:-1].clone(), torch.ones(B, dtype=torch.int32, device=up.device)
    path = torch.full((T + 1,), -1, dtype=torch.int32, device=up.device)
    path[cur] = 0
    for _ in range(s["depth"]):  # one step of every sequence's walk; the last one ends where all have stopped
        p = s["target"][cur].double()
        q = s["draft"][cur].double() if s["draft"] is not None else None
        a, mass, w = p.new_zeros(B, 1), p.new_ones(B, 1), p
        nxt = torch.full_like(cur, -1)
        for r in range(s["fan"]):
            c = kids[cur, r]
            live = ((c >= 0) & (nxt < 0))[:, None]
            v = s["tokens"][c.clamp(min=0)].long()[:, None]
            u = s["u"][c.clamp(min=0)].double()[:, None]
            wv = w.gather(1, v)
            ok = live & (u * mass * (q.gather(1, v) if q is not None else 1.0) < wv)
            nxt = torch.where(ok[:, 0], c, nxt)
            no = live & ~ok
            if q is not None:
                a = torch.where(no, a + mass, a)
                w = torch.clamp(p - a * q, min=0)
                mass = torch.where(no, w.sum(1, keepdim=True), mass)
            else:
                mass = torch.where(no, mass - wv, mass)
                w = w.scatter(1, v, torch.where(no, torch.zeros_like(wv), wv))
        go = nxt >= 0
        path[torch.where(go, cu[:-1] + count, T)] = (nxt - cu[:-1]).to(torch.int32)
        count = count + go
        cur = torch.where(go, nxt, cur)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    upto = torch.cumsum(w, 1)
    token = (upto <= s["u_next"].double()[:, None] * upto[:, -1:]).sum(1)
    last = V - 1 - (w.flip(1) > 0).to(torch.uint8).argmax(1)
    return path[:T], count.to(torch.int32), torch.minimum(token, last).to(torch.int32)


def _plain_keep(s):
    seq, place = _tokens(s)
    go = (place < s["count"][seq])[None, :, None]
    to = (s["ctx"][seq] + place).long()
    frm = (s["ctx"][seq] + torch.clamp(s["path"], min=0)).long()
    at = [s["table"][seq, x // s["page"]].long() for x in (to, frm)]
    pools = [s[x] for x in ("k", "v", "ks", "vs") if s[x] is not None]
    moved = [x.view(torch.uint8)[:, at[1], :, frm % s["page"]] for x in pools]  # [T, layers, Hkv, bytes]
    stay = [x.view(torch.uint8)[:, at[0], :, to % s["page"]] for x in pools]
    for x, y, z in zip(pools, moved, stay):
        x.view(torch.uint8)[:, at[0], :, to % s["page"]] = torch.where(go.transpose(0, 1)[..., None], y, z)
    return pools


def _handles(s, pa):
    """What a program keeps: the layers' pages, the frequencies."""
    if "rot" in s and "rope" not in s:
        base, factor, original = _rope_setting(s)
        s["rope"] = pa.Rotary(s["rot"], base, interleaved=s["inter"], scaling=s["scaling"], factor=factor, original=original)
    if "table" in s and "cache" not in s:
        if s["op"] == "keep":
            s["cache"] = [pa.PagedCache(*(None if s[x] is None else s[x][i] for x in ("k", "v", "ks", "vs"))) for i in range(s["layers"])]
            s["cache"] = pa.CacheLayers(s["cache"])
        else:
            s["cache"] = pa.PagedCache(s["k"], s["v"], s["ks"], s["vs"])


def run(state):
    s = state
    if not own:
        return {"rotary": _plain_rotary, "append": _plain_append, "tree": _plain_tree, "verify": _plain_verify,
                "keep": _plain_keep}[s["op"]](s)
    import structured_sparse_long_gb300 as pa
    _handles(s, pa)
    if s["op"] == "rotary":
        H, Hkv = s["H"], s["Hkv"]
        if s["back"]:
            g = s["dqkv"].transpose(1, 2)
            pa.rotary_bwd(s["dq"], s["dk"], s["rope"], s["start"], s["pos"], g[:, :H], g[:, H:H + Hkv])
            return s["dqkv"]
        x = s["qkv"].transpose(1, 2)
        return pa.rotary(x[:, :H], x[:, H:H + Hkv], s["rope"], s["start"], s["pos"])
    if s["op"] == "append":
        q = pa.rotary_append(s["q"], s["k_new"], s["v_new"], s["rope"], s["cache"], s["table"], s["cu"], s["ctx"], s["parent"])
        if s["kv"] == "bf16":
            return q, s["k"], s["v"]
        return (q, *pa.cache_read(s["cache"], s["table"], s["cu"], s["ctx"], s["T"]))
    if s["op"] == "tree":
        return pa.extend_tree(s["q"], s["cache"], s["table"], s["cu"], s["ctx"], s["parent"], s["alpha"], s["k_local"], s["period"],
                              s["S"], pa.MODE_ECP if s["ecp"] else pa.MODE_PI)
    if s["op"] == "verify":
        return pa.verify_tree(s["target"], s["draft"], s["tokens"], s["cu"], s["parent"], s["u"], s["u_next"])
    pa.cache_keep(s["cache"], s["table"], s["cu"], s["ctx"], s["path"], s["count"])
    return [s[x] for x in ("k", "v", "ks", "vs") if s[x] is not None]


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    return 2 * case["d"] if case["kv"] == "bf16" else case["d"] + case["d"] // 32


def _tree_work(case, ctx, par):
    """Attended (node, key) pairs, and distinct cache rows, of one sequence."""
    c, deep = case["k_local"], []
    for p in par:
        deep.append(deep[p] + 1 if p >= 0 else 0)
    pairs, far = 0, set()
    lowest, top = ctx, ctx + max(deep)
    for g in deep:
        pos = ctx + g
        lo = max(0, (pos // c - 1) * c) if case["ecp"] else max(0, pos - c)
        ms = [] if case["ecp"] else [m * case["period"] for m in range(1, case["S"] + 1) if c < m * case["period"] <= pos]
        pairs += pos - lo + 1 + len(ms)
        lowest = min(lowest, lo)
        far.update(pos - m for m in ms if pos - m < ctx)
    return pairs, ctx - lowest + len(par) + sum(x < lowest for x in far)


def work(case):
    if case["op"] == "rotary":
        size = 4 if case["dtype"] == "fp32" else 2
        rows = case["B"] * case["N"] * (case["H"] + case["Hkv"])
        return {"bytes": 2 * rows * case["d"] * size + (4 * case["B"] * case["N"] if case["packed"] else 0), "flops": 0}
    ctx, n = _lengths(case)
    T = sum(n)
    if case["op"] == "append":
        row = _row_bytes(case)
        back = 0 if case["kv"] == "bf16" else 2 * T * case["Hkv"] * (row + 2 * case["d"])  # the rows read back
        return {"bytes": T * case["d"] * 4 * case["H"] + 2 * T * case["Hkv"] * (2 * case["d"] + row) + back, "flops": 0}
    if case["op"] == "tree":
        trees = _trees(case, n, case["shape"], roots=case["roots"])
        pairs, keys = (sum(x) for x in zip(*(_tree_work(case, c, p) for c, p in zip(ctx, trees))))
        H, Hkv, d = case["H"], case["Hkv"], case["d"]
        return {"bytes": T * (H * (4 * d + 4 + (0 if case["ecp"] else 4)) + 4) + 2 * keys * Hkv * _row_bytes(case), "flops": 4 * d * H * pairs}
    if case["op"] == "verify":  # the last node's row at least
        return {"bytes": 4 * case["B"] * case["V"] + 20 * T + 12 * case["B"], "flops": 0}
    rng, moved = random.Random(case["shape"] + 1), 0
    for m in n:
        c = rng.randint(1, min(m, case["most"]))
        moved += sum(x != j for j, x in enumerate([0] + sorted(rng.sample(range(1, m), c - 1))))
    return {"bytes": 4 * moved * case["layers"] * case["Hkv"] * _row_bytes(case) + 4 * (T + 4 * case["B"]), "flops": 0}


# ------------------------------------------------------------------ 64 bits

def _exact_block(x, kv):
    """Codes (as values) times scales of x [..., d], in 64 bits."""
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
    return (codes * power(e)[..., None]).reshape(x.shape)


def _exact_angles(case):
    """[rot / 2] turns per position and the factor, from Python's own arithmetic."""
    base, factor, original = _rope_setting(case)
    rot, out = case["rot"], []
    for t in range(rot // 2):
        f = base ** (-2 * t / rot)
        if case["scaling"] == "linear":
            f /= factor
        elif case["scaling"] == "ntk":
            f = (base * factor ** (rot / (rot - 2))) ** (-2 * t / rot)
        elif case["scaling"] == "yarn":
            turns = original * f / (2 * math.pi)
            part = min(1.0, max(0.0, (turns - 1) / 31))
            f = part * f + (1 - part) * f / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda"), 1 + 0.1 * math.log(factor) if case["scaling"] == "yarn" else 1.0


def _exact_rotate(x, pos, case, sign=1):
    """x [..., d] by pos [...] as a product of complex numbers."""
    f, mul = _exact_angles(case)
    rot, y = case["rot"], x.double().clone()
    turn = torch.polar(torch.full_like(f, mul).expand(*pos.shape, -1).contiguous(), sign * pos[..., None].double() * f)
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
    z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_verify(s, case, n):
    paths, counts, tokens = [], [], []
    par, tok, u = s["parent"].tolist(), s["tokens"].tolist(), s["u"].double().tolist()
    at = 0
    for b, m in enumerate(n):
        x, path = 0, [0]
        while True:
            p = s["target"][at + x].double()
            w, left = p.clone(), 1.0
            took = None
            for c in range(x + 1, m):
                if par[at + c] != x:
                    continue
                v = tok[at + c]
                if case["drawn"]:
                    q = s["draft"][at + x].double()
                    if u[at + c] * float(q[v]) < float(w[v]) / left:
                        took = c
                        break
                    w = torch.clamp(w / left - q, min=0)  # the residual, weighed by `left` from now on
                    left = float(w.sum())
                else:
                    if u[at + c] * left < float(w[v]):
                        took = c
                        break
                    left -= float(w[v])
                    w[v] = 0
            if took is None:
                break
            x = took
            path.append(x)
        if not float(w.sum()) > 0:
            w = p
        upto = torch.cumsum(w, 0)
        tokens.append(min(int(torch.searchsorted(upto, upto[-1:] * s["u_next"][b].double(), right=True)), int(torch.nonzero(w)[-1])))
        paths += path + [-1] * (m - len(path))
        counts.append(len(path))
        at += m
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (paths, counts, tokens))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        B, N, H, Hkv = (case[x] for x in ("B", "N", "H", "Hkv"))
        pos = (torch.arange(N, device="cuda") + case["start"]).expand(B, N) if s["pos"] is None else s["pos"]
        if case["back"]:
            out = s["dqkv"].double()
            for b in range(B):
                for h in range(H + Hkv):
                    x = s["dq"][b, h] if h < H else s["dk"][b, h - H]
                    out[b, :, h] = _exact_rotate(x, pos[b], case, -1)
            return out
        y = torch.stack([torch.stack([_exact_rotate(s["qkv"][b, :, h], pos[b], case) for h in range(H + Hkv)]) for b in range(B)])
        return y[:, :H], y[:, H:]
    ctx, n = _lengths(case)
    if case["op"] == "verify":
        return _exact_verify(s, case, n)
    page, Hkv, d, kv = (case[x] for x in ("page", "Hkv", "d", "kv"))
    tables = s["table"].tolist()
    if case["op"] == "keep":
        pools = [s[x] for x in ("k", "v", "ks", "vs") if s[x] is not None]
        out = [x.clone() for x in pools]
        path, count, at = s["path"].tolist(), s["count"].tolist(), 0
        for b, m in enumerate(n):
            for j in range(count[b]):
                i, t = ctx[b] + path[at + j], ctx[b] + j
                for x, y in zip(out, pools):
                    x[:, tables[b][t // page], :, t % page] = y[:, tables[b][i // page], :, i % page]
            at += m
        return [x.double() if x.dtype.is_floating_point else x for x in out]
    trees = _trees(case, n, case["shape"], roots=case.get("roots", 1)) if s["parent"] is not None else [list(range(-1, m - 1)) for m in n]
    depths = []
    for par in trees:
        deep = []
        for p in par:
            deep.append(deep[p] + 1 if p >= 0 else 0)
        depths.append(deep)
    if case["op"] == "append":
        pos = torch.tensor([c + g for c, deep in zip(ctx, depths) for g in deep], device="cuda")
        q = torch.stack([_exact_rotate(s["q"][:, h], pos, case) for h in range(case["H"])], 1)
        k = torch.stack([_exact_rotate(s["k_new"][:, h], pos, case) for h in range(Hkv)], 1)
        v = s["v_new"].double()
        if kv != "bf16":
            return q, _exact_block(k, kv), _exact_block(v, kv)
        pages = [s["k"].double(), s["v"].double()]
        t = 0
        for b, m in enumerate(n):
            p, end = ctx[b], ctx[b] + m
            while p < end:
                x = min(page - p % page, end - p)
                for y, z in zip(pages, (k, v)):
                    y[tables[b][p // page], :, p % page:p % page + x] = z[t:t + x].transpose(0, 1)
                p, t = p + x, t + x
        return q, *pages

    def rows(name, b, lo, hi):  # [hi - lo, Hkv, d]
        at = s["table"][b, lo // page:-(-hi // page)].long()
        x = s[name][at].double()
        if kv != "bf16":
            x = x.reshape(*x.shape[:-1], -1, 32) * torch.exp2(s[name + "s"][at].double() - 127)[..., None]
            x = x.reshape(*x.shape[:-2], d)
        x = x.transpose(1, 2).reshape(-1, Hkv, d)
        return x[lo - lo // page * page:][:hi - lo]

    H, c, outs, lses, t = case["H"], case["k_local"], [], [], 0
    for b, (par, deep) in enumerate(zip(trees, depths)):
        m, end = len(par), ctx[b] + len(par)
        lo = max(0, (ctx[b] // c - 1) * c) if case["ecp"] else max(0, ctx[b] - max(c, case["S"] * case["period"]))
        # the position that a row holds for a node: its own for the cache, its depth's for the node's line of ancestors
        line = torch.arange(lo, end, device="cuda").expand(m, -1).clone()
        mine = torch.ones(m, end - lo, dtype=torch.bool)
        mine[:, ctx[b] - lo:] = False
        for j in range(m):
            x = j
            while x >= 0:
                mine[j, ctx[b] - lo + x] = True
                x = par[x]
        line[:, ctx[b] - lo:] = ctx[b] + torch.tensor(deep, device="cuda")
        i = ctx[b] + torch.tensor(deep, device="cuda")[:, None]
        gap, mine = i - line, mine.cuda()
        if case["ecp"]:
            band, skip = mine & (line // c >= i // c - 1), torch.zeros_like(mine)
        else:
            band = mine & (gap <= c)
            skip = mine & (gap > c) & (gap % max(1, case["period"]) == 0) & (gap <= case["S"] * case["period"])
        q = s["q"][t:t + m].double().transpose(0, 1).reshape(Hkv, -1, m, d)
        K, V = (rows(x, b, lo, end).transpose(0, 1)[:, None] for x in ("k", "v"))
        w = torch.exp(q @ K.transpose(-1, -2) / math.sqrt(d)).reshape(H, m, -1)
        if case["ecp"]:
            w = w * band
        else:
            a = s["alpha"][t:t + m].double().T[..., None]
            w = w * (a * band + (1 - a) * skip)
        total = w.sum(-1, keepdim=True)
        outs.append(((w / total).reshape(Hkv, -1, m, end - lo) @ V).reshape(H, m, d).transpose(0, 1))
        lses.append(torch.log(total[..., 0]).T)
        t += m
    return torch.cat(outs), torch.cat(lses)
