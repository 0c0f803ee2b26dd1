"""Cases that time the operators of the 8-bit block-scaled KV cache: the store that appends
tokens, attention over the cache, attention over blocks that a cheap score selects, and
eviction by accumulated attention weight.

The cache, as the library lays it out: codes [L, 2, B, H, T, d] in 8 bits (int8 or e4m3,
s = 0 keys, s = 1 values), one fp32 scale, a power of two, for every block of tb tokens of
every head [L, 2, B, H, T / tb], for the keys of every block the least and the largest code of
every channel [L, B, H, T / tb, 2, d] (int8), and the attention weight that every block has
drawn so far [L, B, H, T / tb] (fp32).  A code c of a block with scale s stands for s c.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) where
`own` is false, and through the library's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

TOP = {"int8": 127.0, "e4m3": 448.0}   # the largest code


def listed():
    return [
        # one decode step's new keys and values of all layers of a 32-layer model, 8 sequences of
        # ragged lengths, one of them a vacant slot: the smallest store, run once a token
        dict(name="append_step", op="append", code="int8", tb=16, L=32, B=8, H=8, T=1024, d=128, n=1, ragged=False, layer0=0, nl=32),
        # the keys and values of a 4096-token prompt go to the cache at once
        dict(name="append_prompt", op="append", code="e4m3", tb=64, L=32, B=1, H=8, T=4224, d=128, n=4096, ragged=False, layer0=0, nl=32),
        # a ragged batch of prompt pieces of one layer, odd lengths, starts inside blocks
        dict(name="append_pieces", op="append", code="int8", tb=32, L=2, B=12, H=4, T=2048, d=64, n=517, ragged=True, layer0=1, nl=1),
        # one sequence, one layer, a short history: latency
        dict(name="attend_one", op="attend", code="int8", tb=16, L=2, B=1, H=2, T=1024, d=64, Hq=8, nq=1, max=777, layer0=1, nl=1, mass=False),
        # one decode step of a 32-layer cache of 4096 tokens, 32 query heads over 8 KV heads
        dict(name="attend_32layers", op="attend", code="int8", tb=16, L=32, B=1, H=8, T=4096, d=128, Hq=32, nq=1, max=4096, layer0=0, nl=32, mass=False),
        # one layer of a serving batch: 64 sequences of ragged lengths
        dict(name="attend_batch", op="attend", code="e4m3", tb=64, L=1, B=64, H=8, T=8192, d=128, Hq=32, nq=1, max=8192, layer0=0, nl=1, mass=False),
        # four draft tokens verified at once, the blocks' attention weight kept for eviction
        dict(name="attend_verify_mass", op="attend", code="int8", tb=32, L=1, B=12, H=4, T=16384, d=128, Hq=32, nq=4, max=16001, layer0=0, nl=1, mass=True),
        # one long sequence, one layer: 64 of 2048 blocks are read
        dict(name="sparse_one", op="sparse", code="int8", tb=16, L=1, B=1, H=8, T=32768, d=128, Hq=32, nq=1, max=32768, layer0=0, nl=1, k=64, sink=1, recent=2),
        # one layer of a serving batch with long histories: 128 of up to 1024 blocks
        dict(name="sparse_batch", op="sparse", code="e4m3", tb=32, L=1, B=32, H=8, T=32768, d=128, Hq=32, nq=1, max=32768, layer0=0, nl=1, k=128, sink=1, recent=2),
        # draft tokens with lists of their own, small heads, an odd number of blocks
        dict(name="sparse_drafts", op="sparse", code="int8", tb=64, L=2, B=6, H=4, T=20480, d=64, Hq=16, nq=3, max=19999, layer0=0, nl=2, k=33, sink=2, recent=3),
        # one layer of a small batch is cut from up to 4096 tokens to 1024
        dict(name="evict_layer", op="evict", code="int8", tb=16, L=1, B=4, H=8, T=4096, d=128, keep=64, sink=4, recent=8, layer0=0, nl=1),
        # a whole 32-layer cache is cut by half
        dict(name="evict_32layers", op="evict", code="e4m3", tb=32, L=32, B=2, H=8, T=4096, d=128, keep=64, sink=1, recent=4, layer0=0, nl=32),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = dict(op=rng.choice(["append", "attend", "sparse", "evict"]), code=rng.choice(["int8", "e4m3"]), tb=rng.choice([16, 32, 64]),
                 d=rng.choice([64, 128]), H=rng.choice([1, 2, 4, 8]), B=log(1, 48))
        c["L"] = log(1, 32) if c["op"] in ("append", "evict") or c["B"] < 4 else 1
        c["layer0"] = rng.randrange(c["L"])
        c["nl"] = rng.randint(1, c["L"] - c["layer0"])
        if c["op"] == "append":
            c["n"] = log(1, 4096)
            c["ragged"] = rng.random() < 0.5
            c["T"] = 64 * (-(-c["n"] // 64) + 2 + log(1, 16))
        else:
            c["T"] = 64 * log(4, 600)
        if c["op"] in ("attend", "sparse"):
            c["Hq"] = c["H"] * rng.choice([1, 2, 3, 4, 5, 8])
            c["nq"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
            c["max"] = c["T"] - rng.randrange(64)
        if c["op"] == "attend":
            c["mass"] = rng.random() < 0.4
        nb = c["T"] // c["tb"]
        if c["op"] == "sparse":
            c["k"] = max(4, min(nb, log(4, 256)))
            c["sink"], c["recent"] = rng.randint(0, 2), rng.randint(0, 2)
        if c["op"] == "evict":
            c["keep"] = min(nb, log(8, max(9, nb)))
            c["sink"], c["recent"] = rng.randint(0, min(3, c["keep"] // 4)), rng.randint(1, min(5, c["keep"] // 2))
        # no dearer than the largest listed case, neither in its work nor in what it holds
        held = 2 * c["L"] * c["B"] * c["H"] * c["T"] * c["d"]
        w = work(c)
        picked = c["B"] * c["H"] * c["nl"] * c["nq"] * c["k"] * c["tb"] * 2 * c["d"] if c["op"] == "sparse" else 0
        if held <= 1.1e9 and w["bytes"] <= 8e8 and w["flops"] <= 1.6e10 and picked <= 2.7e8:
            return c


# ---- inputs ------------------------------------------------------------------------------


def lengths(case):
    """The sequences' lengths of a case, before the seed puts them in order: from the longest
    down to a quarter of it, and in a batch of eight or more one slot that is vacant."""
    B = case["B"]
    if case["op"] == "append":
        room = case["T"] - case["n"] - 2 * case["tb"]
        v = [int(room * ((0.37 + b * 0.618034) % 1.0)) for b in range(B)]
        if B >= 8:
            v[-1] = 0
        return v
    m = case.get("max", case["T"] - 5)
    v = [max(1, int(m * (1.0 - 0.75 * ((b * 0.618034) % 1.0)))) for b in range(B)]
    if B >= 8:
        v[-1] = 0
    return v


def counts(case):
    """How many of the n new tokens each sequence takes: all of them, or ragged down to none."""
    B, n = case["B"], case["n"]
    if not case["ragged"]:
        return [n] * B
    return [n - int(n * ((b * 0.618034) % 1.0)) if b + 1 < B or B == 1 else 0 for b in range(B)]


def power(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def exponent(amax, code):
    """The least e, -126 or more, with amax <= top 2^e."""
    m, x = torch.frexp(amax)
    e = x - 7 + (m > 254 / 256).int() if code == "int8" else x - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp_min(-126)


def rounded(y, code):
    """fp32 values on the grid of the codes, still fp32."""
    return y.round() if code == "int8" else y.to(torch.float8_e4m3fn).float()


def raw(v, code):
    """Values on the grid as the cache's bytes."""
    return (v.to(torch.int8) if code == "int8" else v.to(torch.float8_e4m3fn)).view(torch.uint8)


def values(codes, code):
    return codes.view(torch.int8 if code == "int8" else torch.float8_e4m3fn).float()


def bound_units(lo, hi, code):
    """int8 bounds of the least and largest code values of a channel: the values themselves, or
    in units of 448 / 127, rounded outwards (e4m3 values are multiples of 2^-9: whole numbers here)."""
    if code == "int8":
        return lo, hi
    lo, hi = (lo * 512).int() * 127, (hi * 512).int() * 127
    unit = 448 * 512
    return torch.div(lo, unit, rounding_mode="floor").float(), -torch.div(-hi, unit, rounding_mode="floor").float()


def make_cache(case, gen):
    """A filled cache.  Channels of keys have gains of their own, two of them far out, and
    values drift along the tokens, as caches of trained models do."""
    L, B, H, T, d, tb, code = (case[k] for k in ("L", "B", "H", "T", "d", "tb", "code"))
    dev = "cuda"
    codes = torch.empty((L, 2, B, H, T, d), dtype=torch.uint8, device=dev)
    scales = torch.empty((L, 2, B, H, T // tb), dtype=torch.float32, device=dev)
    bounds = torch.empty((L, B, H, T // tb, 2, d), dtype=torch.int8, device=dev)
    step = max(1, (1 << 27) // (H * T * d))
    for l in range(L):
        gain = torch.randn((1, H, 1, d), generator=gen, device=dev).mul(0.5).exp()
        gain[..., 3] *= 6
        gain[..., d // 2 + 1] *= 6
        for s in range(2):
            for b in range(0, B, step):
                n = min(step, B - b)
                x = torch.randn((n, H, T, d), generator=gen, device=dev)
                drift = torch.randn((n, H, T // tb, 1, 1), generator=gen, device=dev).mul(0.7).exp()
                x = x * gain if s == 0 else x
                x = (x.view(n, H, T // tb, tb, d) * drift).bfloat16().float()
                e = exponent(x.abs().amax((-1, -2)), code)
                sc = power(e)
                v = rounded(x / sc[..., None, None], code)
                codes[l, s, b:b + n] = raw(v, code).view(n, H, T, d)
                scales[l, s, b:b + n] = sc
                if s == 0:
                    lo, hi = bound_units(v.amin(3), v.amax(3), code)
                    bounds[l, b:b + n, :, :, 0] = lo.to(torch.int8)
                    bounds[l, b:b + n, :, :, 1] = hi.to(torch.int8)
    return codes, scales, bounds


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1009 + 17)
    B, nl, d, H = case["B"], case["nl"], case["d"], case["H"]
    order = torch.from_numpy(np.random.RandomState(seed % (1 << 31)).permutation(B))
    codes, scales, bounds = make_cache(case, gen)
    st = dict(case=dict(case), codes=codes, scales=scales, bounds=bounds, mine={})
    st["lens"] = torch.tensor(lengths(case), dtype=torch.int32)[order].cuda()
    if case["op"] == "append":
        x = torch.randn((nl, 2, B, H, case["n"], d), generator=gen, device="cuda")
        x[:, 0, ..., 3] *= 12
        # later tokens of some heads are larger than what their blocks hold
        x *= torch.randn((nl, 2, B, H, 1, 1), generator=gen, device="cuda").exp()
        st["new"] = x.bfloat16()
        st["counts"] = torch.tensor(counts(case), dtype=torch.int32)[order].cuda() if case["ragged"] else None
    if case["op"] in ("attend", "sparse"):
        q = torch.randn((nl, B, case["Hq"], case["nq"], d), generator=gen, device="cuda")
        st["q"] = (q * torch.randn((nl, B, case["Hq"], 1, 1), generator=gen, device="cuda").mul(0.3).exp()).bfloat16()
        st["out"] = torch.empty(st["q"].shape, dtype=torch.float32, device="cuda")
        if case["op"] == "sparse":
            st["sel"] = torch.empty((nl, B, H, case["nq"], case["k"]), dtype=torch.int32, device="cuda")
    nb = case["T"] // case["tb"]
    st["mass"] = torch.zeros((case["L"], B, H, nb), dtype=torch.float32, device="cuda")
    if case["op"] == "evict":
        st["mass"].exponential_(generator=gen).pow_(3)
        keep, tb = case["keep"], case["tb"]
        T2 = -(-keep * tb // 64) * 64 + 64      # the smaller cache has room for new tokens
        st["to"] = dict(T=T2, codes=torch.zeros((case["L"], 2, B, H, T2, d), dtype=torch.uint8, device="cuda"),
                        scales=torch.zeros((case["L"], 2, B, H, T2 // tb), dtype=torch.float32, device="cuda"),
                        bounds=torch.zeros((case["L"], B, H, T2 // tb, 2, d), dtype=torch.int8, device="cuda"),
                        mass=torch.zeros((case["L"], B, H, T2 // tb), dtype=torch.float32, device="cuda"),
                        lens=torch.zeros((B,), dtype=torch.int32, device="cuda"),
                        kept=torch.zeros((nl, B, H, keep), dtype=torch.int32, device="cuda"))
    return st


# ---- plain forms --------------------------------------------------------------------------


def typed(codes, case):
    """The cache's bytes as the numbers they are."""
    return codes.view(torch.int8 if case["code"] == "int8" else torch.float8_e4m3fn)


def append_plain(st):
    c = st["case"]
    code, tb, d, n, nl, l0 = c["code"], c["tb"], c["d"], c["n"], c["nl"], c["layer0"]
    B, H = c["B"], c["H"]
    codes, scales, bounds = st["codes"][l0:l0 + nl], st["scales"][l0:l0 + nl], st["bounds"][l0:l0 + nl]
    pos = st["lens"].long()
    cnt = torch.full_like(pos, n) if st["counts"] is None else st["counts"].long()
    W = (n + tb - 2) // tb + 1                      # blocks that n tokens touch at most
    first = pos // tb
    at = first[:, None] * tb + torch.arange(W * tb, device="cuda")         # [B, W tb] tokens of the cache
    j = at - pos[:, None]                                                   # their place among the new ones
    fresh = ((j >= 0) & (j < cnt[:, None])).view(1, 1, B, 1, W, tb, 1)
    older = (j < 0).view(1, 1, B, 1, W, tb, 1)
    full = (nl, 2, B, H, W * tb, d)
    pick = j.clamp(0, n - 1)[None, None, :, None, :, None].expand(full)
    x = st["new"].gather(4, pick).float().view(nl, 2, B, H, W, tb, d)
    place = at[None, None, :, None, :, None].expand(full)
    was = codes.gather(4, place)
    v = values(was, code).view(nl, 2, B, H, W, tb, d)
    blocks = (first[:, None] + torch.arange(W, device="cuda"))[None, None, :, None].expand(nl, 2, B, H, W)
    s_was = scales.gather(4, blocks)
    some = fresh.any(5)[..., 0]                     # blocks that take a token
    has = older.any(5)[..., 0]                      # blocks that hold older ones
    s = power(exponent(torch.where(fresh, x.abs(), torch.zeros_like(x)).amax((5, 6)), code))
    s = torch.where(has, torch.maximum(s, s_was), s)
    s = torch.where(some, s, s_was)
    grew = has & some & (s > s_was)
    ratio = torch.where(grew, s_was / s, torch.ones_like(s))
    kept = torch.where(grew[..., None, None], rounded(v * ratio[..., None, None], code), v)
    now = torch.where(fresh, rounded(torch.where(fresh, x, torch.zeros_like(x)) / s[..., None, None], code), kept)
    now_raw = torch.where(fresh | (older & grew[..., None, None]), raw(now, code), was.view(now.shape))
    codes.scatter_(4, place, now_raw.view(full))
    scales.scatter_(4, blocks, s)
    # bounds of the keys: of the whole block where it is new or its scale grew, else widened
    f, o, g = fresh[:, 0], older[:, 0], grew[:, 0, ..., None]
    counted = f | (o & g[..., None])
    lo = torch.where(counted, now[:, 0], torch.full_like(now[:, 0], TOP[code])).amin(4)
    hi = torch.where(counted, now[:, 0], torch.full_like(now[:, 0], -TOP[code])).amax(4)
    lo, hi = bound_units(lo, hi, code)
    where = blocks[:, 0, ..., None, None].expand(nl, B, H, W, 2, d)
    b_was = bounds.gather(3, where)
    widen = has[:, 0, ..., None].expand(nl, B, H, W, 1) & ~g
    lo = torch.where(widen, torch.minimum(lo, b_was[..., 0, :].float()), lo)
    hi = torch.where(widen, torch.maximum(hi, b_was[..., 1, :].float()), hi)
    b_now = torch.where(some[:, 0, ..., None, None].expand(where.shape), torch.stack((lo, hi), 4).to(torch.int8), b_was)
    bounds.scatter_(3, where, b_now)
    return {"codes": typed(st["codes"], c), "scales": st["scales"], "bounds": st["bounds"]}


def read_plain(codes, scales, case):
    """The values that codes [..., T, d] stand for."""
    nb, tb, d = scales.shape[-1], case["tb"], case["d"]
    v = values(codes, case["code"])
    return (v.view(v.shape[:-2] + (nb, tb, d)) * scales[..., None, None]).view(v.shape)


def softmax_plain(s, seen):
    """Softmax over the last axis of the scores that are seen; rows that see none are zero."""
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-37)


def last_seen(st):
    """The last token that each query token sees, [B, nq] (negative: none)."""
    nq = st["case"]["nq"]
    return st["lens"].long()[:, None] - nq + torch.arange(nq, device="cuda")


def attend_plain(st):
    c = st["case"]
    nl, l0, B, H, d, nq, T, tb = (c[k] for k in ("nl", "layer0", "B", "H", "d", "nq", "T", "tb"))
    G = c["Hq"] // H
    k = read_plain(st["codes"][l0:l0 + nl, 0], st["scales"][l0:l0 + nl, 0], c)
    v = read_plain(st["codes"][l0:l0 + nl, 1], st["scales"][l0:l0 + nl, 1], c)
    q = st["q"].float().view(nl, B, H, G * nq, d)
    s = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    seen = torch.arange(T, device="cuda") <= last_seen(st)[..., None]              # [B, nq, T]
    p = softmax_plain(s.view(nl, B, H, G, nq, T), seen[None, :, None, None])
    out = torch.matmul(p.view(nl, B, H, G * nq, T), v).view(nl, B, c["Hq"], nq, d)
    if not c["mass"]:
        return {"out": out}
    st["mass"][l0:l0 + nl] = p.sum((3, 4)).view(nl, B, H, T // tb, tb).sum(-1)
    return {"out": out, "mass": st["mass"]}


def select_plain(st):
    c = st["case"]
    nl, l0, B, H, d, nq, T, tb = (c[k] for k in ("nl", "layer0", "B", "H", "d", "nq", "T", "tb"))
    G, NB, k = c["Hq"] // H, T // tb, c["k"]
    q = st["q"].float().view(nl, B, H, G * nq, d)
    unit = power(exponent(q.abs().amax(-1), "int8"))                                # [nl, B, H, G nq]
    q8 = (q / unit[..., None]).round()
    lo = st["bounds"][l0:l0 + nl, :, :, :, 0].float().transpose(-1, -2)
    hi = st["bounds"][l0:l0 + nl, :, :, :, 1].float().transpose(-1, -2)
    # whole numbers below 2^24: exact in any order
    dot = torch.matmul(q8.clamp_min(0), hi) + torch.matmul(q8.clamp_max(0), lo)
    score = dot * unit[..., None] * st["scales"][l0:l0 + nl, 0][:, :, :, None]
    score = score.view(nl, B, H, G, nq, NB).amax(3)
    nb = (torch.div(last_seen(st), tb, rounding_mode="floor") + 1).clamp_min(0)[None, :, None, :, None]
    i = torch.arange(NB, device="cuda")
    score = torch.where((i < c["sink"]) | (i >= nb - c["recent"]), torch.full_like(score, math.inf), score)
    score = torch.where(i < nb, score, torch.full_like(score, -math.inf))
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    best = torch.where(best < nb, best, torch.full_like(best, NB)).sort(-1).values
    return torch.where(best < NB, best, torch.full_like(best, -1)).to(torch.int32)


def sparse_plain(st):
    c = st["case"]
    nl, l0, B, H, d, nq, T, tb, k = (c[n] for n in ("nl", "layer0", "B", "H", "d", "nq", "T", "tb", "k"))
    G, NB = c["Hq"] // H, T // tb
    sel = select_plain(st)                                                           # [nl, B, H, nq, k]
    at = sel.long().clamp_min(0).view(nl, 1, B, H, nq * k).expand(nl, 2, B, H, nq * k)
    codes = st["codes"][l0:l0 + nl].view(nl, 2, B, H, NB, tb * d)
    picked = codes.gather(4, at[..., None].expand(nl, 2, B, H, nq * k, tb * d)).view(nl, 2, B, H, nq * k * tb, d)
    kv = read_plain(picked, st["scales"][l0:l0 + nl].gather(4, at), c).view(nl, 2, B, H, nq, k * tb, d)
    token = (sel.long()[..., None] * tb + torch.arange(tb, device="cuda")).view(nl, B, H, nq, k * tb)
    seen = (token <= last_seen(st)[None, :, None, :, None]) & (sel >= 0).repeat_interleave(tb, -1)
    q = st["q"].float().view(nl, B, H, G, nq, d).transpose(3, 4)                     # [nl, B, H, nq, G, d]
    s = torch.matmul(q, kv[:, 0].transpose(-1, -2)) * (1.0 / math.sqrt(d))
    p = softmax_plain(s, seen[..., None, :])
    out = torch.matmul(p, kv[:, 1]).transpose(3, 4).reshape(nl, B, c["Hq"], nq, d)
    return {"sel": sel, "out": out}


def evict_plain(st):
    c, to = st["case"], st["to"]
    nl, l0, B, H, d, T, tb, keep = (c[k] for k in ("nl", "layer0", "B", "H", "d", "T", "tb", "keep"))
    NB = T // tb
    lens = st["lens"].long()
    nb = torch.div(lens + tb - 1, tb, rounding_mode="floor")[None, :, None, None]
    i = torch.arange(NB, device="cuda")
    w = st["mass"][l0:l0 + nl]
    key = torch.where((i < c["sink"]) | (i >= nb - c["recent"]), torch.full_like(w, math.inf), w)
    key = torch.where(i < nb, key, torch.full_like(key, -math.inf))
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < nb, best, torch.full_like(best, NB)).sort(-1).values      # [nl, B, H, keep]
    there = best < NB
    at = torch.where(there, best, torch.zeros_like(best))
    to["kept"].copy_(torch.where(there, best, torch.full_like(best, -1)))
    n = nb[0, :, 0, 0]
    to["lens"].copy_(torch.where(n > keep, lens - (n - keep) * tb, lens))
    at2, there2 = at[:, None].expand(nl, 2, B, H, keep), there[:, None]
    src = st["codes"][l0:l0 + nl].view(nl, 2, B, H, NB, tb * d).gather(4, at2[..., None].expand(nl, 2, B, H, keep, tb * d))
    dst = to["codes"][l0:l0 + nl].view(nl, 2, B, H, to["T"] // tb, tb * d)[..., :keep, :]
    dst.copy_(torch.where(there2[..., None], src, dst))
    dst = to["scales"][l0:l0 + nl][..., :keep]
    dst.copy_(torch.where(there2, st["scales"][l0:l0 + nl].gather(4, at2), dst))
    src = st["bounds"][l0:l0 + nl].view(nl, B, H, NB, 2 * d).gather(3, at[..., None].expand(nl, B, H, keep, 2 * d))
    dst = to["bounds"][l0:l0 + nl].view(nl, B, H, to["T"] // tb, 2 * d)[..., :keep, :]
    dst.copy_(torch.where(there[..., None], src, dst))
    dst = to["mass"][l0:l0 + nl]
    dst.zero_()
    dst[..., :keep] = torch.where(there, w.gather(3, at), torch.zeros_like(at, dtype=torch.float32))
    return {"kept": to["kept"], "lens": to["lens"], "codes": typed(to["codes"], c), "scales": to["scales"], "bounds": to["bounds"], "mass": to["mass"]}


# ---- the library's calls --------------------------------------------------------------------


def handles(st):
    """What a program makes once: descriptors and workspaces."""
    from quantization_cg_encode_b200 import cg
    c, m = st["case"], st["mine"]
    if not m:
        m["cg"] = cg
        m["kv"] = cg.kv_desc(c["L"], c["B"], c["H"], c["T"], c["d"])
        m["c8"] = cg.cache8_desc(cg.CACHE8_INT8 if c["code"] == "int8" else cg.CACHE8_E4M3, c["tb"])
        if c["op"] in ("attend", "sparse"):
            m["at"] = cg.cache8_attn_desc(c["Hq"], c["max"], q_tokens=c["nq"], layer0=c["layer0"], n_layers=c["nl"], d_head=c["d"],
                                          n_select=c.get("k", 0))
            m["ws"] = torch.empty(cg.cg_cache8_attention_workspace_size(m["kv"], m["c8"], m["at"], c.get("mass", False)),
                                  dtype=torch.uint8, device="cuda")
        if c["op"] == "sparse":
            m["sd"] = cg.cache8_select_desc(c["Hq"], c["max"], c["k"], q_tokens=c["nq"], sink_blocks=c["sink"], recent_blocks=c["recent"],
                                            layer0=c["layer0"], n_layers=c["nl"])
            m["ws2"] = torch.empty(cg.cg_cache8_select_workspace_size(m["kv"], m["c8"], m["sd"]), dtype=torch.uint8, device="cuda")
        if c["op"] == "evict":
            m["ev"] = cg.cache8_evict_desc(c["keep"], sink_blocks=c["sink"], recent_blocks=c["recent"], layer0=c["layer0"], n_layers=c["nl"])
            m["kv2"] = cg.kv_desc(c["L"], c["B"], c["H"], st["to"]["T"], c["d"])
    return m


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return {"append": append_plain, "attend": attend_plain, "sparse": sparse_plain, "evict": evict_plain}[op](st)
    c, m = st["case"], handles(st)
    cg = m["cg"]
    if op == "append":
        cg.cg_cache8_append(m["kv"], m["c8"], c["layer0"], st["new"], st["lens"], st["counts"], st["codes"], st["scales"], st["bounds"])
        return {"codes": typed(st["codes"], c), "scales": st["scales"], "bounds": st["bounds"]}
    if op == "attend":
        cg.cg_cache8_attention(m["kv"], m["c8"], m["at"], st["q"], st["codes"], st["scales"], st["lens"], st["out"], m["ws"],
                               mass=st["mass"] if c["mass"] else None)
        return {"out": st["out"], "mass": st["mass"]} if c["mass"] else {"out": st["out"]}
    if op == "sparse":
        cg.cg_cache8_select(m["kv"], m["c8"], m["sd"], st["q"], st["scales"], st["bounds"], st["lens"], st["sel"], m["ws2"])
        cg.cg_cache8_attention(m["kv"], m["c8"], m["at"], st["q"], st["codes"], st["scales"], st["lens"], st["out"], m["ws"], sel=st["sel"])
        return {"sel": st["sel"], "out": st["out"]}
    to = st["to"]
    cg.cg_cache8_evict(m["kv"], m["c8"], m["ev"], st["lens"], st["codes"], st["scales"], st["bounds"], st["mass"],
                       m["kv2"], to["codes"], to["scales"], to["bounds"], to["mass"], to["lens"], to["kept"])
    return {"kept": to["kept"], "lens": to["lens"], "codes": typed(to["codes"], c), "scales": to["scales"], "bounds": to["bounds"], "mass": to["mass"]}


# ---- what a pass cannot do without ------------------------------------------------------------


def work(case):
    c = case
    d, tb, H, nl = c["d"], c["tb"], c["H"], c["nl"]
    lens = lengths(c)
    if c["op"] == "append":
        tokens = sum(counts(c)) * nl * 2 * H
        blocks = sum(-(-(p % tb + n) // tb) if n else 0 for p, n in zip(lens, counts(c))) * nl * 2 * H
        return {"bytes": tokens * d * 3 + blocks * 4 + blocks // 2 * 2 * d, "flops": tokens * d * 2}
    if c["op"] == "evict":
        kept = sum(min(c["keep"], -(-n // tb)) for n in lens) * nl * H
        return {"bytes": 2 * kept * (2 * tb * d + 8 + 2 * d + 4) + sum(-(-n // tb) for n in lens) * nl * H * 4, "flops": 0}
    rows = c["Hq"] * c["nq"] * nl
    io = c["B"] * rows * d * 6
    if c["op"] == "attend":
        tokens = sum(lens) * nl * H
        return {"bytes": tokens * 2 * d + tokens // tb * 8 + io + (c["L"] * c["B"] * H * (c["T"] // tb) * 4 if c["mass"] else 0),
                "flops": 4 * d * sum(lens) * rows}
    blocks = sum(-(-n // tb) for n in lens) * nl * H
    read = sum(min(c["k"] * tb, n) for n in lens) * nl * H * c["nq"]
    return {"bytes": blocks * (2 * d + 4) + min(read, sum(lens) * nl * H) * 2 * d + io,
            "flops": 2 * 2 * d * blocks * c["nq"] * (c["Hq"] // H) + 4 * d * read * (c["Hq"] // H)}


# ---- the definitions in 64 bits -----------------------------------------------------------------


def _two(e):
    """2^e in fp64 for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _up(y):
    """The least whole e with y <= 2^e, for y > 0."""
    m, x = torch.frexp(y)
    return torch.where(m > 0.5, x, x - 1)


def _numbers(codes, code):
    """fp64 values of the cache's bytes, from the formats' definitions."""
    b = codes.to(torch.int64)
    if code == "int8":
        return torch.where(b > 127, b - 256, b).double()
    sign, ex, man = 1.0 - 2.0 * (b >> 7).double(), (b >> 3) & 15, (b & 7).double()
    return sign * torch.where(ex == 0, man * 2.0 ** -9, (1 + man / 8) * _two(ex - 7))


def _grid(y, code):
    """fp64 numbers to the nearest code, ties to even."""
    if code == "int8":
        return torch.round(y)
    ulp = _two((torch.frexp(y.abs())[1] - 1).clamp_min(-6) - 3)
    return torch.round(y / ulp) * ulp


def _exact_append(st):
    c = st["case"]
    code, tb, top = c["code"], c["tb"], TOP[c["code"]]
    if c["nl"] * c["B"] * c["H"] * c["n"] * c["d"] > 3e7:
        return None
    val = _numbers(st["codes"], code)
    sc = st["scales"].double()
    for b in range(c["B"]):
        pos = int(st["lens"][b])
        cnt = c["n"] if st["counts"] is None else int(st["counts"][b])
        t = pos
        while t < pos + cnt:
            blk, end = t // tb, min(pos + cnt, (t // tb + 1) * tb)
            x = st["new"][:, :, b, :, t - pos:end - pos].double()
            a = x.abs().amax((-1, -2))
            s = _two(_up((a / top).clamp_min(2.0 ** -126)))
            ll = slice(c["layer0"], c["layer0"] + c["nl"])
            if t % tb:
                was = sc[ll, :, b, :, blk]
                s = torch.maximum(s, was)
                old = val[ll, :, b, :, blk * tb:t]
                val[ll, :, b, :, blk * tb:t] = _grid(old * (was / s)[..., None, None], code)
            val[ll, :, b, :, t:end] = _grid(x / s[..., None, None], code)
            sc[ll, :, b, :, blk] = s
            t = end
    return {"codes": None if code == "int8" else val, "scales": sc, "bounds": None}


def _exact_head(q, kc, vc, ks, vs, tb, p, code):
    """One KV head: q [G, d] fp64, codes [n, d] of the tokens 0 .. p, scales a block."""
    k = _numbers(kc, code) * ks.double().repeat_interleave(tb)[:kc.shape[0], None]
    v = _numbers(vc, code) * vs.double().repeat_interleave(tb)[:vc.shape[0], None]
    w = torch.softmax(q @ k[:p].T / math.sqrt(q.shape[-1]), -1)
    return w @ v[:p], w


def _exact_attend(st):
    c = st["case"]
    nl, l0, B, H, d, nq, tb = (c[k] for k in ("nl", "layer0", "B", "H", "d", "nq", "tb"))
    G = c["Hq"] // H
    if c["nl"] * B * H * nq > 3000:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    mass = torch.zeros(st["mass"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        for l in range(nl):
            for h in range(H):
                for i in range(nq):
                    p = n - nq + i + 1
                    if p <= 0:
                        continue
                    j = slice(h * G, h * G + G)
                    m = -(-p // tb)
                    o, w = _exact_head(st["q"][l, b, j, i].double(), st["codes"][l0 + l, 0, b, h, :p], st["codes"][l0 + l, 1, b, h, :p],
                                       st["scales"][l0 + l, 0, b, h, :m], st["scales"][l0 + l, 1, b, h, :m], tb, p, c["code"])
                    out[l, b, j, i] = o
                    mass[l0 + l, b, h, :m] += torch.nn.functional.pad(w.sum(0), (0, m * tb - p)).view(m, tb).sum(1)
    return {"out": out, "mass": mass} if c["mass"] else {"out": out}


def _exact_sparse(st):
    c = st["case"]
    nl, l0, B, H, d, nq, tb, k = (c[n] for n in ("nl", "layer0", "B", "H", "d", "nq", "tb", "k"))
    G = c["Hq"] // H
    if nl * B * H * nq > 1500:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    sel = torch.full((nl, B, H, nq, k), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        for l in range(nl):
            for h in range(H):
                for i in range(nq):
                    p = n - nq + i + 1
                    if p <= 0:
                        continue
                    j, m = slice(h * G, h * G + G), -(-p // tb)
                    q = st["q"][l, b, j, i].double()
                    u = _two(_up((q.abs().amax(-1) / 127).clamp_min(2.0 ** -126)))
                    q8 = torch.round(q / u[:, None])
                    bd = st["bounds"][l0 + l, b, h, :m].double()
                    sc = torch.maximum(q8[:, None] * bd[:, 0], q8[:, None] * bd[:, 1]).sum(-1) * u[:, None]
                    sc = sc.amax(0) * st["scales"][l0 + l, 0, b, h, :m].double()
                    sc[:c["sink"]] = math.inf
                    sc[max(0, m - c["recent"]):] = math.inf
                    s = sc.sort(dim=-1, descending=True, stable=True).indices[:k].sort().values
                    sel[l, b, h, i, :s.numel()] = s.int()
                    t = (s[:, None] * tb + torch.arange(tb, device="cuda")).view(-1)
                    live = t < p
                    t = t.clamp_max(p - 1)
                    kk = _numbers(st["codes"][l0 + l, 0, b, h, t], c["code"]) * st["scales"][l0 + l, 0, b, h, t // tb].double()[:, None]
                    vv = _numbers(st["codes"][l0 + l, 1, b, h, t], c["code"]) * st["scales"][l0 + l, 1, b, h, t // tb].double()[:, None]
                    w = torch.softmax((q @ kk.T / math.sqrt(d)).masked_fill(~live, -math.inf), -1)
                    out[l, b, j, i] = w @ vv
    return {"sel": sel, "out": out}


def exact(case, seed):
    if case["op"] == "evict":       # selections and copies: nothing is computed
        return None
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sparse": _exact_sparse}[case["op"]](st)
