"""The 8-bit KV cache with a scale for each block of tokens and head, in plain fp64 and loops
(test infrastructure only).

codes [L, 2, B, H, T, d] uint8 (int8 or e4m3 bit patterns), scales [L, 2, B, H, T/tb] powers of
two, bounds [L, B, H, T/tb, 2, d] int8, mass [L, B, H, T/tb].  The functions that store change
their arrays in place.
"""
import numpy as np

INT8, E4M3 = 0, 1
TOP = (127.0, 448.0)


def _e4m3_table():
    """Values of the 256 e4m3 patterns: s eeee mmm, bias 7, no infinities, 0x7f and 0xff NaN."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = np.nan if (b & 127) == 127 else (-x if b & 128 else x)
    return v


E4M3_VALUES = _e4m3_table()


def decode(codes, code):
    codes = np.asarray(codes, np.uint8)
    return codes.view(np.int8).astype(np.float64) if code == INT8 else E4M3_VALUES[codes]


def encode(x, code):
    """Nearest code, ties to even (of |x| <= top)."""
    x = np.asarray(x, np.float64)
    if code == INT8:
        return np.rint(x).astype(np.int8).view(np.uint8)
    grid = E4M3_VALUES[:127]
    a = np.abs(x)
    i = np.clip(np.searchsorted(grid, a), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    c = np.where(up, i, i - 1).astype(np.uint8)
    # the sign of a zero is kept, as IEEE rounding keeps it
    return c | (np.signbit(x).astype(np.uint8) << 7)


def scale_of(amax, code):
    """The least power of two s >= 2^-126 with amax <= top s."""
    s = 2.0 ** -126
    m, x = np.frexp(float(amax) / TOP[code])
    return s if amax == 0 else max(s, 2.0 ** (x if m > 0.5 else x - 1))


def bound_pair(v, code):
    """int8 [2, d] of code values v [n, d]."""
    lo, hi = v.min(0), v.max(0)
    if code == E4M3:  # exact: multiples of 2^-9 times 127 over 448
        lo = np.array([(int(x * 512) * 127) // (448 * 512) for x in lo])
        hi = np.array([-((-int(x * 512) * 127) // (448 * 512)) for x in hi])
    return np.stack([lo, hi]).astype(np.int8)


def append(codes, scales, bounds, new, pos, counts, code, tb, layer0=0):
    """new [nl, 2, B, H, n, d]; pos [B]; counts [B] or None."""
    nl, _, B, H, n, d = new.shape
    T = codes.shape[4]
    for b in range(B):
        p, cnt = int(pos[b]), n if counts is None else min(n, int(counts[b]))
        if p < 0 or cnt <= 0:
            continue
        end = min(p + cnt, T)
        for lz in range(nl):
            for s in range(2):
                for h in range(H):
                    at, l = p, layer0 + lz
                    while at < end:
                        blk = at // tb
                        b0, to = blk * tb, min(end, blk * tb + tb)
                        x = np.asarray(new[lz, s, b, h, at - p:to - p], np.float64)
                        sc = scale_of(np.abs(x).max(), code)
                        old, grew = float(scales[l, s, b, h, blk]), False
                        holds = at > b0 and 0 < old < np.inf
                        if holds:
                            grew = sc > old
                            if grew:
                                v = decode(codes[l, s, b, h, b0:at], code) * (old / sc)
                                codes[l, s, b, h, b0:at] = encode(v, code)
                            else:
                                sc = old
                        codes[l, s, b, h, at:to] = encode(x / sc, code)
                        scales[l, s, b, h, blk] = sc
                        if s == 0 and bounds is not None:
                            pair = bound_pair(decode(codes[l, s, b, h, b0 if grew else at:to], code), code)
                            if holds and not grew:
                                was = bounds[l, b, h, blk]
                                pair = np.stack([np.minimum(pair[0], was[0]), np.maximum(pair[1], was[1])])
                            bounds[l, b, h, blk] = pair
                        at = to


def attention(q, codes, scales, lens, code, tb, scale, layer0=0, max_tokens=None, sel=None):
    """q [nl, B, Hq, nq, d] -> (out of the same shape, mass [nl, B, H, T/tb], sum p |v|, and per row the
    largest scale sum_c |q_c k_c|), fp64."""
    nl, B, Hq, nq, d = q.shape
    H, T = codes.shape[3], codes.shape[4]
    G = Hq // H
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    mass, big = np.zeros((nl, B, H, T // tb)), np.zeros(q.shape[:-1])
    for lz in range(nl):
        for b in range(B):
            n = min(max(int(lens[b]), 0), T if max_tokens is None else max_tokens)
            for h in range(H):
                l = layer0 + lz
                # behind the length may stand anything
                k = decode(codes[l, 0, b, h, :n], code) * np.repeat(np.asarray(scales[l, 0, b, h], np.float64), tb)[:n, None]
                v = decode(codes[l, 1, b, h, :n], code) * np.repeat(np.asarray(scales[l, 1, b, h], np.float64), tb)[:n, None]
                for i in range(nq):
                    p = n - nq + i + 1
                    if p <= 0:
                        continue
                    t = np.arange(p)
                    if sel is not None:
                        blocks = [int(x) for x in sel[lz, b, h, i] if 0 <= x <= (p - 1) // tb]
                        t = np.concatenate([np.arange(x * tb, min(p, x * tb + tb)) for x in blocks] or [np.zeros(0, int)])
                        if not len(t):
                            continue
                    for j in range(h * G, h * G + G):
                        s = k[t] @ q[lz, b, j, i] * scale
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        out[lz, b, j, i] = w @ v[t]
                        spread[lz, b, j, i] = w @ np.abs(v[t])
                        big[lz, b, j, i] = (np.abs(k[t]) @ np.abs(q[lz, b, j, i])).max() * scale
                        np.add.at(mass[lz, b, h], t // tb, w)
    return out, mass, spread, big


def _pick(key, nb, k, sink, recent):
    """k blocks of nb, ascending: the first `sink`, the last `recent`, the highest keys (ties low)."""
    if nb <= k:
        return list(range(nb))
    forced = list(range(sink)) + list(range(nb - recent, nb))
    rest = sorted(range(sink, nb - recent), key=lambda i: (-key[i], i))
    return sorted(forced + rest[:k - sink - recent])


def scores(q, bounds, scales):
    """q [G, d], bounds [nb, 2, d], key scales [nb] -> [nb] fp64 (every step exact)."""
    best = np.full(bounds.shape[0], -np.inf)
    for row in np.asarray(q, np.float64):
        unit = scale_of(np.abs(row).max(), INT8)
        q8 = np.rint(row / unit)
        dot = np.maximum(q8 * bounds[:, 0].astype(np.float64), q8 * bounds[:, 1].astype(np.float64)).sum(1)
        best = np.maximum(best, dot * unit)
    return best * np.asarray(scales, np.float64)


def select(q, bounds, scales, lens, tb, k, sink, recent, H, layer0=0, max_tokens=None):
    """q [nl, B, Hq, nq, d] -> int32 [nl, B, H, nq, k]."""
    nl, B, Hq, nq, _ = q.shape
    G = Hq // H
    sel = np.full((nl, B, H, nq, k), -1, np.int32)
    for lz in range(nl):
        for b in range(B):
            n = max(int(lens[b]), 0) if max_tokens is None else min(max(int(lens[b]), 0), max_tokens)
            for h in range(H):
                for i in range(nq):
                    nb = -(-max(0, n - nq + i + 1) // tb)
                    sc = scores(q[lz, b, h * G:h * G + G, i], bounds[layer0 + lz, b, h, :nb], scales[layer0 + lz, 0, b, h, :nb])
                    got = _pick(sc, nb, k, sink, recent)
                    sel[lz, b, h, i, :len(got)] = got
    return sel


def evict(codes, scales, bounds, mass, lens, to, tb, keep, sink, recent, layer0=0, n_layers=1):
    """`to` (codes, scales, bounds, mass, lens) is written in place; returns kept [nl, B, H, keep]."""
    tc, ts, tbd, tm, tl = to
    L, _, B, H, T, d = codes.shape
    kept = np.full((n_layers, B, H, keep), -1, np.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), T)
        nb = -(-n // tb)
        tl[b] = n - (nb - keep) * tb if nb > keep else n
        for lz in range(n_layers):
            l = layer0 + lz
            for h in range(H):
                key = np.where(np.isnan(mass[l, b, h]), -np.inf, mass[l, b, h])
                got = _pick(key, nb, keep, sink, recent)
                kept[lz, b, h, :len(got)] = got
                tm[l, b, h] = 0
                for j, i in enumerate(got):
                    tc[l, :, b, h, j * tb:j * tb + tb] = codes[l, :, b, h, i * tb:i * tb + tb]
                    ts[l, :, b, h, j] = scales[l, :, b, h, i]
                    if bounds is not None:
                        tbd[l, b, h, j] = bounds[l, b, h, i]
                    tm[l, b, h, j] = mass[l, b, h, i]
    return kept
