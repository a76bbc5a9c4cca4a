"""Plain 64-bit statements of rotary positions and of a cache held to a budget, with bounds on what the
kernels' roundings can change."""
import math

import numpy as np
import torch

import paged_util as pu


def frequencies(R, base=10000.0):
    return base ** (-2.0 * np.arange(R // 2) / R)


def turn(x, pos, freq, interleaved, factor=1.0, inverse=False):
    """x (Z, H, N, D) float64, pos (Z, N) integers; returns (turned, |a| + |b| of each element's pair)."""
    R = 2 * len(freq)
    angle = pos[:, None, :, None].astype(np.float64) * freq * (-1 if inverse else 1)
    wave = factor * np.exp(1j * angle)
    out, size = x.copy(), np.zeros_like(x)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y = (x[..., a] + 1j * x[..., b]) * wave
    out[..., a], out[..., b] = y.real, y.imag
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, size


def turn_bound(want, size, dtype, factor, far, freq_max=1.0):
    """On |kernel - want|: the position's fraction of a turn in fp32 is off by 2^-25 half turns (pi 2^-25 radians),
    sine and cosine by 2 units of 2^-24 and their product with factor by one more, each of the two products and
    sums by 2^-24 of the pair: below 2^-21 of (|a| + |b|) |factor| in all; `far`, the largest position: the
    frequency's own rounding, p f 2^-52, here and in the statement (numpy reduces p f, rounded to 53 bits); then the
    rounding to the output type, in fp16 also half a subnormal step."""
    u = torch.finfo(pu.DT[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    return size * abs(factor) * (2.0 ** -21 + abs(far) * freq_max * 2.0 ** -50) + u * np.abs(want) * (1 + u) + tiny


def score(q, lse, k, lens, new, scores, decay, scale):
    """(scores after, bound on |kernel's - them|): q (Z, Hq, T, D), lse (Z, Hq, T), scores (Z, Hkv, C) float64; k a
    list of (Hkv, lens[z] + new[z], D).

    A score is a sum of D products, exact in fp32, added by the tensor core (which may truncate): off by at most
    (D + 2) 2^-23 sum |q k| |scale|; its difference to lse, in one rounding (or as the last products of the same
    sum, three 16-bit pieces of lse / scale that hold 24 bits of it), and that times log2 e by 2^-23 of the
    difference; the exponential by 2^-22.  A sum of n weights in fp32 is off by n 2^-24 of itself, joining decay
    times the old score adds two roundings."""
    Z, Hq, T, D = q.shape
    out, bound = scores.copy(), np.zeros_like(scores)
    for z in range(Z):
        n, m = int(lens[z]), int(new[z])
        Hkv = scores.shape[1]
        G = Hq // Hkv
        for hk in range(Hkv):
            w, e, count = np.zeros(n + m), np.zeros(n + m), 0
            for h in range(hk * G, hk * G + G):
                if m == 0:
                    continue
                x = scale * (q[z, h, :m] @ k[z][hk].T)
                size = abs(scale) * (np.abs(q[z, h, :m]) @ np.abs(k[z][hk]).T)
                arg = x - lse[z, h, :m, None]
                seen = np.arange(n + m)[None] <= n + np.arange(m)[:, None]
                seen &= (lse[z, h, :m] != -math.inf)[:, None]
                p = np.where(seen, np.exp(np.where(seen, arg, 0.0)), 0.0)
                w += p.sum(0)
                e += (p * ((D + 2) * 2.0 ** -23 * size + 2.0 ** -22 * np.where(seen, np.abs(arg), 0.0) + 2.0 ** -22)).sum(0)
                count += m
            old = np.concatenate([decay * scores[z, hk, :n] if decay else np.zeros(n), np.zeros(m)])
            out[z, hk, :n + m] = old + w
            bound[z, hk, :n + m] = e + w * (count + 8) * 2.0 ** -24 + (np.abs(old) + w) * 2.0 ** -23 + 1e-37
    return out, bound


def evict(table, lens, refs, scores, page, budget, keep, first, recent):
    """The books of fa_cache_evict on plain lists: (table, lens, refs, missing, kept), kept[z] None or an index
    array (L, H, n); scores an array (L, Z, H, C)."""
    L, Z, H, _ = scores.shape
    M = len(table[0]) if table else 0
    kept, wants = [None] * Z, []
    for z in range(Z):
        n = budget if keep is None else min(budget, keep[z])
        if n < 0 or lens[z] <= n:
            continue
        f = min(first, n)
        r = min(recent, n - f)
        idx = np.empty((L, H, n), dtype=np.int64)
        for la in range(L):
            for h in range(H):
                # best first: a NaN above everything, ties to the lowest position
                middle = sorted(range(f, lens[z] - r),
                                key=lambda j: (-math.inf if math.isnan(scores[la, z, h, j]) else 0,
                                               0.0 if math.isnan(scores[la, z, h, j]) else -scores[la, z, h, j], j))
                idx[la, h] = sorted([*range(f), *middle[:n - f - r], *range(lens[z] - r, lens[z])])
        kept[z] = idx
        moves = np.argwhere((idx != np.arange(n)).any((0, 1)))
        start = int(moves[0, 0]) if len(moves) else n
        wants += [(z, c) for c in range(start // page, pu.cdiv(n, page)) if table[z][c] >= 0 and refs[table[z][c]] > 1]
    free = [p for p, c in enumerate(refs) if c == 0]
    missing = max(0, len(wants) - len(free))
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    if missing:
        return table, lens, refs, missing, [None] * Z
    for (z, c), p in zip(wants, free):
        refs[table[z][c]] -= 1
        refs[p] += 1
        table[z][c] = p
    for z in range(Z):
        if kept[z] is None:
            continue
        n = kept[z].shape[2]
        for c in range(pu.cdiv(n, page), M):
            if table[z][c] >= 0:
                refs[table[z][c]] -= 1
            table[z][c] = -1
        lens[z] = n
    return table, lens, refs, missing, kept


def move(cache, was, now, kept, page):
    """The rows of a cache (L, P, H, page, D) after evict (was, now: the tables before and after)."""
    before = cache.clone()
    for z, idx in enumerate(kept):
        if idx is None:
            continue
        L, H, n = idx.shape
        for la in range(L):
            for h in range(H):
                for i, j in enumerate(idx[la, h]):
                    cache[la, now[z][i // page], h, i % page] = before[la, was[z][j // page], h, j % page]
    return cache
