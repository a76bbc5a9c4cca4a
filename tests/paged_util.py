"""Plain 64-bit statements of the paged-cache operators, one sequence and one row at a time, and
random caches to run them on."""
import math

import numpy as np
import torch

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def cdiv(a, b):
    return -(-a // b)


def make_cache(seed, lens, Hkv, D, page, dtype, *, extra=5, cols=None, garbage=float("nan"), layout="phnd", layers=None):
    """K and V caches holding sequences of `lens` positions over shuffled pages (positions behind the
    last one and unused pages hold `garbage`), the block table, and the rows themselves as lists of
    (Hkv, len, D) float64 arrays."""
    g = torch.Generator().manual_seed(seed)
    n = [cdiv(int(x), page) for x in lens]
    P = sum(n) + extra
    ids = torch.randperm(P, generator=g).tolist()
    M = max([1] + n) if cols is None else cols
    table = torch.full((len(lens), M), -1, dtype=torch.int32)
    L = 1 if layers is None else layers
    caches, rows = [], []
    at = 0
    for z, k in enumerate(n):
        table[z, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        at += k
    for _ in range(2):
        c = torch.full((L, P, Hkv, page, D), garbage, dtype=DT[dtype])
        mine = []
        for z, m in enumerate(lens):
            x = torch.randn((L, Hkv, int(m), D), generator=g).to(DT[dtype])
            for i in range(n[z]):
                w = x[:, :, i * page:(i + 1) * page]
                c[:, table[z, i], :, :w.shape[2]] = w
            mine.append(x.double().numpy() if layers is not None else x[0].double().numpy())
        if layout == "pnhd":  # (page, slot, head, d) storage seen as (page, head, slot, d)
            c = c.transpose(2, 3).contiguous().transpose(2, 3)
        elif layout == "padded":
            pad = torch.full((L, P, Hkv, page + 1, D + 8), garbage, dtype=DT[dtype])
            pad[:, :, :, :page, :D] = c
            c = pad[:, :, :, :page, :D]
        caches.append(c if layers is not None else c[0])
        rows.append(mine)
    return caches[0], caches[1], table, rows[0], rows[1]


def like(c):
    """The same tensor on the GPU with the same strides."""
    base = torch.empty(sum((s - 1) * t for s, t in zip(c.shape, c.stride())) + 1, dtype=c.dtype, device="cuda")
    out = base.as_strided(c.shape, c.stride())
    out.copy_(c)
    return out


def tree_words(seen):
    """(Z, T, T) truth values -> (Z, T, ceil(T/32)) int32 words."""
    Z, T, _ = seen.shape
    bits = np.zeros((Z, T, 32 * cdiv(T, 32)), dtype=bool)
    bits[:, :, :T] = seen
    return torch.from_numpy(np.packbits(bits, axis=2, bitorder="little").view(np.int32).copy())


def random_tree(seed, Z, T):
    """Ancestor-or-self relations of random trees."""
    r = np.random.RandomState(seed)
    seen = np.zeros((Z, T, T), dtype=bool)
    for z in range(Z):
        for t in range(T):
            if t:
                seen[z, t] = seen[z, r.randint(max(0, t - 5), t)]
            seen[z, t, t] = True
    return seen


def attention(q, k, v, lens, new, seen, scale):
    """q (Z, Hq, T, D) float64; k, v lists of (Hkv, lens[z] + new[z], D); seen (Z, T, T) or None (chain)."""
    Z, Hq, T, D = q.shape
    o, lse = np.zeros((Z, Hq, T, D)), np.full((Z, Hq, T), -math.inf)
    for z in range(Z):
        for h in range(Hq):
            hk = h // (Hq // k[z].shape[0])
            for t in range(int(new[z])):
                keep = np.zeros(int(lens[z]) + int(new[z]), dtype=bool)
                keep[:int(lens[z])] = True
                keep[int(lens[z]):] = (np.arange(int(new[z])) <= t) if seen is None else seen[z, t, :int(new[z])]
                if not keep.any():
                    continue
                s = scale * (k[z][hk][keep] @ q[z, h, t])
                m = s.max()
                p = np.exp(s - m)
                o[z, h, t] = p @ v[z][hk][keep] / p.sum()
                lse[z, h, t] = m + math.log(p.sum())
    return o, lse


def tolerances(q, k, v, dtype, scale):
    """(O, lse) bounds, absolute, from the roundings that the kernel makes.

    A score is a sum of D exact products in fp32: off by at most (D + 2) 2^-24 sum |q k| |scale|
    = delta.  A weight 2^x: delta from its score, 2^-22 from the exponential.  P is rounded to the
    input type before P V, and O at the end, each by at most eps / 2 of the value (|O| <= max |v|);
    moving weights by e relative moves O by at most 2 e max |v|.  The sums in fp32 of n weights or
    products add less than 2^-20 each at these sizes.  lse: delta + the sum's 2^-20 + its own fp32
    rounding."""
    u = torch.finfo(DT[dtype]).eps / 2
    D = q.shape[-1]
    big = max([float((np.abs(x)).max()) for x in k if x.size] + [0.0])
    prod = float(np.abs(q).sum(-1).max()) * big * abs(scale)
    delta = (D + 2) * 2.0 ** -24 * prod
    vmax = max([float(np.abs(x).max()) for x in v if x.size] + [0.0])
    o = vmax * (2 * u + 2 * (delta + 2.0 ** -22 + 2.0 ** -20))
    return o, delta + 2.0 ** -20 + 2.0 ** -22 * (prod + 12)


def fork(table, lens, refs, source, room, page):
    """The bookkeeping of fa_cache_fork on plain lists: (table, lens, refs, missing, tails), tails a
    list of (from page, to page, rows)."""
    Z, M = len(table), len(table[0]) if table else 0
    before = [list(r) for r in table]
    out, newlens, refs = [list(r) for r in table], list(lens), list(refs)
    free = [p for p, c in enumerate(refs) if c == 0]
    missing, tails = 0, []
    for z in range(Z):
        a = z if source is None else source[z]
        n = lens[a] if a >= 0 else 0
        newlens[z] = n
        first = cdiv(n, page)
        row = before[z][:]
        if a != z:
            first = n // page
            for p in row:
                if p >= 0:
                    refs[p] -= 1
            row = [before[a][c] if a >= 0 and c < first else -1 for c in range(M)]
            for p in row:
                if p >= 0:
                    refs[p] += 1
        need = cdiv(n + room, page) if a >= 0 else 0
        for c in range(first, need):
            if c >= M:
                missing += 1
            elif row[c] < 0:
                if not free:
                    missing += 1
                    continue
                row[c] = free.pop(0)
                refs[row[c]] += 1
                if a != z and c == n // page and n % page:
                    tails.append((before[a][c], row[c], n % page))
        out[z] = row
    return out, newlens, refs, missing, tails
