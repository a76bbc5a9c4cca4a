"""Measured cases of the paged-cache operators: attention of new or drafted tokens over a paged
cache (fa_fwd_paged), writing new rows to it (fa_cache_append), moving accepted drafted rows
together (fa_cache_commit), and forking / freeing sequences (fa_cache_fork).

Each operator has a plain form (elementary torch operations, fp32, rounded once) and the call of
the framework's own kernel, and `exact` states the same result in 64 bits (or, for the operators
that only move data, by one slice assignment per sequence).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _attn(name, Z, Hq, Hkv, D, T, lo, hi, page, dtype, mask, ragged):
    return {"name": name, "op": "attention", "Z": Z, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "lo": lo, "hi": hi,
            "page": page, "dtype": dtype, "mask": mask, "ragged": ragged}


def listed():
    return [
        # one user, one token at a time after a short prompt: latency only
        _attn("decode_one", 1, 32, 8, 128, 1, 1024, 1024, 16, "bf16", "chain", False),
        # a serving batch of ragged contexts, one token each: streams the cache
        _attn("decode_batch", 64, 32, 8, 128, 1, 256, 4096, 64, "bf16", "chain", False),
        # two long documents, no shared heads: few rows, work must be cut along the keys
        _attn("decode_long", 2, 16, 16, 64, 1, 30000, 32768, 16, "fp16", "chain", False),
        # speculative decoding of a small batch: 32 drafted tokens in a tree
        _attn("tree_chat", 8, 32, 8, 128, 32, 500, 3000, 32, "bf16", "tree", False),
        # a large batch with wide trees over long contexts: the largest case
        _attn("tree_wide", 32, 32, 8, 128, 64, 4096, 8192, 64, "bf16", "tree", False),
        # wide heads, an odd group, odd page and tree sizes, ragged drafts, contexts down to one token
        _attn("tree_d256", 5, 12, 2, 256, 17, 1, 2000, 48, "fp16", "tree", True),
        # a decode step writes one row a sequence
        {"name": "append_step", "op": "append", "Z": 64, "Hkv": 8, "D": 128, "T": 1, "lo": 100, "hi": 500, "page": 16,
         "dtype": "bf16", "ragged": False},
        # prompts of ragged lengths enter the cache
        {"name": "append_prompts", "op": "append", "Z": 5, "Hkv": 8, "D": 128, "T": 2011, "lo": 0, "hi": 300,
         "page": 64, "dtype": "fp16", "ragged": True},
        # a few sequences keep their accepted drafts, all layers at once
        {"name": "commit_few", "op": "commit", "Z": 4, "L": 16, "Hkv": 8, "D": 128, "T": 32, "A": 5, "lo": 20,
         "hi": 100, "page": 16, "dtype": "bf16"},
        # a serving batch keeps its accepted drafts
        {"name": "commit_batch", "op": "commit", "Z": 64, "L": 16, "Hkv": 8, "D": 128, "T": 64, "A": 9, "lo": 5,
         "hi": 90, "page": 32, "dtype": "fp16"},
        # eight beams of one prompt are re-chosen
        {"name": "fork_beams", "op": "fork", "Z": 8, "L": 16, "Hkv": 8, "D": 128, "lo": 500, "hi": 700, "page": 16,
         "room": 1, "dtype": "bf16"},
        # a batch of parallel samples: weak ones replaced, some ended
        {"name": "fork_batch", "op": "fork", "Z": 96, "L": 8, "Hkv": 2, "D": 128, "lo": 200, "hi": 1200, "page": 16,
         "room": 33, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "commit", "fork"])
    dtype = rng.choice(["bf16", "fp16"])
    page = 16 * rng.choice([1, 1, 2, 3, 4, 8])
    D = rng.choice([64, 128, 128, 256])
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        G = rng.choice([g for g in (1, 2, 3, 4, 6, 8) if Hkv * g <= 32])
        T = 1 if rng.random() < 0.4 else _log_int(rng, 2, 64)
        hi = _log_int(rng, 16, 32768)
        lo = rng.randint(1, hi)
        # at most about the largest listed case's cache reads and score products
        most = min(1.6e8 / (hi * Hkv * D), 2e10 / (hi * Hkv * G * T * D))
        Z = max(1, min(64, _log_int(rng, 1, max(1.0, most))))
        return {"op": op, "Z": Z, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "T": T, "lo": lo, "hi": hi, "page": page,
                "dtype": dtype, "mask": "tree" if T > 1 and rng.random() < 0.7 else "chain",
                "ragged": T > 1 and rng.random() < 0.5}
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "append":
        T = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2048)
        Z = _log_int(rng, 1, max(1, min(128, 16000 // T)))
        return {"op": op, "Z": Z, "Hkv": Hkv, "D": D, "T": T, "lo": 0, "hi": rng.randint(1, 400), "page": page,
                "dtype": dtype, "ragged": T > 1 and rng.random() < 0.6}
    L = _log_int(rng, 1, 16)
    if op == "commit":
        T = _log_int(rng, 8, 64)
        return {"op": op, "Z": _log_int(rng, 1, max(1, min(64, 4096 // (L * Hkv)))), "L": L, "Hkv": Hkv, "D": D,
                "T": T, "A": rng.randint(1, min(9, T // 2)), "lo": rng.randint(0, 40), "hi": rng.randint(41, 90),
                "page": page, "dtype": dtype}
    hi = rng.randint(17, 1200)
    return {"op": op, "Z": _log_int(rng, 2, 48), "L": min(L, 8), "Hkv": min(Hkv, 2), "D": min(D, 128),
            "lo": rng.randint(0, hi), "hi": hi, "page": page, "room": rng.choice([0, 1, 1, 17, 64]), "dtype": dtype}


# ------------------------------------------------------------------ sizes that a case fixes for every seed

def _spread(lo, hi, Z):
    """Z lengths spread evenly over lo .. hi (their order is the seed's)."""
    return np.linspace(lo, hi, Z).round().astype(np.int64) if Z > 1 else np.array([hi])


def _new_lens(case):
    """How many of the T new tokens each sequence has."""
    return _spread((case["T"] + 1) // 2, case["T"], case["Z"]) if case["ragged"] else np.full(case["Z"], case["T"])


def _accepted_lens(case):
    return _spread(1, case["A"], case["Z"])


def _pages(tokens, page):
    return (np.asarray(tokens) + page - 1) // page


def _fork_roles(case):
    """(survivors, children, ended): half the sequences stay, most others become copies, an eighth ends."""
    Z = case["Z"]
    keep = max(1, Z // 2)
    ended = Z // 8
    return keep, Z - keep - ended, ended


# ------------------------------------------------------------------ inputs

def _table(rng, tokens, page, slack):
    """A block table over shuffled pages, -1 past each sequence's last page; (table, pool pages)."""
    n = _pages(tokens, page)
    pool = int(n.sum()) + slack
    ids = rng.permutation(pool)[:int(n.sum())]
    table = np.full((len(n), int(max(1, n.max()))), -1, dtype=np.int32)
    at = 0
    for z, k in enumerate(n):
        table[z, :k] = ids[at:at + k]
        at += k
    return table, pool


def _normal(gen, shape, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        flat[i:i + (1 << 26)].normal_(generator=gen)
    return out


def _tree_bits(rng, Z, T):
    """Ancestor bits of random draft trees: token i's parent is one of the eight tokens before it."""
    words = (T + 31) // 32
    bits = np.zeros((Z, T, 32 * words), dtype=bool)
    for i in range(T):
        if i:
            parent = rng.randint(max(0, i - 8), i, Z)
            bits[:, i] = bits[np.arange(Z), parent]
        bits[:, i, i] = True
    packed = np.packbits(bits, axis=2, bitorder="little").view(np.uint32)
    return packed.reshape(Z, T, words).view(np.int32)


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, Z, page = DTYPES[case["dtype"]], case["Z"], case["page"]
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    lens = rng.permutation(_spread(case["lo"], case["hi"], Z))
    # one workspace that a serving loop keeps for all of its calls
    s = {"op": case["op"], "page": page, "ws": torch.empty(96 << 20, dtype=torch.uint8, device="cuda")}
    if case["op"] == "attention":
        new = rng.permutation(_new_lens(case))
        table, pool = _table(rng, lens + case["T"], page, 7)
        shape = (pool, case["Hkv"], page, case["D"])
        s |= {"q": _normal(gen, (Z, case["Hq"], case["T"], case["D"]), dt), "k": _normal(gen, shape, dt),
              "v": _normal(gen, shape, dt), "table": cuda(table), "lens": cuda(lens.astype(np.int32)),
              "new": cuda(new.astype(np.int32)) if case["ragged"] else None,
              "mask": cuda(_tree_bits(rng, Z, case["T"])) if case["mask"] == "tree" else None}
        return s
    if case["op"] == "append":
        new = rng.permutation(_new_lens(case))
        table, pool = _table(rng, lens + case["T"], page, 7)
        rows = (Z, case["T"], case["Hkv"], case["D"])  # a projection's output, seen as (Z, Hkv, T, D)
        s |= {"k_new": _normal(gen, rows, dt).transpose(1, 2), "v_new": _normal(gen, rows, dt).transpose(1, 2),
              "k": _normal(gen, (pool, case["Hkv"], page, case["D"]), dt),
              "v": _normal(gen, (pool, case["Hkv"], page, case["D"]), dt), "table": cuda(table),
              "lens": cuda(lens.astype(np.int32)), "new": cuda(new.astype(np.int32)) if case["ragged"] else None}
        return s
    if case["op"] == "commit":
        kept = rng.permutation(_accepted_lens(case))
        table, pool = _table(rng, lens + case["T"], page, 7)
        path = np.zeros((Z, case["A"]), dtype=np.int32)
        for z in range(Z):  # the root, then drafted tokens of deeper levels, each below the one before
            path[z, 1:kept[z]] = np.sort(kept[z] + rng.permutation(case["T"] - kept[z])[:kept[z] - 1])
        shape = (case["L"], pool, case["Hkv"], page, case["D"])
        s |= {"k": _normal(gen, shape, dt), "v": _normal(gen, shape, dt), "table": cuda(table),
              "lens": cuda(lens.astype(np.int32)), "path": cuda(path), "kept": cuda(kept.astype(np.int32))}
        return s
    keep, children, ended = _fork_roles(case)
    room = int(_pages(case["hi"] + case["room"], page))
    table, pool = _table(rng, lens, page, Z * (2 + int(_pages(case["room"], page))) * 2)
    table = np.concatenate([table, np.full((Z, max(0, room + 1 - table.shape[1])), -1, dtype=np.int32)], axis=1)
    order = rng.permutation(Z)
    source = np.arange(Z, dtype=np.int32)
    source[order[keep:keep + children]] = order[rng.randint(0, keep, children)]
    source[order[keep + children:]] = -1
    refs = np.bincount(table[table >= 0], minlength=pool).astype(np.int32)
    shape = (case["L"], pool, case["Hkv"], page, case["D"])
    s |= {"k": _normal(gen, shape, dt), "v": _normal(gen, shape, dt), "table": cuda(table), "refs": cuda(refs),
          "lens": cuda(lens.astype(np.int32)), "source": cuda(source), "room": case["room"],
          "missing": torch.zeros(1, dtype=torch.int32, device="cuda")}
    return s


# ------------------------------------------------------------------ plain forms

def _plain_attention(q, k, v, table, lens, new, mask, page):
    Z, Hq, T, D = q.shape
    Hkv, M = k.shape[1], table.shape[1]
    N = M * page
    dev = q.device
    pos = torch.arange(N, device=dev)
    end = lens + (T if new is None else new)
    there = pos[None] < end[:, None]                                                     # (Z, N)
    pages = table.clamp(min=0).long()

    def rows(cache):
        x = cache[pages].permute(0, 2, 1, 3, 4).reshape(Z, Hkv, N, D).float()
        return torch.where(there[:, None, :, None], x, torch.zeros((), device=dev))

    x = q.float().reshape(Z, Hkv, Hq // Hkv * T, D) @ rows(k).transpose(2, 3) * (1 / math.sqrt(D))
    x = x.view(Z, Hkv, Hq // Hkv, T, N)
    draft = pos[None] - lens[:, None]                                                    # (Z, N)
    t = torch.arange(T, device=dev)
    if mask is None:
        seen = draft[:, None] <= t[None, :, None]
    else:
        word = (draft.clamp(0, T - 1) >> 5)[:, None].expand(Z, T, N)
        bit = mask.gather(2, word.long()) >> (draft.clamp(0, T - 1) & 31)[:, None] & 1
        seen = (draft < 0)[:, None] | (bit != 0)
    seen = seen & there[:, None] & (lens[:, None] + t[None] < end[:, None])[:, :, None]  # (Z, T, N)
    x = torch.where(seen[:, None, None], x, torch.full((), -math.inf, device=dev))
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros((), device=dev), top)
    x = torch.exp(x - base)
    total = x.sum(-1, keepdim=True)
    o = x.view(Z, Hkv, -1, N) @ rows(v)
    o = o.view(Z, Hkv, Hq // Hkv, T, D) / torch.where(total == 0, torch.ones((), device=dev), total)
    lse = (top + torch.log(total)).squeeze(-1)
    lse = torch.where(total.squeeze(-1) == 0, torch.full((), -math.inf, device=dev), lse)
    return o.reshape(Z, Hq, T, D).to(q.dtype), lse.reshape(Z, Hq, T)


def _plain_append(k_new, v_new, k, v, table, lens, new, page):
    Z, Hkv, T, D = k_new.shape
    t = torch.arange(T, device=k.device)
    pos = lens[:, None] + t[None]
    z, i = torch.nonzero(t[None] < (torch.full_like(lens, T) if new is None else new)[:, None], as_tuple=True)
    at = table[z, pos[z, i] // page].long(), pos[z, i] % page
    k[at[0], :, at[1]] = k_new[z, :, i]
    v[at[0], :, at[1]] = v_new[z, :, i]
    return k, v


def _plain_commit(k, v, table, lens, path, kept, page):
    z, i = torch.nonzero(torch.arange(path.shape[1], device=k.device)[None] < kept[:, None], as_tuple=True)
    frm, to = lens[z] + path[z, i], lens[z] + i
    fp, tp = table[z, frm // page].long(), table[z, to // page].long()
    k[:, tp, :, to % page] = k[:, fp, :, frm % page]
    v[:, tp, :, to % page] = v[:, fp, :, frm % page]
    return k, v


def _plain_fork(k, v, table, lens, refs, source, room, missing, page):
    Z, M = table.shape
    dev = table.device
    col = torch.arange(M, device=dev)[None]
    same = source == torch.arange(Z, device=dev)
    live = source >= 0
    frm = source.clamp(min=0).long()
    length = torch.where(live, lens[frm], 0)
    full = length // page
    start = torch.where(same, (length + page - 1) // page, full)       # pages kept or shared
    shared = live[:, None] & (col < full[:, None])
    after = torch.where(same[:, None], table, torch.where(shared, table[frm], -1))
    need = torch.where(live, (length + room + page - 1) // page, 0)
    want = (col >= start[:, None]) & (col < need[:, None]) & (after < 0)
    rank = torch.cumsum(want.view(-1), 0).view(Z, M) - 1
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True).to(torch.int32)  # free pages first, lowest first
    count = (refs == 0).sum()
    got = want & (rank < count)
    after = torch.where(got, free[rank.clamp(0, refs.numel() - 1)], after)
    missing.copy_((want.sum() - got.sum() + (need - M).clamp(min=0).sum()).view(1))
    # one reference less for each page that a changed sequence held, one more for each that it holds now
    change = torch.zeros(refs.numel() + 1, dtype=torch.int32, device=dev)
    old = torch.where(same[:, None] | (table < 0), refs.numel(), table).view(-1).long()
    now = torch.where((same[:, None] & ~got) | (after < 0), refs.numel(), after).view(-1).long()
    change.index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    change.index_add_(0, now, torch.ones_like(now, dtype=torch.int32))
    tail = length % page
    z = torch.nonzero(~same & live & (tail > 0), as_tuple=True)[0]
    fp, tp = table[frm[z], full[z].clamp(max=M - 1).long()].long(), after[z, full[z].clamp(max=M - 1).long()].long()
    z, fp, tp = z[tp >= 0], fp[tp >= 0], tp[tp >= 0]
    row = (torch.arange(page, device=dev)[None] < tail[z][:, None])[None, :, None, :, None]
    k[:, tp] = torch.where(row, k[:, fp], k[:, tp])
    v[:, tp] = torch.where(row, v[:, fp], v[:, tp])
    refs += change[:-1]
    table.copy_(after)
    lens.copy_(length)
    return k, v, table, lens, refs, missing


def run(s):
    if s["op"] == "attention":
        if own:
            import exact_attention_44_gb300 as fa
            return fa.fa_fwd_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], new_lens=s["new"],
                                   tree_mask=s["mask"], workspace=s["ws"])
        return _plain_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["new"], s["mask"], s["page"])
    if s["op"] == "append":
        if own:
            import exact_attention_44_gb300 as fa
            fa.fa_cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], new_lens=s["new"])
            return s["k"], s["v"]
        return _plain_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], s["new"], s["page"])
    if s["op"] == "commit":
        if own:
            import exact_attention_44_gb300 as fa
            fa.fa_cache_commit(s["k"], s["v"], s["table"], s["lens"], s["path"], s["kept"])
            return s["k"], s["v"]
        return _plain_commit(s["k"], s["v"], s["table"], s["lens"], s["path"], s["kept"], s["page"])
    if own:
        import exact_attention_44_gb300 as fa
        fa.fa_cache_fork(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["source"], room=s["room"],
                         missing=s["missing"], workspace=s["ws"])
        return s["k"], s["v"], s["table"], s["lens"], s["refs"], s["missing"]
    return _plain_fork(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["source"], s["room"], s["missing"],
                       s["page"])


# ------------------------------------------------------------------ what the path cannot do without

def work(case):
    Z, D, page = case["Z"], case["D"], case["page"]
    lens = _spread(case["lo"], case["hi"], Z)
    if case["op"] == "attention":
        new = _new_lens(case)
        G = case["Hq"] // case["Hkv"]
        # (which draft count meets which length is the seed's: means)
        cached = float((lens + new).sum())
        rows = float(new.sum()) * case["Hq"]
        per_row = float((lens.mean() + (new.mean() + 1) / 2))
        table = 4 * float(_pages(lens + new, page).sum())
        mask = 4 * Z * case["T"] * ((case["T"] + 31) // 32) if case["mask"] == "tree" else 0
        return {"bytes": cached * case["Hkv"] * D * 4 + rows * D * 2 + Z * case["Hq"] * case["T"] * (2 * D + 4) +
                table + mask + 4 * Z, "flops": 4.0 * rows * per_row * D if G else 0.0}
    if case["op"] == "append":
        rows = float(_new_lens(case).sum())
        return {"bytes": rows * case["Hkv"] * D * 2 * 4 + 4 * rows / page + 8 * Z, "flops": 0}
    if case["op"] == "commit":
        rows = float((_accepted_lens(case) - 1).sum())  # the root stays where it is
        return {"bytes": max(16.0, rows * case["L"] * case["Hkv"] * D * 2 * 4 + 4 * Z * (case["A"] + 3)), "flops": 0}
    keep, children, ended = _fork_roles(case)
    tail = float((lens % page).mean()) * children
    pages = float(_pages(lens, page).mean())
    return {"bytes": tail * case["L"] * case["Hkv"] * D * 2 * 4 + 4 * pages * (children * 3 + ended * 2) * 2 +
            4 * float(_pages(lens, page).sum()) + 16 * Z, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits, one sequence at a time

def exact(case, seed):
    s = prepare(case, seed)
    page, table, lens = case["page"], s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    if case["op"] == "attention":
        return _exact_attention(case, s, table, lens)
    k, v = s["k"], s["v"]
    if case["op"] == "append":
        new = s["new"].cpu().numpy() if s["new"] is not None else np.full(case["Z"], case["T"])
        for z in range(case["Z"]):
            t = 0
            while t < new[z]:
                p, slot = divmod(int(lens[z]) + t, page)
                n = min(page - slot, int(new[z]) - t)
                k[table[z, p], :, slot:slot + n] = s["k_new"][z, :, t:t + n]
                v[table[z, p], :, slot:slot + n] = s["v_new"][z, :, t:t + n]
                t += n
        return k, v
    if case["op"] == "commit":
        path, kept = s["path"].cpu().numpy(), s["kept"].cpu().numpy()
        for z in range(case["Z"]):
            for i in range(kept[z]):
                a, b = divmod(int(lens[z] + path[z, i]), page), divmod(int(lens[z]) + i, page)
                if a != b:
                    k[:, table[z, b[0]], :, b[1]] = k[:, table[z, a[0]], :, a[1]]
                    v[:, table[z, b[0]], :, b[1]] = v[:, table[z, a[0]], :, a[1]]
        return k, v
    source, refs = s["source"].cpu().numpy(), s["refs"].cpu().numpy().copy()
    before, M = table.copy(), table.shape[1]
    free = [int(p) for p in np.flatnonzero(refs == 0)]
    missing, out = 0, lens.copy()
    for z in range(case["Z"]):
        a = int(source[z])
        n = int(lens[a]) if a >= 0 else 0
        out[z] = n
        row = [int(p) for p in before[z]]
        first = -(-n // page)
        if a != z:
            for p in row:
                if p >= 0:
                    refs[p] -= 1
            row = [-1] * M
            first = n // page
            for c in range(first):
                row[c] = int(before[a, c])
                refs[row[c]] += 1
        for c in range(first, -(-(n + case["room"]) // page) if a >= 0 else 0):
            if c >= M or (row[c] < 0 and not free):
                missing += 1
            elif row[c] < 0:
                row[c] = free.pop(0)
                refs[row[c]] += 1
                if a != z and c == n // page and n % page:
                    k[:, row[c], :, :n % page] = k[:, before[a, c], :, :n % page]
                    v[:, row[c], :, :n % page] = v[:, before[a, c], :, :n % page]
        table[z] = row
    whole = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32))  # noqa: E731
    return k, v, whole(table), whole(out), whole(refs), whole([missing])


def _exact_attention(case, s, table, lens):
    Z, Hq, Hkv, T, D = case["Z"], case["Hq"], case["Hkv"], case["T"], case["D"]
    new = s["new"].cpu().numpy() if s["new"] is not None else np.full(Z, T)
    o = torch.zeros((Z, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((Z, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    if s["mask"] is None:
        trees = np.tril(np.ones((T, T), dtype=bool))[None].repeat(Z, 0)
    else:
        words = s["mask"].cpu().numpy().view(np.uint8).reshape(Z, T, -1)
        trees = np.unpackbits(words, axis=2, bitorder="little")[:, :, :T].astype(bool)
    for z in range(Z):
        n, m = int(lens[z]), int(new[z])
        ids = torch.from_numpy(table[z, :-(-(n + m) // case["page"])].astype(np.int64)).cuda()
        if m == 0:
            continue
        keys = s["k"][ids].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :n + m]
        vals = s["v"][ids].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :n + m]
        hide = torch.zeros((m, n + m), dtype=torch.bool, device="cuda")
        hide[:, n:] = torch.from_numpy(~trees[z, :m, :m]).cuda()
        for h in range(Hq):
            x = (s["q"][z, h, :m].double() @ keys[h * Hkv // Hq].T / math.sqrt(D)).masked_fill(hide, -math.inf)
            norm = torch.logsumexp(x, -1)
            lse[z, h, :m] = norm
            w = torch.where(hide, 0.0, torch.exp(x - norm.clamp(min=-1e300)[:, None]))
            o[z, h, :m] = w @ vals[h * Hkv // Hq]
    return o, lse
