"""Measured cases of the operators of a cache that is held to a budget: rotary positions (fa_rope and
rotary, forward and gradients), rotary positions of new tokens on their way into the paged cache
(fa_cache_append_rope), the attention weight that each cached position has received
(fa_cache_score), and keeping the positions that received most (fa_cache_evict).

Each operator has a plain form (elementary torch operations, fp32 where 32 bits do, rounded once) and
the call of the framework's own kernel, and `exact` states the same result in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _rope(name, Z, Hq, Hk, N, D, R, layout, scaling, dtype, train, far, packed):
    return {"name": name, "op": "rope", "Z": Z, "Hq": Hq, "Hk": Hk, "N": N, "D": D, "R": R, "layout": layout,
            "scaling": scaling, "dtype": dtype, "train": train, "far": far, "packed": packed}


def _append(name, Z, Hq, Hkv, D, R, T, lo, hi, page, layout, scaling, dtype, far, ragged):
    return {"name": name, "op": "append", "Z": Z, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "T": T, "lo": lo, "hi": hi,
            "page": page, "layout": layout, "scaling": scaling, "dtype": dtype, "far": far, "ragged": ragged}


def _score(name, Z, Hq, Hkv, D, T, lo, hi, page, dtype, decay, ragged):
    return {"name": name, "op": "score", "Z": Z, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "lo": lo, "hi": hi,
            "page": page, "dtype": dtype, "decay": decay, "ragged": ragged}


def _evict(name, Z, L, Hkv, D, lo, hi, page, budget, first, recent, dtype, shared):
    return {"name": name, "op": "evict", "Z": Z, "L": L, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "page": page,
            "budget": budget, "first": first, "recent": recent, "dtype": dtype, "shared": shared}


def listed():
    return [
        # one long document enters a model with grouped heads: the forward of one layer
        _rope("rope_document", 1, 32, 8, 32768, 128, 128, "half", "none", "bf16", False, 0, False),
        # a training step's layer: both directions through autograd
        _rope("rope_train", 4, 16, 16, 1024, 128, 128, "half", "none", "bf16", True, 0, False),
        # wide heads of which a quarter turns, neighbouring pairs, packed sequences of odd lengths, stretched context
        _rope("rope_packed", 1, 12, 2, 5003, 256, 64, "interleaved", "linear", "fp16", True, 0, True),
        # a decode step of a batch whose cache is held to a budget: positions run far ahead of the slots
        _append("append_step", 64, 32, 8, 128, 128, 1, 100, 500, 16, "half", "ramp", "bf16", 100000, False),
        # prompts of ragged lengths enter the cache
        _append("append_prompts", 5, 16, 8, 128, 64, 2011, 0, 300, 64, "interleaved", "none", "fp16", 0, True),
        # one user, one token after a short prompt: latency only
        _score("score_one", 1, 32, 8, 128, 1, 1024, 1024, 16, "bf16", 1.0, False),
        # a serving batch of ragged contexts, one token each, older weight fading
        _score("score_batch", 64, 32, 8, 128, 1, 256, 4096, 64, "bf16", 0.99, False),
        # the last 32 tokens of long prompts say what of them matters
        _score("score_window", 32, 32, 8, 128, 32, 4096, 8192, 64, "bf16", 0.0, False),
        # wide heads, an odd group, odd page and chunk sizes, contexts down to one token
        _score("score_d256", 5, 12, 2, 256, 17, 1, 2000, 48, "fp16", 1.0, True),
        # chunks of prompts, every token counted: the largest case
        _score("score_prompt", 4, 32, 8, 128, 2000, 0, 3000, 64, "bf16", 1.0, True),
        # one user's cache is cut back to its budget
        _evict("evict_one", 1, 16, 8, 128, 1200, 1200, 16, 1024, 4, 256, "bf16", False),
        # a batch, parts of whose prompts are shared, is cut back
        _evict("evict_batch", 32, 8, 8, 128, 1500, 2900, 64, 1024, 4, 128, "bf16", True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "score", "score", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 128, 128, 256])
    page = 16 * rng.choice([1, 1, 2, 3, 4, 8])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "base", "ramp"])
    R = max(16, D // rng.choice([1, 1, 2, 4]))
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 6, 8) if Hkv * g <= 32])
    far = rng.choice([0, 1000, 1000000])
    if op == "rope":
        tokens = _log_int(rng, 1, min(32768, 1.6e8 / ((Hq + Hkv) * D)))
        packed = rng.random() < 0.3
        Z = 1 if packed else _log_int(rng, 1, min(tokens, 64))
        return {"op": op, "Z": Z, "Hq": Hq, "Hk": Hkv, "N": max(1, tokens // Z), "D": D, "R": R, "layout": layout,
                "scaling": scaling, "dtype": dtype, "train": rng.random() < 0.6, "far": far, "packed": packed}
    if op == "append":
        T = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2048)
        return {"op": op, "Z": _log_int(rng, 1, max(1, min(128, 10000 // T))), "Hq": Hq, "Hkv": Hkv, "D": D, "R": R,
                "T": T, "lo": 0, "hi": rng.randint(1, 400), "page": page, "layout": layout, "scaling": scaling,
                "dtype": dtype, "far": far, "ragged": T > 1 and rng.random() < 0.6}
    if op == "score":
        T = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2048)
        hi = _log_int(rng, 16, 32768 if T <= 64 else 4096)
        # at most about the largest listed cases' cache reads, products and weights
        most = min(2e8 / (hi * Hkv * D), 8e10 / ((hi + T) * Hq * T * D), 1.2e9 / ((hi + T) * Hq * T))
        return {"op": op, "Z": max(1, min(64, _log_int(rng, 1, max(1.0, most)))), "Hq": Hq, "Hkv": Hkv, "D": D, "T": T,
                "lo": rng.randint(0, hi), "hi": hi, "page": page, "dtype": dtype, "decay": rng.choice([0.0, 0.9, 1.0]),
                "ragged": T > 1 and rng.random() < 0.5}
    hi = _log_int(rng, 40, 8000)
    Hkv = min(Hkv, 8)
    L = _log_int(rng, 1, 16)
    budget = rng.randint(max(8, hi // 8), hi)
    first = rng.randint(0, min(8, budget))
    return {"op": op, "Z": max(1, min(64, _log_int(rng, 1, max(1.0, 5e8 / (L * hi * Hkv * D))))), "L": L, "Hkv": Hkv,
            "D": D, "lo": rng.randint(1, hi), "hi": hi, "page": page, "budget": budget, "first": first,
            "recent": rng.randint(0, budget - first), "dtype": dtype, "shared": rng.random() < 0.5}


# ------------------------------------------------------------------ sizes that a case fixes for every seed

def _spread(lo, hi, Z):
    """Z lengths spread evenly over lo .. hi (their order is the seed's)."""
    return np.linspace(lo, hi, Z).round().astype(np.int64) if Z > 1 else np.array([hi])


def _new_lens(case):
    """How many of the T new tokens each sequence has."""
    return _spread((case["T"] + 1) // 2, case["T"], case["Z"]) if case["ragged"] else np.full(case["Z"], case["T"])


def _pages(tokens, page):
    return (np.asarray(tokens) + page - 1) // page


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


def _normal(gen, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        flat[i:i + (1 << 26)].normal_(0.0, scale, generator=gen)
    return out


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# Four times the context that the frequencies were made for, where it is stretched.
STRETCH, CONTEXT = 4.0, 4096


def _frequencies(case):
    """Radians a position of each pair, float64."""
    R = case["R"]
    i = torch.arange(R // 2, dtype=torch.float64)
    base, freq = 10000.0, None
    if case["scaling"] == "base" and R > 2:
        base *= STRETCH ** (R / (R - 2))
    freq = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        freq = freq / STRETCH
    if case["scaling"] == "ramp":  # pairs that turn fewer than once over the context are stretched, more than 32 times not
        stay = ((CONTEXT * freq / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        freq = freq * (stay + (1.0 - stay) / STRETCH)
    return freq


def _factor(case):
    """What both sides are multiplied by: softer scores in the stretched context."""
    return 0.1 * math.log(STRETCH) + 1.0 if case["scaling"] == "ramp" else 1.0


def _plan_rope(case, s):
    """What a model keeps of its rotary positions."""
    s["factor"], s["interleaved"] = _factor(case), case["layout"] == "interleaved"
    if own:
        import exact_attention_44_gb300 as fa
        freq = fa.fa_rope_frequencies(case["R"], scaling=case["scaling"], stretch=STRETCH, context=CONTEXT)
        s["turns"] = fa.fa_rope_turns(freq)
    else:
        s["freq"] = _frequencies(case).cuda()


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, Z, D = DTYPES[case["dtype"]], case["Z"], case["D"]
    s = {"op": case["op"]}
    if case["op"] == "rope":
        N = case["N"]
        # projections' outputs, seen as (Z, H, N, D)
        s |= {"q": _normal(gen, (Z, N, case["Hq"], D), dt).transpose(1, 2),
              "k": _normal(gen, (Z, N, case["Hk"], D), dt).transpose(1, 2), "train": case["train"]}
        at = rng.randint(0, case["far"] + 1, (Z, 1))
        pos = at + np.arange(N)
        if case["packed"]:  # sequences of odd lengths one behind the other, each from 0
            cuts = np.unique(np.concatenate([[0], rng.randint(0, N, 6)]))
            pos = (np.arange(N) - cuts[np.searchsorted(cuts, np.arange(N), side="right") - 1])[None]
        s["pos"] = _cuda(pos.astype(np.int32)) if case["packed"] or case["far"] else None
        if case["train"]:
            s["q"].requires_grad_()
            s["k"].requires_grad_()
            # gradients come back from attention as (Z, H, N, D)
            s["dq"] = _normal(gen, (Z, case["Hq"], N, D), dt)
            s["dk"] = _normal(gen, (Z, case["Hk"], N, D), dt)
        _plan_rope(case, s)
        return s
    page = s["page"] = case["page"]
    lens = rng.permutation(_spread(case["lo"], case["hi"], Z))
    s["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")  # one workspace that a serving loop keeps
    if case["op"] == "append":
        new = rng.permutation(_new_lens(case))
        table, pool = _table(rng, lens + case["T"], page, 7)
        row = (Z, case["T"])
        pos = lens[:, None] + rng.randint(0, case["far"] + 1, (Z, 1)) + np.arange(case["T"])
        shape = (pool, case["Hkv"], page, D)
        s |= {"q": _normal(gen, (*row, case["Hq"], D), dt).transpose(1, 2),
              "k_new": _normal(gen, (*row, case["Hkv"], D), dt).transpose(1, 2),
              "v_new": _normal(gen, (*row, case["Hkv"], D), dt).transpose(1, 2),
              "q_out": torch.zeros((*row, case["Hq"], D), dtype=dt, device="cuda").transpose(1, 2),
              "k": _normal(gen, shape, dt), "v": _normal(gen, shape, dt), "table": _cuda(table),
              "lens": _cuda(lens.astype(np.int32)), "new": _cuda(new.astype(np.int32)) if case["ragged"] else None,
              "pos": _cuda(pos.astype(np.int32)) if case["far"] else None}
        _plan_rope(case, s)
        return s
    if case["op"] == "score":
        new = rng.permutation(_new_lens(case))
        table, pool = _table(rng, lens + case["T"], page, 7)
        s |= {"q": _normal(gen, (Z, case["Hq"], case["T"], D), dt, 2.0),
              "k": _normal(gen, (pool, case["Hkv"], page, D), dt), "table": _cuda(table),
              "lens": _cuda(lens.astype(np.int32)), "new": _cuda(new.astype(np.int32)) if case["ragged"] else None,
              "decay": case["decay"]}
        s["lse"] = _lse(s, lens, new)
        s["scores"] = torch.empty((Z, case["Hkv"], table.shape[1] * page), dtype=torch.float32, device="cuda")
        s["scores"].exponential_(generator=gen)  # weight received so far
        return s
    table, pool = _table(rng, lens, page, 0)
    M = table.shape[1]
    if case["shared"]:  # every second sequence was forked from the one before, in the middle of the shorter one
        for z in range(1, Z, 2):
            n = int(min(lens[z - 1], lens[z])) // page // 2
            table[z, :n] = table[z - 1, :n]
    pool += int(_pages(case["budget"], page)) * Z if case["shared"] else 3
    # the bookkeeping and the scores in one piece: block table, lengths, counts, scores
    L, Hkv = case["L"], case["Hkv"]
    ints = np.concatenate([table.ravel(), lens, np.bincount(table[table >= 0], minlength=pool)]).astype(np.int32)
    books = torch.empty(len(ints) + L * Z * Hkv * M * page, dtype=torch.float32, device="cuda")
    books[:len(ints)] = _cuda(ints).view(torch.float32)
    # weight received is spread over orders of magnitude
    books[len(ints):].normal_(0.0, 2.0, generator=gen).exp_()
    shape = (L, pool, Hkv, page, D)
    s |= {"k": _normal(gen, shape, dt), "v": _normal(gen, shape, dt), "books": books, "was": books.clone(),
          "table": books[:Z * M].view(torch.int32).view(Z, M), "lens": books[Z * M:Z * M + Z].view(torch.int32),
          "refs": books[Z * M + Z:len(ints)].view(torch.int32), "scores": books[len(ints):].view(L, Z, Hkv, M * page),
          "missing": torch.zeros(1, dtype=torch.int32, device="cuda"), "budget": case["budget"],
          "first": case["first"], "recent": case["recent"]}
    if own:
        import exact_attention_44_gb300 as fa
        s["ws"] = torch.empty(fa.fa_cache_evict_workspace_size(L, Z, Hkv, M, case["budget"]), dtype=torch.uint8,
                              device="cuda")
    return s


def _rows(cache, table, z, n, page):
    """Positions 0 .. n - 1 of sequence z: (Hkv, n, D)."""
    ids = table[z, :-(-n // page)].long()
    return cache[ids].transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def _lse(s, lens, new):
    """The log-sum-exps that the attention of these tokens has left (its fp32 output)."""
    Z, Hq, T, D = s["q"].shape
    Hkv = s["k"].shape[1]
    out = torch.full((Z, Hq, T), -math.inf, dtype=torch.float32, device="cuda")
    for z in range(Z):
        n, m = int(lens[z]), int(new[z])
        keys = _rows(s["k"], s["table"], z, n + m, s["page"]).float()
        x = s["q"][z, :, :m].float().reshape(Hkv, Hq // Hkv * m, D) @ keys.transpose(1, 2) * (1 / math.sqrt(D))
        hide = torch.ones((m, n + m), dtype=torch.bool, device="cuda").triu(n + 1)
        x = x.view(Hkv, Hq // Hkv, m, n + m).masked_fill_(hide, -math.inf)
        top = x.amax(-1)
        out[z, :, :m] = (top + (x - top[..., None]).exp_().sum(-1).log()).view(Hq, m)
    return out


# ------------------------------------------------------------------ plain forms

def _plain_turn(x, pos, freq, interleaved, factor, sign):
    """The rows of x (Z, H, N, D), turned by their positions, in fp32."""
    R = 2 * freq.numel()
    angle = pos.double()[:, None, :, None] * freq * sign                    # in 64 bits: far positions
    c, sn = (angle.cos() * factor).float(), (angle.sin() * factor).float()  # (Z, 1, N, R / 2)
    y = x.float()
    if interleaved:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    return torch.cat([turned, y[..., R:]], -1).to(x.dtype)


def _plain_score(q, lse, k, table, lens, new, scores, decay, page):
    Z, Hq, T, D = q.shape
    Hkv, N = k.shape[1], table.shape[1] * page
    dev = q.device
    pos, t = torch.arange(N, device=dev), torch.arange(T, device=dev)
    nl = torch.full_like(lens, T) if new is None else new
    there = pos[None] < (lens + nl)[:, None]                                            # (Z, N)
    rows = k[table.clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(Z, Hkv, N, D).float()
    rows = torch.where(there[:, None, :, None], rows, torch.zeros((), device=dev))
    x = q.float().reshape(Z, Hkv, Hq // Hkv * T, D) @ rows.transpose(2, 3) * (1 / math.sqrt(D))
    x = x.view(Z, Hkv, Hq // Hkv, T, N) - lse.view(Z, Hkv, Hq // Hkv, T, 1)
    seen = (pos[None, None] <= (lens[:, None] + t[None])[..., None]) & there[:, None] & (t[None] < nl[:, None])[..., None]
    w = torch.where(seen[:, None, None], torch.exp(x), torch.zeros((), device=dev)).sum((2, 3))
    old = pos[None] < lens[:, None]
    before = torch.where(old[:, None], scores * decay if decay else torch.zeros((), device=dev), torch.zeros((), device=dev))
    scores.copy_(torch.where(there[:, None], before + w, scores))
    return scores


def _plain_evict(k, v, table, lens, refs, scores, budget, first, recent, missing, page):
    L, Z, H, C = scores.shape
    dev = table.device
    pos = torch.arange(C, device=dev)
    cut = lens > budget
    n = lens[None, :, None, None]
    must = (pos < first) | (pos >= n - recent)
    # candidates by score, ties to the lowest position; what must stay before them, what is not there last
    order = torch.argsort(scores, dim=-1, descending=True, stable=True)
    group = torch.where(must, 0, 1).expand(L, Z, H, C)
    group = torch.where(pos < n, group, 2).gather(3, order)
    order = order.gather(3, torch.argsort(group, dim=-1, stable=True))
    idx = order[..., :budget].sort(-1).values                                           # (L, Z, H, budget)
    i = torch.arange(idx.shape[-1], device=dev)
    moved = torch.where(idx != i, i, budget).amin((0, 2, 3))                            # (Z) first row that moves
    # pages that are rewritten belong to the sequence alone
    col = torch.arange(table.shape[1], device=dev)
    need = -(-budget // page)
    held = table.clamp(min=0).long()
    want = cut[:, None] & (col >= (moved // page)[:, None]) & (col < need) & (refs[held] > 1)
    rank = torch.cumsum(want.view(-1), 0).view_as(want) - 1
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True).to(torch.int32)      # free pages first, lowest first
    lack = (want.sum() - (refs == 0).sum()).clamp(min=0)
    missing.copy_(lack.view(1))
    cut = cut & (lack == 0)
    want = want & (lack == 0)
    after = torch.where(want, free[rank.clamp(0, refs.numel() - 1)], table)
    after = torch.where(cut[:, None] & (col >= need), -1, after)
    z = torch.nonzero(cut, as_tuple=True)[0]
    if z.numel():
        at = idx[:, z]                                                                  # (L, z, H, budget)
        fp = table[z].long()[None, :, None].expand(L, -1, H, -1).gather(3, at // page)
        tp = after[z].long()[None, :, None].expand(L, -1, H, -1).gather(3, (i // page).expand_as(at))
        la, h = torch.arange(L, device=dev)[:, None, None, None], torch.arange(H, device=dev)[None, None, :, None]
        for c in (k, v):
            c[la, tp, h, i % page] = c[la, fp, h, at % page]
        scores[:, z, :, :idx.shape[-1]] = scores[:, z].gather(3, at)
    change = torch.zeros(refs.numel() + 1, dtype=torch.int32, device=dev)
    for t, by in ((table, -1), (after, 1)):
        t = torch.where(t < 0, refs.numel(), t).view(-1).long()
        change.index_add_(0, t, torch.full_like(t, by, dtype=torch.int32))
    refs += change[:-1]
    table.copy_(after)
    lens.copy_(torch.where(cut, budget, lens))
    return k, v, table, lens, refs, scores, missing


def run(s):
    if own:
        import exact_attention_44_gb300 as fa
    if s["op"] == "rope":
        q, k = s["q"], s["k"]
        if own:
            kw = {"interleaved": s["interleaved"], "factor": s["factor"]}
            if not s["train"]:
                return fa.fa_rope(q, k, s["turns"], s["pos"], **kw)
            y = fa.rotary(q, k, s["turns"], s["pos"], **kw)
            return (*y, *torch.autograd.grad(y, (q, k), (s["dq"], s["dk"])))
        pos = torch.arange(q.shape[2], device=q.device)[None] if s["pos"] is None else s["pos"]
        turn = lambda x, sign: _plain_turn(x, pos, s["freq"], s["interleaved"], s["factor"], sign)  # noqa: E731
        with torch.no_grad():
            y = turn(q, 1), turn(k, 1)
            # the gradient of a turn is the turn back
            return (*y, turn(s["dq"], -1), turn(s["dk"], -1)) if s["train"] else y
    if s["op"] == "append":
        if own:
            fa.fa_cache_append_rope(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], s["turns"],
                                    positions=s["pos"], new_lens=s["new"], interleaved=s["interleaved"],
                                    factor=s["factor"], q_out=s["q_out"])
            return s["q_out"], s["k"], s["v"]
        T = s["q"].shape[2]
        t = torch.arange(T, device=s["k"].device)
        slot = s["lens"][:, None] + t[None]
        pos = slot if s["pos"] is None else s["pos"]
        z, i = torch.nonzero(t[None] < (torch.full_like(s["lens"], T) if s["new"] is None else s["new"])[:, None],
                             as_tuple=True)
        at = s["table"][z, slot[z, i] // s["page"]].long(), slot[z, i] % s["page"]
        turn = lambda x: _plain_turn(x, pos, s["freq"], s["interleaved"], s["factor"], 1)  # noqa: E731
        s["q_out"][z, :, i] = turn(s["q"])[z, :, i]
        s["k"][at[0], :, at[1]] = turn(s["k_new"])[z, :, i]
        s["v"][at[0], :, at[1]] = s["v_new"][z, :, i]
        return s["q_out"], s["k"], s["v"]
    if s["op"] == "score":
        if own:
            fa.fa_cache_score(s["q"], s["lse"], s["k"], s["table"], s["lens"], s["scores"], new_lens=s["new"],
                              decay=s["decay"], workspace=s["ws"])
            return s["scores"]
        return _plain_score(s["q"], s["lse"], s["k"], s["table"], s["lens"], s["new"], s["scores"], s["decay"], s["page"])
    # the sequences have grown again since they were last cut (their tokens and scores as then)
    s["books"].copy_(s["was"])
    if own:
        fa.fa_cache_evict(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["scores"], s["budget"], s["missing"],
                          first=s["first"], recent=s["recent"], workspace=s["ws"])
        return s["k"], s["v"], s["table"], s["lens"], s["refs"], s["scores"], s["missing"]
    return _plain_evict(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["scores"], s["budget"], s["first"],
                        s["recent"], s["missing"], s["page"])


# ------------------------------------------------------------------ what the path cannot do without

def work(case):
    Z, D = case["Z"], case["D"]
    if case["op"] == "rope":
        rows = Z * case["N"] * (case["Hq"] + case["Hk"]) * (2 if case["train"] else 1)
        pos = 4 * Z * case["N"] if case["packed"] or case["far"] else 0
        return {"bytes": rows * D * 4 + pos + 4 * case["R"], "flops": rows * case["R"] * 3}
    lens, page = _spread(case["lo"], case["hi"], Z), case["page"]
    if case["op"] == "append":
        n = float(_new_lens(case).sum())
        return {"bytes": n * (case["Hq"] + 2 * case["Hkv"]) * D * 4 + 4 * n / page + 8 * Z + 4 * case["R"] +
                (4 * n if case["far"] else 0), "flops": n * (case["Hq"] + case["Hkv"]) * case["R"] * 3}
    if case["op"] == "score":
        new = _new_lens(case)
        cached, rows = float((lens + new).sum()), float(new.sum()) * case["Hq"]
        # (which new length meets which cached one is the seed's: means)
        pairs = rows * float(lens.mean() + (new.mean() + 1) / 2)
        return {"bytes": cached * case["Hkv"] * (D * 2 + 4) + rows * (D * 2 + 4) +
                (4 * float(lens.sum()) * case["Hkv"] if case["decay"] else 0) + 4 * float(_pages(lens + new, page).sum()),
                "flops": 2.0 * pairs * D}
    cut = lens > case["budget"]
    heads, kept = case["L"] * case["Hkv"], case["budget"] - case["first"]
    return {"bytes": max(16.0, float(cut.sum()) * heads * kept * (D * 2 * 4 + 4) + 4.0 * heads * float(lens[cut].sum()) +
                         8.0 * float(_pages(lens, page).sum())) + 8.0 * case["Z"] * heads * case["hi"], "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_turn(x, pos, case, sign):
    """Pairs as complex numbers, each times e^(i position frequency)."""
    R, x = case["R"], x.detach().double()
    wave = torch.polar(torch.full((R // 2,), _factor(case), dtype=torch.float64, device=x.device)[None, None],
                       sign * pos.double()[..., None] * _frequencies(case).to(x.device))[:, None]
    out = x.clone()
    pairs = (slice(0, R, 2), slice(1, R, 2)) if case["layout"] == "interleaved" else (slice(0, R // 2), slice(R // 2, R))
    turned = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * wave
    out[..., pairs[0]], out[..., pairs[1]] = turned.real, turned.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        pos = torch.arange(case["N"], device="cuda").expand(case["Z"], -1) if s["pos"] is None else s["pos"]
        out = [_exact_turn(s["q"], pos, case, 1), _exact_turn(s["k"], pos, case, 1)]
        return (*out, _exact_turn(s["dq"], pos, case, -1), _exact_turn(s["dk"], pos, case, -1)) if case["train"] else tuple(out)
    page, Z = case["page"], case["Z"]
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    if case["op"] == "evict":
        return _exact_evict(case, s, table, lens)
    new = s["new"].cpu().numpy() if s["new"] is not None else np.full(Z, case["T"])
    if case["op"] == "append":
        q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
        for z in range(Z):
            n, m = int(lens[z]), int(new[z])
            pos = torch.arange(n, n + m, device="cuda")[None] if s["pos"] is None else s["pos"][z:z + 1, :m]
            q[z, :, :m] = _exact_turn(s["q"][z:z + 1, :, :m], pos, case, 1)[0]
            turned = _exact_turn(s["k_new"][z:z + 1, :, :m], pos, case, 1)[0]
            for p in range(n // page, -(-(n + m) // page)):
                a, b = max(n, p * page), min(n + m, (p + 1) * page)
                k[table[z, p], :, a - p * page:b - p * page] = turned[:, a - n:b - n]
                v[table[z, p], :, a - p * page:b - p * page] = s["v_new"][z, :, a - n:b - n].double()
        return q, k, v
    Hkv, G, D = case["Hkv"], case["Hq"] // case["Hkv"], case["D"]
    out = s["scores"].double()
    for z in range(Z):
        n, m = int(lens[z]), int(new[z])
        out[z, :, :n] *= case["decay"]
        out[z, :, n:n + m] = 0.0
        keys = _rows(s["k"], s["table"], z, n + m, page).double()
        hide = torch.arange(n + m, device="cuda")[None] > n + torch.arange(m, device="cuda")[:, None]
        for h in range(Hkv * G):
            x = s["q"][z, h, :m].double() @ keys[h // G].T / math.sqrt(D) - s["lse"][z, h, :m, None].double()
            out[z, h // G, :n + m] += torch.exp(x).masked_fill(hide, 0.0).sum(0)
    return out


def _exact_evict(case, s, table, lens):
    """One (layer, sequence, head) after the other on the host; the rows are copied a sequence at a time."""
    L, Z, H, page, B = case["L"], case["Z"], case["Hkv"], case["page"], case["budget"]
    refs, scores = s["refs"].cpu().numpy().copy(), s["scores"].cpu().numpy().copy()
    was, keep, wants = table.copy(), {}, []
    for z in range(Z):
        n = int(lens[z])
        if n <= B:
            continue
        r = min(case["recent"], B - case["first"])
        middle = np.arange(case["first"], n - r)
        stay = np.concatenate([np.arange(case["first"]), np.arange(n - r, n)])
        idx = np.empty((L, H, B), dtype=np.int64)
        for a in range(L):
            for h in range(H):
                best = middle[np.argsort(-scores[a, z, h, middle], kind="stable")[:B - len(stay)]]
                idx[a, h] = np.sort(np.concatenate([stay, best]))
        keep[z] = idx
        still = (idx == np.arange(B)).all((0, 1))
        first = B if still.all() else int(np.argmin(still))
        wants += [(z, c) for c in range(first // page, -(-B // page)) if refs[table[z, c]] > 1]
    free = np.flatnonzero(refs == 0)
    missing = max(0, len(wants) - len(free))
    whole = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32))  # noqa: E731
    k, v = s["k"], s["v"]
    if missing == 0:
        for (z, c), p in zip(wants, free):
            refs[table[z, c]] -= 1
            refs[p] += 1
            table[z, c] = p
        for z, idx in keep.items():
            for c in range(-(-B // page), table.shape[1]):
                if table[z, c] >= 0:
                    refs[table[z, c]] -= 1
                    table[z, c] = -1
            lens[z] = B
            at = _cuda(idx)
            for a in range(L):
                for cache in (k, v):
                    # (no page that a sequence reads is written by another one)
                    rows = _rows(cache[a], _cuda(was), z, was.shape[1] * page, page)
                    rows = rows.gather(1, at[a][..., None].expand(-1, -1, case["D"]))
                    for c in range(-(-B // page)):
                        part = rows[:, c * page:(c + 1) * page]
                        cache[a, table[z, c], :, :part.shape[1]] = part
                for h in range(H):
                    scores[a, z, h, :B] = scores[a, z, h, idx[a, h]]
    return k, v, whole(table), whole(lens), whole(refs), torch.from_numpy(scores), whole([missing])
