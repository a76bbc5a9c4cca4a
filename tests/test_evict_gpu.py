"""Cutting a cache back to its best positions: rows, scores and books bit by bit against a plain statement, and a
run of it with the calls around it."""
import math

import numpy as np
import pytest
import torch

import budget_util as bu
import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16).cpu()


def state(seed, lens, page, Hkv, D, L, *, extra=5, cols=None, dtype="fp16", layout="phnd", share=(), room=0):
    """share: (z, y, pages): sequence z holds the first pages of y."""
    kc, vc, table, _, _ = pu.make_cache(seed, lens, Hkv, D, page, dtype, layers=L, extra=extra, cols=cols, garbage=3.0,
                                        layout=layout)
    for z, y, n in share:
        table[z, :n] = table[y, :n]
    refs = np.bincount(table[table >= 0].numpy(), minlength=kc.shape[-4]).tolist()
    return kc, vc, table, refs


def check(kc, vc, table, lens, refs, scores, page, budget, *, keep=None, first=0, recent=0, pad=0):
    """One call against the statement; returns what lacked."""
    import exact_attention_44_gb300 as fa
    layers = kc.dim() == 5
    c5 = [c if layers else c[None] for c in (kc, vc)]
    s4 = scores if layers else scores[None]
    t, n, r, lack, kept = bu.evict(table.tolist(), lens, refs, s4.double().numpy(), page, budget, keep, first, recent)
    kg, vg, tg, lg, rg, missing = pu.like(kc), pu.like(vc), table.cuda(), i32(lens), i32(refs), i32([-1])
    held = torch.full((*scores.shape[:-1], scores.shape[-1] + pad), 77.0, device="cuda")
    sg = held[..., :scores.shape[-1]]
    sg.copy_(scores)
    fa.fa_cache_evict(kg, vg, tg, lg, rg, sg, budget, missing, keep=None if keep is None else i32(keep), first=first,
                      recent=recent)
    assert fa.fa_device_status()[0] == 0
    assert missing.item() == lack and tg.tolist() == t and lg.tolist() == n and rg.tolist() == r
    s4 = s4.clone()
    for z, idx in enumerate(kept):
        if idx is not None:
            i = torch.from_numpy(idx)
            s4[:, z, :, :i.shape[2]] = s4[:, z].gather(2, i)
    assert torch.equal(bits(sg), bits(s4 if layers else s4[0])) and (held[..., scores.shape[-1]:] == 77).all()
    for got, c in zip((kg, vg), c5):
        bu.move(c, table.tolist(), t, kept, page)
        assert torch.equal(bits(got), bits(c if layers else c[0]))
    return lack


@pytest.mark.parametrize("D,L,page", [(16, 1, 16), (32, None, 48), (64, 3, 16), (128, 2, 48), (256, 1, 32)])
@pytest.mark.parametrize("budget,first,recent", [(0, 0, 0), (1, 0, 0), (20, 4, 5), (33, 0, 40), (64, 100, 0), (64, 0, 64),
                                                 (50, 0, 0), (200, 3, 3)])
def test_evict(D, L, page, budget, first, recent):
    lens = [0, 1, 33, 64, 65, 150, 200]
    kc, vc, table, refs = state(D, lens, page, 2, D, L)
    g = torch.Generator().manual_seed(budget)
    shape = (len(lens), 2, table.shape[1] * page)
    scores = torch.randn(shape if L is None else (L, *shape), generator=g).exp()
    check(kc, vc, table, lens, refs, scores, page, budget, first=first, recent=recent)


@pytest.mark.parametrize("layout", ["phnd", "pnhd", "padded"])
def test_layouts(layout):
    lens = [100, 47]
    kc, vc, table, refs = state(3, lens, 16, 3, 64, 2, layout=layout)
    check(kc, vc, table, lens, refs, torch.rand(2, 2, 3, table.shape[1] * 16), 16, 30, first=2, recent=7, pad=8)


def test_ties_and_special_values():
    lens = [300] * 5
    kc, vc, table, refs = state(4, lens, 16, 1, 16, 1)
    s = torch.zeros(1, 5, 1, table.shape[1] * 16)
    r = np.random.RandomState(1)
    s[0, 0, 0, :300] = torch.from_numpy(r.randint(0, 3, 300).astype(np.float32))
    s[0, 1] = 1.0                                                  # all alike: the lowest stay
    s[0, 2, 0, :300] = torch.from_numpy(r.choice([0.0, -0.0, 1e-45, -1e-45], 300).astype(np.float32))
    s[0, 3, 0, :300] = torch.from_numpy(r.choice([np.inf, -np.inf, np.nan, 3e38, -3e38], 300).astype(np.float32))
    s[0, 4, 0, :300] = torch.from_numpy(-np.abs(r.randn(300)).astype(np.float32))
    for budget in (100, 150, 299):
        check(*[c.clone() for c in (kc, vc)], table, lens, refs, s, 16, budget, recent=10)


def test_keep_for_each_sequence():
    lens = [100, 100, 100, 100, 30, 0]
    kc, vc, table, refs = state(5, lens, 16, 2, 64, 2)
    s = torch.rand(2, 6, 2, table.shape[1] * 16)
    check(kc, vc, table, lens, refs, s, 16, 60, keep=[-1, 0, 50, 99, 10, 5], first=1, recent=20)


def test_long_sequences():
    """More candidates than are held in shared memory, and many equal ones."""
    lens = [20000, 9000]
    kc, vc, table, refs = state(6, lens, 128, 1, 16, 1)
    s = torch.randn(1, 2, 1, table.shape[1] * 128).exp()
    s[0, 1] = s[0, 1].round()
    check(kc, vc, table, lens, refs, s, 128, 8500, first=4, recent=100)


def test_many_sequences():
    r = np.random.RandomState(7)
    lens = r.randint(0, 50, 1100).tolist()
    kc, vc, table, refs = state(7, lens, 16, 1, 16, 1, extra=40, share=[(z, z - 1, 1) for z in range(1, 60, 2)
                                                                       if min(lens[z], lens[z - 1]) > 16])
    check(kc, vc, table, lens, refs, torch.rand(1, 1100, 1, table.shape[1] * 16), 16, 20, first=1)


@pytest.mark.parametrize("extra,lacks", [(20, False), (3, True)])
def test_shared_pages(extra, lacks):
    """Forked sequences: pages that are rewritten become the sequence's own, unless too few are free; then nothing
    changes."""
    lens = [150, 140, 130, 40]
    kc, vc, table, refs = state(8, lens, 16, 2, 64, 2, extra=extra, share=[(1, 0, 8), (2, 0, 5), (3, 0, 2)])
    # (pages that the copies held before are free too)
    held = set(table[table >= 0].tolist())
    if lacks:
        refs = [c if p in held else 1 for p, c in enumerate(refs)]
        spare = [p for p in range(len(refs)) if p not in held][:3]
        for p in spare:
            refs[p] = 0
    s = torch.rand(2, 4, 2, table.shape[1] * 16)
    lack = check(kc, vc, table, lens, refs, s, 16, 60, first=20, recent=10)
    assert (lack > 0) == lacks


def test_shared_pages_that_stay():
    """The first pages stay whole in every head: they go on being shared; the last one, partly filled after the cut,
    does not, even where no row of it moves."""
    lens = [100, 100]
    kc, vc, table, refs = state(9, lens, 16, 2, 64, 1, extra=3, share=[(1, 0, 6)])
    s = torch.arange(table.shape[1] * 16, 0, -1).float().expand(1, 2, 2, -1).contiguous()  # the oldest are best
    check(*[c.clone() for c in (kc, vc)], table, lens, refs, s, 16, 56)
    check(*[c.clone() for c in (kc, vc)], table, lens, refs, s, 16, 48)  # whole pages: nothing is copied


def test_room_is_released_and_bad_pages_are_reported():
    import exact_attention_44_gb300 as fa
    lens = [70, 70]
    kc, vc, table, refs = state(10, [96, 96], 16, 1, 64, 1)
    s = torch.rand(1, 2, 1, table.shape[1] * 16)
    check(*[c.clone() for c in (kc, vc)], table, lens, refs, s, 16, 40)
    bad = table.clone()
    bad[0, 1], bad[1, 3] = -1, 9999
    s[0, :, 0] = torch.arange(table.shape[1] * 16)
    kg, tg, lg, rg, m = kc.cuda(), bad.cuda(), i32(lens), i32(refs), i32([0])
    fa.fa_cache_evict(kg, vc.cuda(), tg, lg, rg, s.cuda(), 40, m)
    assert fa.fa_device_status()[0] == fa.FA_ERR_PAGE
    assert lg.tolist() == [40, 40] and m.item() == 0
    want = kc[0].clone()
    for z in range(2):
        for i in range(40):
            f, t = bad[z, (i + 30) // 16], bad[z, i // 16]
            if 0 <= f < kc.shape[1] and 0 <= t < kc.shape[1]:
                want[t, :, i % 16] = kc[0, f, :, (i + 30) % 16]
    assert torch.equal(bits(kg[0]), bits(want))


def test_wide_tables():
    """Far more columns than the sequences need, room in some of them."""
    lens = [100, 7, 260]
    kc, vc, table, refs = state(14, [160, 16, 300], 16, 2, 64, 2, cols=3001)
    check(kc, vc, table, lens, refs, torch.rand(2, 3, 2, table.shape[1] * 16), 16, 50, first=1, recent=9)


def test_nothing_to_do():
    import exact_attention_44_gb300 as fa
    kc, vc, table, refs = state(11, [30, 5], 16, 1, 64, 1)
    s = torch.rand(1, 2, 1, table.shape[1] * 16)
    check(kc, vc, table, [30, 5], refs, s, 16, 30)
    check(kc, vc, table, [30, 5], refs, s, 16, 2 ** 31 - 1, first=2 ** 31 - 1, recent=2 ** 31 - 1)
    m = i32([5])
    fa.fa_cache_evict(kc[:, :0].cuda(), vc[:, :0].cuda(), table.cuda(), i32([0, 0]), i32([]), s.cuda(), 3, m)
    assert m.item() == 0
    m.fill_(5)
    fa.fa_cache_evict(kc.cuda(), vc.cuda(), table[:0].cuda(), i32([]), i32(refs), s[:, :0].cuda(), 3, m)
    assert m.item() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_bounded_serving_run(dtype):
    """Prompts, then decode steps over a cache held to a budget: turned rows in, attention, received weight, eviction
    every few steps.  Each step's attention and scores are checked against what each layer and head should hold, and
    the same steps replayed from one captured graph end in the same bits."""
    import exact_attention_44_gb300 as fa
    Z, L, Hq, Hkv, D, page, steps, budget = 4, 2, 6, 2, 64, 16, 9, 40
    P, M = 60, 6
    dt = pu.DT[dtype]
    g = torch.Generator().manual_seed(13)
    kc = torch.full((L, P, Hkv, page, D), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    table, lens, refs = torch.full((Z, M), -1, dtype=torch.int32, device="cuda"), i32([0] * Z), i32([0] * P)
    missing, positions = i32([0]), i32([0] * Z)
    scores = torch.full((L, Z, Hkv, M * page), float("nan"), device="cuda")
    freq = bu.frequencies(32)
    turns = turns = fa.fa_rope_turns(torch.from_numpy(freq))
    T0, n0 = 50, [50, 12, 33, 1]
    q, k, v = (torch.randn(L, Z, h, T0, D, generator=g).to(dt).cuda() for h in (Hq, Hkv, Hkv))
    fa.fa_cache_fork(kc, vc, table, lens, refs, room=T0 + 2, missing=missing)
    for la in range(L):
        tq = fa.fa_cache_append_rope(q[la], k[la], v[la], kc[la], vc[la], table, lens, turns, new_lens=i32(n0))
        _, lse = fa.fa_fwd_paged(tq, kc[la], vc[la], table, lens, new_lens=i32(n0))
        fa.fa_cache_score(tq, lse, kc[la], table, lens, scores[la], new_lens=i32(n0))
    lens += i32(n0)
    positions += i32(n0)

    def held(z, la, cache, n):
        ids = table[z, :pu.cdiv(n, page)].long()
        return cache[la, ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double().cpu().numpy()

    # what each sequence holds: turned K rows as they were written, V rows
    for la in range(L):
        tk, _ = fa.fa_rope(k[la], None, turns)
        for z in range(Z):
            assert np.array_equal(held(z, la, kc, n0[z]), tk[z, :, :n0[z]].double().cpu().numpy())
            assert np.array_equal(held(z, la, vc, n0[z]), v[la][z, :, :n0[z]].double().cpu().numpy())
    buf = dict(q=torch.zeros(L, Z, Hq, 1, D, dtype=dt, device="cuda"), k=torch.zeros(L, Z, Hkv, 1, D, dtype=dt, device="cuda"),
               v=torch.zeros(L, Z, Hkv, 1, D, dtype=dt, device="cuda"), keep=i32([-1] * Z),
               tq=torch.zeros(L, Z, Hq, 1, D, dtype=dt, device="cuda"), o=torch.zeros(L, Z, Hq, 1, D, dtype=dt, device="cuda"),
               lse=torch.zeros(L, Z, Hq, 1, device="cuda"), lacks=i32([0]))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        fa.fa_fwd_paged_workspace_size(D), fa.fa_cache_score_workspace_size(), fa.fa_cache_evict_workspace_size(L, Z, Hkv, M, budget))]

    def step():
        fa.fa_cache_fork(kc, vc, table, lens, refs, room=1, missing=missing, all_or_nothing=True)
        for la in range(L):
            fa.fa_cache_append_rope(buf["q"][la], buf["k"][la], buf["v"][la], kc[la], vc[la], table, lens, turns,
                                    positions=positions[:, None], factor=1.25, q_out=buf["tq"][la])
            fa.fa_fwd_paged(buf["tq"][la], kc[la], vc[la], table, lens, buf["o"][la], buf["lse"][la], workspace=ws[0])
            fa.fa_cache_score(buf["tq"][la], buf["lse"][la], kc[la], table, lens, scores[la], decay=0.875, workspace=ws[1])
        lens.add_(1)
        positions.add_(1)
        fa.fa_cache_evict(kc, vc, table, lens, refs, scores, budget, buf["lacks"], keep=buf["keep"], first=2, recent=4,
                          workspace=ws[2])

    names = (kc, vc, table, lens, refs, positions, scores)
    start = [t.clone() for t in names]
    plans = [[torch.randn(L, Z, h, 1, D, generator=g).to(dt) for h in (Hq, Hkv, Hkv)] +
             [[budget if s % 3 == 1 else -1 for _ in range(Z)]] for s in range(steps)]

    def fill(plan):
        for name, x in zip(("q", "k", "v"), plan[:3]):
            buf[name].copy_(x)
        buf["keep"].copy_(i32(plan[3]))

    ends = []
    scale = 1 / math.sqrt(D)
    for plan in plans:
        fill(plan)
        n = lens.tolist()
        was = [[held(z, la, c, n[z]) for z in range(Z)] for la in range(L) for c in (kc, vc)]
        s_was, seen = scores.clone(), positions.tolist()
        step()
        assert fa.fa_device_status()[0] == 0 and missing.item() == 0 and buf["lacks"].item() == 0
        s_now = torch.zeros(L, Z, Hkv, M * page, dtype=torch.float64)
        tol = np.zeros((L, Z, Hkv, M * page))
        rows = []
        for la in range(L):
            at = np.array(seen)[:, None]
            tq, sq = bu.turn(plan[0][la].double().numpy(), at, freq, False, 1.25)
            got_q = buf["tq"][la].double().cpu().numpy()
            assert (np.abs(got_q - tq) <= bu.turn_bound(tq, sq, dtype, 1.25, 100)).all()
            tk, _ = fa.fa_rope(plan[1][la].cuda(), None, turns, positions=i32(seen)[:, None], factor=1.25)
            ks = [np.concatenate([was[2 * la][z], tk[z].double().cpu().numpy()], 1) for z in range(Z)]
            vs = [np.concatenate([was[2 * la + 1][z], plan[2][la][z].double().numpy()], 1) for z in range(Z)]
            rows.append((ks, vs))
            want, wl = pu.attention(got_q, ks, vs, n, [1] * Z, None, scale)
            to, tl = pu.tolerances(got_q, ks, vs, dtype, scale)
            assert np.abs(buf["o"][la].double().cpu().numpy() - want).max() <= to
            assert np.abs(buf["lse"][la].double().cpu().numpy() - wl).max() <= tl
            sc, b = bu.score(got_q, buf["lse"][la].double().cpu().numpy(), ks, n, [1] * Z,
                             np.nan_to_num(s_was[la].double().cpu().numpy()), 0.875, scale)
            s_now[la], tol[la] = torch.from_numpy(sc), b
        # which positions stayed: by the kernel's own scores, which the next lines check
        cut = [plan[3][z] >= 0 and n[z] + 1 > budget for z in range(Z)]
        got_s = scores.double().cpu()
        for z in range(Z):
            m = budget if cut[z] else n[z] + 1
            assert lens[z].item() == m
            for la in range(L):
                kz, vz = held(z, la, kc, m), held(z, la, vc, m)
                for h in range(Hkv):
                    full = rows[la][0][z][h]
                    idx = [int(np.argmin(np.abs(full - kz[h, i]).sum(1))) for i in range(m)]  # rows are all different
                    assert idx == sorted(set(idx)) and np.array_equal(full[idx], kz[h])
                    assert np.array_equal(rows[la][1][z][h][idx], vz[h])
                    assert idx[:2] == [0, 1][:m] and idx[-1] == n[z]
                    have, want = got_s[la, z, h, :m].numpy(), s_now[la, z, h, idx].numpy()
                    assert (np.abs(have - want) <= tol[la, z, h, idx]).all()
                    if cut[z]:
                        assert idx[-4:] == list(range(n[z] - 3, n[z] + 1))
                        gone = [j for j in range(n[z] + 1) if j not in idx]
                        low = min(s_now[la, z, h, j].item() for j in idx[2:-4])
                        high = max(s_now[la, z, h, j].item() for j in gone)
                        assert high <= low + 2 * tol[la, z, h].max()
        held_pages = table[table >= 0].cpu().numpy()
        assert np.bincount(held_pages, minlength=P).tolist() == refs.tolist()
        ends.append((buf["o"].clone(), buf["lse"].clone(), table.clone()))
    assert any(all(x >= 0 for x in p[3]) for p in plans) and max(lens.tolist()) <= budget + 3
    final = [t.clone() for t in names]

    def back():
        for t, w in zip(names, start):
            t.copy_(w)

    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    back()
    for plan, (o, lse, t) in zip(plans, ends):
        fill(plan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf["o"], o) and torch.equal(buf["lse"], lse) and torch.equal(table, t)
    for t, w in zip(names, final):
        if t.dtype in (torch.float16, torch.bfloat16, torch.float32):
            assert torch.equal(bits(t), bits(w))
        else:
            assert torch.equal(t, w)
