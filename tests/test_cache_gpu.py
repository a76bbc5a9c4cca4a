"""The paged cache's own operations against plain statements: append, commit and fork bit by bit,
and a run of them with the attention that reads the cache."""
import math

import numpy as np
import pytest
import torch

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
    return t.contiguous().view(torch.int16).cpu()


@pytest.mark.parametrize("D", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T,page", [(1, 16), (5, 48), (70, 32)])
@pytest.mark.parametrize("layout", ["phnd", "pnhd", "padded"])
def test_append(D, T, page, layout):
    import exact_attention_44_gb300 as fa
    lens, new = [0, 1, page - 1, page, 100], [T, 0, T, 1, max(0, T - 2)]
    kc, vc, table, _, _ = pu.make_cache(1, [a + T for a in lens], 3, D, page, "fp16", layout=layout, garbage=7.0)
    rows = [torch.randn(5, T, 3, D).half().transpose(1, 2) for _ in range(2)]
    kg, vg = pu.like(kc), pu.like(vc)
    fa.fa_cache_append(rows[0].cuda(), rows[1].cuda(), kg, vg, table.cuda(), i32(lens), new_lens=i32(new))
    assert fa.fa_device_status()[0] == 0
    for z in range(5):
        for t in range(new[z]):
            p, s = divmod(lens[z] + t, page)
            kc[table[z, p], :, s] = rows[0][z, :, t]
            vc[table[z, p], :, s] = rows[1][z, :, t]
    assert torch.equal(bits(kg), bits(kc)) and torch.equal(bits(vg), bits(vc))


def test_append_bad_pages_and_full_tables():
    import exact_attention_44_gb300 as fa
    kc, vc, table, _, _ = pu.make_cache(2, [40, 40, 40], 2, 64, 16, "bf16", garbage=1.0)
    table[0, 1], table[1, 1] = -1, 5000
    rows = torch.randn(3, 2, 20, 64).bfloat16()
    kg, vg = kc.cuda(), vc.cuda()
    lens = [16, 10, 45]  # the third's table ends at 48
    fa.fa_cache_append(rows.cuda(), rows.cuda(), kg, vg, table.cuda(), i32(lens))
    assert fa.fa_device_status()[0] == fa.FA_ERR_PAGE
    for z in range(3):
        for t in range(20):
            p, s = divmod(lens[z] + t, 16)
            if p < table.shape[1] and 0 <= table[z, p] < kc.shape[0]:
                kc[table[z, p], :, s] = rows[z, :, t]
                vc[table[z, p], :, s] = rows[z, :, t]
    assert torch.equal(bits(kg), bits(kc)) and torch.equal(bits(vg), bits(vc))


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("L", [None, 1, 3])
@pytest.mark.parametrize("layout", ["phnd", "pnhd", "padded"])
def test_commit(D, L, layout):
    import exact_attention_44_gb300 as fa
    page, T, A = 16, 40, 20
    lens = [0, 3, 15, 16, 77, 30]
    kc, vc, table, _, _ = pu.make_cache(3, [a + T for a in lens], 2, D, page, "bf16", layout=layout, layers=L,
                                        garbage=2.0)
    r = np.random.RandomState(4)
    kept = [A, 1, 0, 9, 8, 20]
    path = np.zeros((6, A), dtype=np.int32)
    for z in range(6):
        path[z, :kept[z]] = np.sort(r.permutation(T)[:kept[z]])
    path[5] = np.arange(20)          # everything stays
    path[0] = np.arange(20, 40)      # everything moves
    path[4, :8] = np.arange(1, 9)    # each row takes its neighbour's place
    kg, vg = pu.like(kc), pu.like(vc)
    fa.fa_cache_commit(kg, vg, table.cuda(), i32(lens), i32(path.tolist()), i32(kept))
    assert fa.fa_device_status()[0] == 0
    for c in (kc, vc):
        c5 = c if L is not None else c[None]
        was = c5.clone()
        for z in range(6):
            for i in range(kept[z]):
                a, b = divmod(lens[z] + int(path[z, i]), page), divmod(lens[z] + i, page)
                c5[:, table[z, b[0]], :, b[1]] = was[:, table[z, a[0]], :, a[1]]
    assert torch.equal(bits(kg), bits(kc)) and torch.equal(bits(vg), bits(vc))


def test_commit_bad_pages_and_positions():
    import exact_attention_44_gb300 as fa
    kc, vc, table, _, _ = pu.make_cache(5, [40, 40], 2, 64, 16, "bf16", garbage=2.0)
    table[0, 2] = 9999
    kg, vg = kc.cuda(), vc.cuda()
    path = [[0, 4, 10 ** 9, 2 ** 31 - 1], [-3, 2, 5, 7]]
    fa.fa_cache_commit(kg, vg, table.cuda(), i32([30, 10]), i32(path), i32([4, 1]))
    assert fa.fa_device_status()[0] == fa.FA_ERR_PAGE
    kc[table[1, 0], :, 10] = kc[table[1, 0], :, 7].clone()  # -3 is position 7: inside, so it is moved
    assert torch.equal(bits(kg), bits(kc))


def fork_state(seed, lens, page, Hkv, D, L, extra, cols, room=0):
    kc, vc, table, _, _ = pu.make_cache(seed, lens, Hkv, D, page, "fp16", layers=L, extra=extra, cols=cols, garbage=3.0)
    refs = np.bincount(table[table >= 0].numpy(), minlength=kc.shape[1]).tolist()
    return kc, vc, table, refs


def check_fork(kc, vc, table, lens, refs, source, room, page):
    """One call against the statement; returns the new state (CPU)."""
    import exact_attention_44_gb300 as fa
    kg, vg, tg, lg, rg = pu.like(kc), pu.like(vc), table.cuda(), i32(lens), i32(refs)
    missing = i32([-1])
    fa.fa_cache_fork(kg, vg, tg, lg, rg, None if source is None else i32(source), room=room, missing=missing)
    assert fa.fa_device_status()[0] == 0
    t, n, r, m, tails = pu.fork(table.tolist(), lens, refs, source, room, page)
    assert tg.tolist() == t and lg.tolist() == n and rg.tolist() == r and missing.item() == m
    for c in (kc, vc):
        was = c.clone()
        for a, b, rows in tails:
            c[:, b, :, :rows] = was[:, a, :, :rows]
    assert torch.equal(bits(kg), bits(kc)) and torch.equal(bits(vg), bits(vc))
    return kc, vc, torch.tensor(t, dtype=torch.int32), n, r


@pytest.mark.parametrize("D,L,page", [(16, 1, 16), (64, 3, 16), (128, 2, 48), (256, 1, 32)])
@pytest.mark.parametrize("room", [0, 1, 50])
def test_fork(D, L, page, room):
    lens = [33, 0, 16, 17, 100, 1, 48, 96]
    state = fork_state(6, lens, page, 2, D, L, 60, pu.cdiv(160, page))
    kc, vc, table, refs = state
    # a beam swap (0 <-> 3), copies of one (4 twice), of an empty one, an ended one, one that stays
    kc, vc, table, lens, refs = check_fork(kc, vc, table, lens, refs, [3, 4, 2, 0, 4, 1, -1, 4], room, page)
    kc, vc, table, lens, refs = check_fork(kc, vc, table, lens, refs, None, room + 3, page)
    kc, vc, table, lens, refs = check_fork(kc, vc, table, lens, refs, [7, 7, 7, 7, 7, 7, 7, 7], room, page)
    kc, vc, table, lens, refs = check_fork(kc, vc, table, lens, refs, [-1] * 8, room, page)
    assert set(refs) == {0} and lens == [0] * 8 and (table == -1).all()


def test_fork_runs_out_of_pages_and_columns():
    lens = [30, 20, 5, 64]
    kc, vc, table, refs = fork_state(7, lens, 16, 1, 64, 2, 3, 5)
    check_fork(kc, vc, table, lens, refs, [0, 0, 0, 0], 40, 16)   # 3 free pages, more wanted
    kc, vc, table, refs = fork_state(8, lens, 16, 1, 64, 2, 50, 4)
    check_fork(kc, vc, table, lens, refs, [0, 3, 2, 3], 40, 16)   # columns end before the room does
    kc, vc, table, refs = fork_state(9, lens, 16, 1, 64, 2, 0, 6)
    check_fork(kc, vc, table, lens, refs, [1, 0, 2, 1], 17, 16)   # nothing is free


def test_fork_many_sequences_and_pages():
    r = np.random.RandomState(10)
    Z = 1500
    lens = r.randint(0, 40, Z).tolist()
    kc, vc, table, refs = fork_state(10, lens, 16, 1, 16, 1, 9000, 6)
    source = [int(r.choice([z, r.randint(Z), -1])) for z in range(Z)]
    kc, vc, table, lens, refs = check_fork(kc, vc, table, lens, refs, source, 19, 16)
    check_fork(kc, vc, table, lens, refs, r.permutation(Z).tolist(), 30, 16)


def test_fork_bad_source_is_reported_and_stays():
    import exact_attention_44_gb300 as fa
    kc, vc, table, refs = fork_state(11, [20, 30, 3], 16, 1, 64, 1, 9, 4)
    tg, lg, rg = table.cuda(), i32([20, 30, 3]), i32(refs)
    fa.fa_cache_fork(kc.cuda(), vc.cuda(), tg, lg, rg, i32([3, -2, 0]))
    assert fa.fa_device_status()[0] == fa.FA_ERR_PAGE
    t, n, r, _, _ = pu.fork(table.tolist(), [20, 30, 3], refs, [0, 1, 0], 0, 16)
    assert tg.tolist() == t and lg.tolist() == n and rg.tolist() == r


def test_fork_without_pages_or_columns():
    import exact_attention_44_gb300 as fa
    empty = torch.empty(2, 0, 2, 16, 64, dtype=torch.float16, device="cuda")
    table, lens = torch.empty(3, 0, dtype=torch.int32, device="cuda"), i32([0, 0, 0])
    missing = i32([0])
    fa.fa_cache_fork(empty, empty, table, lens, i32([]), room=5, missing=missing)
    assert missing.item() == 3 and fa.fa_device_status()[0] == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_serving_run(dtype):
    """Prompts, drafted trees, commits, beams and ended sequences, with every step's attention
    checked against the rows that the sequences should hold; the steps run from one captured graph
    as well, and end in the same state."""
    import exact_attention_44_gb300 as fa
    Z, L, Hq, Hkv, D, page, T, A, steps = 5, 2, 6, 2, 64, 16, 12, 4, 4
    P, M = 120, 16
    r = np.random.RandomState(12)
    dt = pu.DT[dtype]
    kc = torch.full((L, P, Hkv, page, D), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    table, lens, refs = torch.full((Z, M), -1, dtype=torch.int32, device="cuda"), i32([0] * Z), i32([0] * P)
    missing = i32([0])
    rows = [[np.zeros((L, Hkv, 0, D)), np.zeros((L, Hkv, 0, D))] for _ in range(Z)]
    n_prompt = [40, 1, 17, 0, 33]
    fa.fa_cache_fork(kc, vc, table, lens, refs, room=40, missing=missing)
    x = [torch.randn(L, Z, Hkv, 40, D).to(dt) for _ in range(2)]
    for la in range(L):
        fa.fa_cache_append(x[0][la].cuda(), x[1][la].cuda(), kc[la], vc[la], table, lens, new_lens=i32(n_prompt))
    lens += i32(n_prompt)
    for z in range(Z):
        rows[z] = [c[:, z, :, :n_prompt[z]].double().numpy() for c in x]
    scale = 1 / math.sqrt(D)
    buf = dict(src=i32(list(range(Z))), acc=i32([[0] * A] * Z), kept=i32([0] * Z),
               kn=torch.zeros(L, Z, Hkv, T, D, dtype=dt, device="cuda"),
               vn=torch.zeros(L, Z, Hkv, T, D, dtype=dt, device="cuda"),
               q=torch.zeros(L, Z, Hq, T, D, dtype=dt, device="cuda"),
               mask=torch.zeros(Z, T, 1, dtype=torch.int32, device="cuda"),
               o=torch.zeros(L, Z, Hq, T, D, dtype=dt, device="cuda"),
               lse=torch.zeros(L, Z, Hq, T, dtype=torch.float32, device="cuda"))

    def step():
        fa.fa_cache_fork(kc, vc, table, lens, refs, buf["src"], room=T, missing=missing)
        for la in range(L):
            fa.fa_cache_append(buf["kn"][la], buf["vn"][la], kc[la], vc[la], table, lens)
            fa.fa_fwd_paged(buf["q"][la], kc[la], vc[la], table, lens, buf["o"][la], buf["lse"][la],
                            tree_mask=buf["mask"])
        fa.fa_cache_commit(kc, vc, table, lens, buf["acc"], buf["kept"])
        lens.add_(buf["kept"])

    start = [t.clone() for t in (kc, vc, table, lens, refs)]
    plans = []
    for s in range(steps):
        source = [int(r.choice([z, z, r.randint(Z)])) for z in range(Z)]
        if s == 2:
            source[3] = -1
        kept = [int(r.randint(0, A + 1)) if source[z] >= 0 else 0 for z in range(Z)]
        path = np.zeros((Z, A), dtype=np.int32)
        for z in range(Z):
            path[z, :kept[z]] = np.sort(r.permutation(T)[:kept[z]])
        seen = pu.random_tree(100 + s, Z, T)
        new = [torch.randn(L, Z, Hkv, T, D).to(dt) for _ in range(2)]
        q = torch.randn(L, Z, Hq, T, D).to(dt)
        plans.append((source, kept, path, seen, new, q))

    def fill(plan):
        source, kept, path, seen, new, q = plan
        buf["src"].copy_(i32(source))
        buf["kept"].copy_(i32(kept))
        buf["acc"].copy_(i32(path.tolist()))
        buf["kn"].copy_(new[0])
        buf["vn"].copy_(new[1])
        buf["q"].copy_(q)
        buf["mask"].copy_(pu.tree_words(seen))

    outs = []
    for plan in plans:
        source, kept, path, seen, new, q = plan
        fill(plan)
        step()
        assert missing.item() == 0
        code = fa.fa_device_status()[0]
        # (the ended sequence has no pages: its drafted rows are skipped and reported)
        assert code == (fa.FA_ERR_PAGE if -1 in source else fa.FA_OK)
        outs.append((buf["o"].clone(), buf["lse"].clone()))
        was = rows
        rows = [[c.copy() for c in was[a]] if a >= 0 else [np.zeros((L, Hkv, 0, D))] * 2 for a in source]
        for la in range(L):
            k = [np.concatenate([rows[z][0][la], new[0][la, z].double().numpy()], 1) for z in range(Z)]
            v = [np.concatenate([rows[z][1][la], new[1][la, z].double().numpy()], 1) for z in range(Z)]
            n = [x.shape[1] - T for x in k]
            live = [z for z in range(Z) if source[z] >= 0]
            qd = q[la].double().numpy()
            want, wl = pu.attention(qd, k, v, n, [T] * Z, seen, scale)
            to, tl = pu.tolerances(qd, k, v, dtype, scale)
            got, lse = buf["o"][la].double().cpu().numpy(), buf["lse"][la].double().cpu().numpy()
            assert np.abs(got[live] - want[live]).max() <= to
            assert np.abs(lse[live] - wl[live]).max() <= tl
        for z in range(Z):
            for c in range(2):
                rows[z][c] = np.concatenate([rows[z][c], new[c][:, z].double().numpy()[:, :, path[z, :kept[z]]]], 2)
    assert lens.tolist() == [x[0].shape[2] for x in rows]
    held = table[table >= 0].cpu().numpy()
    assert np.bincount(held, minlength=P).tolist() == refs.tolist()
    for z in range(Z):
        n = rows[z][0].shape[2]
        for c, cache in enumerate((kc, vc)):
            ids = table[z, :pu.cdiv(n, page)].long()
            have = cache[:, ids].transpose(1, 2).reshape(L, Hkv, -1, D)[:, :, :n].double().cpu().numpy()
            assert np.array_equal(have, rows[z][c])
    # the same steps replayed from one graph
    for t, was in zip((kc, vc, table, lens, refs), start):
        t.copy_(was)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    end = [rows[z][0].shape[2] for z in range(Z)]
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for t, was in zip((kc, vc, table, lens, refs), start):
        t.copy_(was)
    for plan, (o, lse) in zip(plans, outs):
        fill(plan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf["o"], o) and torch.equal(buf["lse"], lse)
    assert lens.tolist() == end
    fa.fa_device_status()


def test_fork_counts_what_lacks_without_overflow():
    import exact_attention_44_gb300 as fa
    kc, vc, table, refs = fork_state(12, [5] * 64, 16, 1, 16, 1, 0, 2)
    missing = i32([0])
    fa.fa_cache_fork(kc.cuda(), vc.cuda(), table.cuda(), i32([5] * 64), i32(refs), room=2 ** 30, missing=missing)
    assert missing.item() == 2 ** 31 - 1  # 64 x 2^26 pages, more than an int32 holds
    fa.fa_cache_fork(kc.cuda(), vc.cuda(), table[:0].cuda(), i32([]), i32(refs), room=1, missing=missing)
    assert missing.item() == 0
