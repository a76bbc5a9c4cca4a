"""The attention weight that cached positions receive, against its definition in 64 bits, element by element."""
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


def check(seed, lens, new, T, Hq, Hkv, D, page, dtype, *, decay=1.0, layout="phnd", scale=None, garbage=float("nan"),
          pad=0, spread=2.0):
    """One call on random sequences against the statement; lse is that of the attention itself."""
    import exact_attention_44_gb300 as fa
    Z = len(lens)
    scale = 1 / math.sqrt(D) if scale is None else scale
    kc, _, table, k, _ = pu.make_cache(seed, [a + b for a, b in zip(lens, new)], Hkv, D, page, dtype, layout=layout,
                                       garbage=garbage)
    g = torch.Generator().manual_seed(seed + 1)
    q = (spread * torch.randn(Z, T, Hq, D, generator=g)).to(pu.DT[dtype]).transpose(1, 2)
    qd = q.double().numpy()
    lse = np.full((Z, Hq, T), -math.inf)
    for z in range(Z):
        for h in range(Hq):
            x = scale * (qd[z, h, :new[z]] @ k[z][h * Hkv // Hq].T)
            x[np.arange(lens[z] + new[z])[None] > lens[z] + np.arange(new[z])[:, None]] = -math.inf
            if new[z]:
                top = x.max(1)
                lse[z, h, :new[z]] = top + np.log(np.exp(x - top[:, None]).sum(1))
    lse32 = torch.from_numpy(lse).float()
    for z in range(Z):  # what is not a token has no say
        q[z, :, new[z]:] = garbage
        lse32[z, :, new[z]:] = garbage
    C = table.shape[1] * page
    was = torch.rand(Z, Hkv, C + pad, generator=g)
    for z in range(Z):  # no score yet behind the old positions
        was[z, :, lens[z]:] = garbage
    if decay == 0:
        was[:] = garbage
    s = was.cuda()[:, :, :C]
    qg = q.transpose(1, 2).cuda().transpose(1, 2)
    fa.fa_cache_score(qg, lse32.cuda(), pu.like(kc), table.cuda(), i32(lens), s,
                      new_lens=None if all(n == T for n in new) else i32(new), decay=decay, scale=scale)
    assert fa.fa_device_status()[0] == 0
    base = was[:, :, :C].double().numpy()
    want, bound = bu.score(qd, lse32.double().numpy(), k, lens, new, np.nan_to_num(base), decay, scale)
    got = s.cpu().double().numpy()
    for z in range(Z):
        n = lens[z] + new[z]
        off = np.abs(got[z, :, :n] - want[z, :, :n])
        assert (off <= bound[z, :, :n]).all(), (z, np.nanmax(off / bound[z, :, :n]))
        assert np.array_equal(got[z, :, n:], base[z, :, n:], equal_nan=True)  # left as they were


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 2, 2), (1, 8, 1), (3, 12, 4), (2, 16, 2), (9, 6, 2), (40, 4, 1)])
def test_every_width(dtype, D, T, Hq, Hkv):
    lens = [0, 1, 15, 16, 100, 333]
    new = [T, 1, max(1, T - 1), 0, T, T]
    check(D + T, lens, new, T, Hq, Hkv, D, 16, dtype)


@pytest.mark.parametrize("page", [16, 48, 64, 128, 112])
@pytest.mark.parametrize("layout", ["phnd", "pnhd", "padded"])
@pytest.mark.parametrize("T", [1, 50])
def test_pages_and_layouts(page, layout, T):
    check(page, [0, 31, 127, 128, 500], [T] * 5, T, 4, 2, 64, page, "fp16", layout=layout, pad=24)


@pytest.mark.parametrize("decay", [0.0, 0.5, -1.5, 1.0])
@pytest.mark.parametrize("T", [1, 37])
def test_decay(decay, T):
    check(7, [0, 5, 130], [T, 0, T], T, 4, 2, 64, 16, "bf16", decay=decay)


@pytest.mark.parametrize("T,G", [(128, 1), (129, 1), (200, 3), (33, 4), (64, 8), (17, 16), (5, 32), (300, 4), (1, 200), (2, 130), (513, 1)])
def test_many_rows(T, G):
    """Chunks longer than a tile, groups that do not divide one, and single tokens of very wide groups."""
    check(T + G, [0, 100, 700, 129], [T, T, max(1, T // 2), T], T, G, 1, 64, 32, "bf16")


@pytest.mark.parametrize("D", [16, 32, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_rows_of_every_width(D, dtype):
    check(D, [0, 250, 90], [150, 60, 0], 150, 4, 2, D, 16, dtype)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-30])
@pytest.mark.parametrize("T", [2, 40])
def test_scales(scale, T):
    check(9, [3, 200], [T, T], T, 2, 1, 64, 16, "fp16", scale=scale, spread=0.5)


def test_sharp_attention():
    """One key takes nearly all of the weight: differences to lse of up to hundreds."""
    check(11, [400, 63], [20, 20], 20, 2, 1, 128, 16, "bf16", spread=40.0)


@pytest.mark.parametrize("Z", [33, 300])
@pytest.mark.parametrize("T", [1, 12])
def test_many_sequences(Z, T):
    r = np.random.RandomState(Z)
    check(Z, r.randint(0, 60, Z).tolist(), r.randint(0, T + 1, Z).tolist(), T, 4, 2, 16, 16, "fp16")


@pytest.mark.parametrize("Z,D,G", [(3, 64, 4), (40, 32, 4), (9, 256, 2), (35, 128, 32)])
def test_many_units_of_few_and_many_tiles(Z, D, G):
    """Chunks of every length up to several tiles, none among them: ranges end in front of, in and behind a unit's tiles."""
    r = np.random.RandomState(Z)
    new = r.randint(0, 301, Z)
    new[::4] = 0
    new[1] = 300
    check(Z, r.randint(0, 600, Z).tolist(), new.tolist(), 300, G, 1, D, 16, "bf16", decay=0.5)


def test_columns_beyond_the_lengths_and_no_work():
    import exact_attention_44_gb300 as fa
    kc = torch.randn(4, 2, 16, 64).half().cuda()
    table = torch.full((3, 5000), -1, dtype=torch.int32, device="cuda")
    scores = torch.ones(3, 2, 80000, device="cuda")
    q, lse = torch.randn(3, 4, 1, 64).half().cuda(), torch.zeros(3, 4, 1, device="cuda")
    fa.fa_cache_score(q, lse, kc, table, i32([0, 0, 0]), scores, new_lens=i32([0, 0, 0]))
    fa.fa_cache_score(q[:, :, :0], lse[:, :, :0], kc, table, i32([0, 0, 0]), scores)
    fa.fa_cache_score(q[:0], lse[:0], kc, table[:0], i32([]), scores[:0])
    fa.fa_cache_score(q, lse, kc[:0], table, i32([7, 0, 0]), scores)
    assert fa.fa_device_status()[0] == 0 and (scores == 1).all()


@pytest.mark.parametrize("T", [1, 64])
def test_bad_pages_read_as_zeros(T):
    import exact_attention_44_gb300 as fa
    kc, _, table, _, _ = pu.make_cache(3, [100 + T], 1, 64, 16, "fp16", garbage=0.0)
    q = torch.randn(1, 2, T, 64).half().cuda()
    lse = torch.full((1, 2, T), 2.0, device="cuda")
    C = table.shape[1] * 16
    bad = table.clone()
    bad[0, 2], bad[0, 5] = -1, 99
    zeros = kc.clone()
    zeros[table[0, 2]] = 0
    zeros[table[0, 5]] = 0
    out = []
    for cache, t in ((kc, bad), (zeros, table)):
        s = torch.zeros(1, 1, C, device="cuda")
        fa.fa_cache_score(q, lse, cache.cuda(), t.cuda(), i32([100]), s)
        out.append((s, fa.fa_device_status()[0]))
    assert torch.equal(out[0][0], out[1][0]) and out[0][1] == fa.FA_ERR_PAGE and out[1][1] == 0


@pytest.mark.parametrize("T", [1, 48])
def test_broadcast_queries(T):
    """Heads that share one row of q: stride 0."""
    import exact_attention_44_gb300 as fa
    kc, _, table, _, _ = pu.make_cache(12, [100 + T] * 2, 2, 64, 16, "fp16", garbage=0.0)
    q = torch.randn(2, 1, T, 64).half().cuda()
    lse = torch.full((2, 4, T), 4.0, device="cuda")
    out = []
    for x in (q.expand(2, 4, T, 64), q.repeat(1, 4, 1, 1)):
        s = torch.zeros(2, 2, table.shape[1] * 16, device="cuda")
        fa.fa_cache_score(x, lse, kc.cuda(), table.cuda(), i32([100, 60]), s)
        out.append(s)
    assert torch.equal(*out) and fa.fa_device_status()[0] == 0


@pytest.mark.parametrize("T", [1, 48])
def test_lengths_past_the_table_are_clamped(T):
    import exact_attention_44_gb300 as fa
    kc, _, table, _, _ = pu.make_cache(4, [64, 64], 1, 64, 16, "fp16")
    q, lse = torch.randn(2, 1, T, 64).half().cuda(), torch.full((2, 1, T), 3.0, device="cuda")
    a, b = (torch.full((2, 1, 64 + 8), 2.0, device="cuda") for _ in range(2))
    fa.fa_cache_score(q, lse, kc.cuda(), table.cuda(), i32([60, 2 ** 31 - 1]), a, new_lens=i32([2 ** 31 - 1, 5]))
    n = min(T, 4)
    fa.fa_cache_score(q, lse, kc.cuda(), table.cuda(), i32([60, 64]), b, new_lens=i32([n, 0]))
    assert fa.fa_device_status()[0] == 0 and torch.equal(a, b) and (a[:, :, 64:] == 2).all()
    assert (a[1, 0, :64] == 2).all()  # decay 1, no new token


def test_rows_without_a_sum_add_nothing():
    import exact_attention_44_gb300 as fa
    kc, _, table, _, _ = pu.make_cache(5, [50], 1, 64, 16, "fp16", garbage=0.0)
    q = torch.randn(1, 2, 20, 64).half().cuda()
    lse = torch.full((1, 2, 20), 1.0, device="cuda")
    out = []
    for drop in (False, True):
        x, y = q.clone(), lse.clone()
        y[0, 1] = -math.inf
        if drop:
            x[0, 1] = 0.0
        s = torch.zeros(1, 1, 64, device="cuda")
        fa.fa_cache_score(x, y, kc.cuda(), table.cuda(), i32([30]), s)
        out.append(s)
    one = torch.zeros(1, 1, 64, device="cuda")
    fa.fa_cache_score(q[:, :1], lse[:, :1].contiguous(), kc.cuda(), table.cuda(), i32([30]), one)
    assert torch.equal(out[0], out[1])
    assert torch.isfinite(out[0]).all() and ((out[0] - one).abs() <= 2.0 ** -20 * one).all()


def test_weights_of_a_chunk_add_up():
    """After fa_fwd_paged each row's weights sum to one: the scores of a call sum to its rows."""
    import exact_attention_44_gb300 as fa
    Z, T, Hq, Hkv, D = 3, 70, 8, 2, 128
    lens = [0, 90, 1000]
    kc, vc, table, _, _ = pu.make_cache(6, [n + T for n in lens], Hkv, D, 32, "bf16")
    q = torch.randn(Z, Hq, T, D).bfloat16().cuda()
    _, lse = fa.fa_fwd_paged(q, kc.cuda(), torch.nan_to_num(vc).cuda(), table.cuda(), i32(lens))
    s = torch.full((Z, Hkv, table.shape[1] * 32), float("nan"), device="cuda")
    fa.fa_cache_score(q, lse, kc.cuda(), table.cuda(), i32(lens), s, decay=0.0)
    for z in range(Z):
        total = s[z, :, :lens[z] + T].double().sum(1)
        # lse is off by the score's rounding and 2^-20 (see paged_util.tolerances): 1e-4 is above all of it
        assert ((total / (T * Hq // Hkv) - 1).abs() <= 1e-4).all()


@pytest.mark.parametrize("T", [1, 90])
def test_repeatable_another_stream_and_graph(T):
    import exact_attention_44_gb300 as fa
    lens = [0, 700, 2000, 31]
    kc, _, table, _, _ = pu.make_cache(8, [n + T for n in lens], 2, 128, 16, "fp16", garbage=0.0)
    kc, table, n = kc.cuda(), table.cuda(), i32(lens)
    q, lse = torch.randn(4, 8, T, 128).half().cuda(), torch.full((4, 8, T), 6.0, device="cuda")
    ws = torch.empty(fa.fa_cache_score_workspace_size(), dtype=torch.uint8, device="cuda").fill_(255)

    def call(stream=None):
        s = torch.ones(4, 2, table.shape[1] * 16, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        fa.fa_cache_score(q, lse, kc, table, n, s, workspace=None if stream is not None else ws, stream=stream)
        torch.cuda.synchronize()
        return s

    want = call()
    assert torch.equal(call(), want)
    # two streams at once, each with a workspace of its own
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.ones_like(want) for _ in side]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o in zip(side, outs):
            fa.fa_cache_score(q, lse, kc, table, n, o, stream=st, decay=0.0)
    torch.cuda.synchronize()
    fresh = torch.zeros_like(want)
    fa.fa_cache_score(q, lse, kc, table, n, fresh, decay=0.0)
    for z in range(4):
        for o in outs:
            assert torch.equal(o[z, :, :lens[z] + T], fresh[z, :, :lens[z] + T])
    # captured once, replayed with other lengths
    s = torch.ones_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_cache_score(q, lse, kc, table, n, s, workspace=ws)
    n.copy_(i32([0, 300, 1999, 31]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s, call())


@pytest.mark.parametrize("Z,T,Hq,Hkv,D,lo,hi", [(24, 32, 32, 8, 128, 500, 2500), (16, 20, 8, 4, 256, 100, 3000), (24, 70, 16, 8, 64, 0, 1500),
                                                (3, 1100, 16, 4, 128, 0, 900), (40, 17, 4, 2, 16, 10, 3000)])
def test_back_to_back(Z, T, Hq, Hkv, D, lo, hi):
    """Many calls that nothing waits between, on different inputs: each leaves the same bits every time.  The units of a
    call pass through slots that several roles fill and free, so a slot that is handed on too early shows here."""
    import exact_attention_44_gb300 as fa
    lens = np.linspace(lo, hi, Z).astype(int).tolist()
    sets = []
    for seed in range(3):
        kc, _, table, _, _ = pu.make_cache(seed, [n + T for n in lens], Hkv, D, 64, "bf16", garbage=0.0)
        g = torch.Generator().manual_seed(seed)
        sets.append((torch.randn(Z, Hq, T, D, generator=g).bfloat16().cuda(), torch.full((Z, Hq, T), 6.0, device="cuda"), kc.cuda(),
                     table.cuda(), i32(lens)))
    outs = [[torch.zeros(Z, Hkv, s[3].shape[1] * 64, device="cuda") for _ in range(100)] for s in sets]
    ws = torch.empty(fa.fa_cache_score_workspace_size(), dtype=torch.uint8, device="cuda")
    for i in range(100):
        for s, o in zip(sets, outs):
            fa.fa_cache_score(*s, o[i], decay=0.0, workspace=ws)
    assert fa.fa_device_status()[0] == 0
    for o in outs:
        first = o[0]
        assert all(torch.equal(x, first) for x in o[1:]) and (first.sum() > 0).item()
