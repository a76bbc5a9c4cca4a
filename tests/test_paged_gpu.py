"""GPU parity of fa_fwd_paged against the plain 64-bit statement, at the lengths, masks, layouts
and pages where it can go wrong."""
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


def run(seed, lens, Hq, Hkv, T, D, page, dtype, *, new=None, seen=None, scale=None, layout="phnd", q_layout="bnsd",
        q_mul=1.0, shared_mask=False, cols=None, edit=None, garbage=float("nan")):
    """One call on random data; returns (o, lse) of the kernel, of the statement, and the bounds."""
    import exact_attention_44_gb300 as fa
    Z = len(lens)
    news = [T] * Z if new is None else list(new)
    kc, vc, table, k, v = pu.make_cache(seed, [a + b for a, b in zip(lens, news)], Hkv, D, page, dtype, layout=layout,
                                        cols=cols, garbage=garbage)
    q = (q_mul * torch.randn((Z, Hq, T, D), generator=torch.Generator().manual_seed(seed + 1))).to(pu.DT[dtype])
    if edit is not None:
        edit(kc, vc, table, k, v)
    scale_ = 1 / math.sqrt(D) if scale is None else scale
    qg = q.cuda()
    o = None
    if q_layout == "bsnd":
        qg = q.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        o = torch.zeros((Z, T, Hq, D), dtype=q.dtype, device="cuda").transpose(1, 2)
    words = None
    if seen is not None:
        words = pu.tree_words(seen)
        words = words[0].cuda() if shared_mask else words.cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got, lse = fa.fa_fwd_paged(qg, pu.like(kc), pu.like(vc), table.cuda(), i32(list(lens)), o,
                               new_lens=None if new is None else i32(news), tree_mask=words, scale=scale)
    assert fa.fa_device_status()[0] == 0
    qd = q.double().numpy()
    want, wlse = pu.attention(qd, k, v, lens, news, seen, scale_)
    fin = [np.where(np.isfinite(x), x, 0) for x in k]
    return got.double().cpu().numpy(), lse.double().cpu().numpy(), want, wlse, *pu.tolerances(qd, fin, v, dtype, scale_)


def check(*args, **kw):
    o, lse, wo, wl, to, tl = run(*args, **kw)
    none = np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), none)
    assert np.isfinite(o).all()
    assert np.abs(o[none]).max(initial=0) == 0
    assert np.abs(o - wo).max(initial=0) <= to, (np.abs(o - wo).max(), to)
    assert np.abs(lse[~none] - wl[~none]).max(initial=0) <= tl, (np.abs(lse[~none] - wl[~none]).max(), tl)


@pytest.mark.parametrize("D", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_head_dims(D, dtype, T):
    check(1, [0, 1, 37, 200], 4, 2, T, D, 16, dtype)


@pytest.mark.parametrize("page", [16, 32, 48, 128, 256])
@pytest.mark.parametrize("T", [1, 3, 70])
def test_pages_end_inside_tiles(page, T):
    check(2, [15, 16, 17, 127, 128, 300], 6, 2, T, 64, page, "bf16")


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (8, 2), (12, 4), (16, 1), (32, 8), (64, 1), (200, 1)])
@pytest.mark.parametrize("T", [1, 5, 33])
def test_groups(Hq, Hkv, T):
    check(3, [70, 5, 129], Hq, Hkv, T, 64, 16, "fp16")


@pytest.mark.parametrize("Hq,Hkv", [(100, 1), (128, 1), (260, 2), (129, 1)])
@pytest.mark.parametrize("T,D", [(1, 256), (2, 256), (3, 128)])
def test_large_groups(Hq, Hkv, T, D):
    check(34, [70, 5, 129, 400], Hq, Hkv, T, D, 16, "bf16")


@pytest.mark.parametrize("T", [2, 17, 31, 32, 33, 64, 65, 100])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 48)])
def test_trees(T, D, page):
    lens = [0, 1, 63, 64, 250]
    check(4, lens, 8, 2, T, D, page, "bf16", seen=pu.random_tree(T, len(lens), T))


def test_shared_tree():
    seen = np.repeat(pu.random_tree(9, 1, 40), 3, 0)
    check(5, [10, 100, 33], 4, 1, 40, 64, 16, "fp16", seen=seen, shared_mask=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [7, 50])
def test_rows_that_see_nothing(D, T):
    # token 0 of the empty sequence, and others, see nothing at all; tokens of other sequences only the context
    seen = pu.random_tree(10, 4, T)
    seen[0, 0], seen[0, 5], seen[2, :] = False, False, False
    check(6, [0, 0, 3, 90], 4, 2, T, D, 16, "bf16", seen=seen, new=[T, 0, T, T - 1])


def test_arbitrary_bits():
    # not a tree: later tokens, tokens the sequence does not have, no bit for the token itself
    r = np.random.RandomState(11)
    seen = r.rand(5, 45, 45) < 0.3
    check(7, [0, 20, 64, 128, 5], 8, 2, 45, 64, 32, "fp16", seen=seen, new=[45, 30, 1, 44, 0])


@pytest.mark.parametrize("T", [1, 4, 64])
@pytest.mark.parametrize("tree", [False, True])
def test_ragged_new_tokens(T, tree):
    new = [0, 1, T, max(1, T // 2), T]
    check(8, [40, 0, 0, 65, 512], 8, 4, T, 128, 16, "bf16", new=new, seen=pu.random_tree(12, 5, T) if tree else None)


@pytest.mark.parametrize("layout", ["phnd", "pnhd", "padded"])
@pytest.mark.parametrize("q_layout", ["bnsd", "bsnd"])
@pytest.mark.parametrize("T", [2, 40])
def test_layouts(layout, q_layout, T):
    check(9, [33, 150], 8, 2, T, 64, 32, "fp16", layout=layout, q_layout=q_layout)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3, 3.0])
@pytest.mark.parametrize("T", [1, 48])
def test_scales(scale, T):
    check(10, [100, 7], 4, 2, T, 64, 16, "fp16", scale=scale)


@pytest.mark.parametrize("T", [2, 64])
def test_large_scores(T):
    # scores of several hundred: maxima jump between tiles and parts
    check(11, [900, 300], 4, 2, T, 64, 16, "fp16", scale=1.0, q_mul=4.0)


@pytest.mark.parametrize("T", [1, 3, 33])
@pytest.mark.parametrize("D", [64, 256])
def test_long_context_is_cut(T, D):
    check(12, [5000, 17, 2500], 4, 1, T, D, 64, "bf16")


def test_many_sequences():
    r = np.random.RandomState(13)
    check(13, list(r.randint(0, 60, 700)), 2, 1, 2, 16, 16, "bf16", new=list(r.randint(0, 3, 700)))


def test_all_empty():
    check(14, [0, 0, 0], 4, 2, 3, 64, 16, "bf16", new=[0, 0, 0], cols=2)


@pytest.mark.parametrize("T", [5, 60])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unseen_keys_may_hold_anything(T, bad):
    # the K of a drafted token that nobody sees but itself
    lens = [20, 130]
    seen = pu.random_tree(15, 2, T)
    seen[:, :, 3] = False

    def edit(kc, vc, table, k, v):
        for z, n in enumerate(lens):
            p, s = divmod(n + 3, 16)
            kc[table[z, p], :, s] = bad
            k[z][:, n + 3] = bad

    check(15, lens, 4, 2, T, 64, 16, "fp16", seen=seen, edit=edit)


@pytest.mark.parametrize("T", [1, 40])
def test_non_finite_seen_scores_reach_the_output(T):
    def edit(kc, vc, table, k, v):
        kc[table[1, 0], :, 2] = float("nan")

    o, lse, _, _, _, _ = run(16, [50, 50], 4, 2, T, 64, 16, "bf16", edit=edit)
    assert np.isfinite(o[0]).all() and np.isnan(o[1]).all() and np.isnan(lse[1]).all()


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("entry", [-1, -7, 10 ** 6, 2 ** 31 - 1])
def test_bad_pages_are_reported_and_not_followed(T, entry):
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(17, [100 + T, 100 + T], 2, 64, 16, "fp16")
    table[1, 2] = entry
    q = torch.randn(2, 4, T, 64).half()
    args = (kc.cuda(), vc.cuda(), table.cuda(), torch.tensor([100, 100], dtype=torch.int32, device="cuda"))
    o, lse = fa.fa_fwd_paged(q.cuda(), *args)
    assert fa.fa_device_status()[0] == fa.FA_ERR_PAGE
    k[1][:, 32:48] = 0  # the positions read as zeros
    v[1][:, 32:48] = 0
    qd = q.double().numpy()
    want, wl = pu.attention(qd, k, v, [100, 100], [T, T], None, 0.125)
    to, tl = pu.tolerances(qd, k, v, "fp16", 0.125)
    assert np.abs(o.double().cpu().numpy() - want).max() <= to
    assert np.abs(lse.double().cpu().numpy() - wl).max() <= tl
    assert fa.fa_device_status()[0] == fa.FA_OK


@pytest.mark.parametrize("T", [2, 40])
def test_lengths_past_the_table_are_clamped(T):
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(18, [96, 96], 1, 64, 16, "bf16")
    q = torch.randn(2, 2, T, 64).bfloat16()
    lens = torch.tensor([96 - T, 95], dtype=torch.int32, device="cuda")  # the second has room for one new token
    o, lse = fa.fa_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens)
    far, flse = fa.fa_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                                torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device="cuda"))
    assert fa.fa_device_status()[0] == 0
    qd = q.double().numpy()
    want, wl = pu.attention(qd, k, [x for x in v], [96 - T, 95], [T, 1], None, 0.125)
    to, tl = pu.tolerances(qd, k, v, "bf16", 0.125)
    assert np.abs(o.double().cpu().numpy() - want).max() <= to
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(wl))
    assert (far[0] == 0).all() and torch.isneginf(flse[0]).all() and torch.isfinite(flse[1]).all()


@pytest.mark.parametrize("T", [1, 20, 64])
def test_bitwise_repeatable(T):
    a = run(19, [3000, 10, 700], 8, 2, T, 128, 16, "bf16")
    b = run(19, [3000, 10, 700], 8, 2, T, 128, 16, "bf16")
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("T", [1, 64])
def test_graph_follows_the_lengths_and_tables_it_finds(T):
    import exact_attention_44_gb300 as fa
    ws = torch.empty(fa.fa_fwd_paged_workspace_size(64), dtype=torch.uint8, device="cuda")
    news = [T, T, T]
    all_lens = [[10, 300, 0], [700, 2, 90], [5, 5, 1300]]
    cols = pu.cdiv(1300 + T, 16)
    caches = [pu.make_cache(20 + i, [a + T for a in lens], 2, 64, 16, "fp16", cols=cols, extra=0)
              for i, lens in enumerate(all_lens)]
    P = max(c[0].shape[0] for c in caches)
    kc = torch.zeros(P, 2, 16, 64, dtype=torch.float16, device="cuda")
    vc, table = torch.zeros_like(kc), torch.zeros(3, cols, dtype=torch.int32, device="cuda")
    lens_g = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.randn(3, 8, T, 64).half()
    qg = q.cuda()
    o, lse = torch.empty_like(qg), torch.empty(3, 8, T, device="cuda")
    call = lambda: fa.fa_fwd_paged(qg, kc, vc, table, lens_g, o, lse, workspace=ws)  # noqa: E731
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for lens, (a, b, tb, k, v) in zip(all_lens, caches):
        kc[:a.shape[0]].copy_(a)
        vc[:b.shape[0]].copy_(b)
        table.copy_(tb)
        lens_g.copy_(torch.tensor(lens))
        graph.replay()
        torch.cuda.synchronize()
        qd = q.double().numpy()
        want, wl = pu.attention(qd, k, v, lens, news, None, 0.125)
        to, tl = pu.tolerances(qd, k, v, "fp16", 0.125)
        assert np.abs(o.double().cpu().numpy() - want).max() <= to
        assert np.abs(lse.double().cpu().numpy() - wl).max() <= tl
        replayed = o.clone()
        call()
        assert torch.equal(o, replayed)
    assert fa.fa_device_status()[0] == 0


def test_other_stream_and_no_lse():
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(30, [77], 2, 64, 16, "fp16")
    q = torch.randn(1, 4, 2, 64).half()
    args = [x.cuda() for x in (q, kc, vc, table, torch.tensor([75], dtype=torch.int32))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, none = fa.fa_fwd_paged(*args, stream=s, want_lse=False)
    s.synchronize()
    b, lse = fa.fa_fwd_paged(*args)
    torch.cuda.synchronize()
    assert none is None and lse is not None and torch.equal(a, b)


def test_workspace_errors():
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(31, [20], 1, 64, 16, "fp16")
    args = [x.cuda() for x in (torch.zeros(1, 1, 1, 64).half(), kc, vc, table, torch.tensor([19], dtype=torch.int32))]
    big = torch.empty(fa.fa_fwd_paged_workspace_size(64) + 256, dtype=torch.uint8, device="cuda")
    for ws in (big[:1024], big[16:]):
        with pytest.raises(fa.FaError) as e:
            fa.fa_fwd_paged(*args, workspace=ws)
        assert e.value.code == fa.FA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(*args[:4], args[4].cpu())


def test_cache_offsets_past_32_bits():
    # pages 4.6 GB apart in elements (strides past 2^31): a cache inside a large padded buffer
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(32, [40], 1, 64, 16, "bf16", extra=0)
    P = kc.shape[0]
    stride = 2 ** 31 + 2048
    base = torch.empty((P - 1) * stride + 16 * 64, dtype=torch.bfloat16, device="cuda")
    far_k = base.as_strided((P, 1, 16, 64), (stride, 1024, 64, 1))
    far_k.copy_(kc)
    q = torch.randn(1, 4, 1, 64).bfloat16().cuda()
    for T in (1, 39):
        qt = q.expand(1, 4, T, 64).contiguous()
        lens = torch.tensor([40 - T], dtype=torch.int32, device="cuda")
        a = fa.fa_fwd_paged(qt, far_k, vc.cuda(), table.cuda(), lens)
        b = fa.fa_fwd_paged(qt, kc.cuda(), vc.cuda(), table.cuda(), lens)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_agrees_with_the_contiguous_forward():
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(33, [512, 512], 2, 128, 64, "bf16")
    q = torch.randn(2, 8, 512, 128).bfloat16()
    kk, vv = (torch.from_numpy(np.stack(x)).bfloat16().cuda() for x in (k, v))
    o, lse = fa.fa_fwd(q.cuda(), kk, vv, causal=True)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    o2, lse2 = fa.fa_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), zero)
    to, tl = pu.tolerances(q.double().numpy(), k, v, "bf16", 1 / math.sqrt(128))
    assert (o.double() - o2.double()).abs().max() <= 2 * to and (lse - lse2).abs().max() <= 2 * tl


def test_stall_times_out_and_recovers():
    import exact_attention_44_gb300 as fa
    args = (40, [300, 1000], 8, 2, 40, 64, 16, "fp16")
    kc, vc, table, k, v = pu.make_cache(40, [340, 1040], 2, 64, 16, "fp16")
    q = torch.randn(2, 8, 40, 64).half().cuda()
    lens = torch.tensor([300, 1000], dtype=torch.int32, device="cuda")
    fa.fa_debug_set_wait_limit_ms(100)
    fa.fa_debug_inject_stall(True)
    try:
        fa.fa_fwd_paged(q, kc.cuda(), vc.cuda(), table.cuda(), lens)
        code, word = fa.fa_device_status()
    finally:
        fa.fa_debug_inject_stall(False)
        fa.fa_debug_set_wait_limit_ms(0)
    assert code == fa.FA_ERR_DEVICE_TIMEOUT and (word >> 16) == 0
    check(*args)


def test_stall_of_a_decode_step_times_out_and_recovers():
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(41, [3001], 2, 64, 16, "fp16")
    q = torch.randn(1, 8, 1, 64).half().cuda()
    lens = torch.tensor([3000], dtype=torch.int32, device="cuda")
    fa.fa_debug_set_wait_limit_ms(100)
    fa.fa_debug_inject_stall(True)
    try:
        fa.fa_fwd_paged(q, kc.cuda(), vc.cuda(), table.cuda(), lens)
        code, word = fa.fa_device_status()
    finally:
        fa.fa_debug_inject_stall(False)
        fa.fa_debug_set_wait_limit_ms(0)
    assert code == fa.FA_ERR_DEVICE_TIMEOUT and (word >> 16) == 0
    check(41, [3000], 8, 2, 1, 64, 16, "fp16")


@pytest.mark.parametrize("T", [1, 40])
def test_cache_without_pages_holds_nothing(T):
    import exact_attention_44_gb300 as fa
    empty = torch.empty(0, 2, 16, 64, dtype=torch.float16, device="cuda")
    q = torch.randn(2, 4, T, 64).half().cuda()
    o, lse = fa.fa_fwd_paged(q, empty, empty, torch.zeros(2, 3, dtype=torch.int32, device="cuda"),
                             torch.tensor([5, 0], dtype=torch.int32, device="cuda"))
    assert fa.fa_device_status()[0] == 0 and (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("D", [16, 64, 128, 256])
@pytest.mark.parametrize("T", [1, 40])
def test_outputs_off_32_byte_boundaries(D, T):
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(42, [340, 1040], 2, D, 16, "bf16")
    args = [kc.cuda(), vc.cuda(), table.cuda(), torch.tensor([300 - T, 1040 - T], dtype=torch.int32, device="cuda")]
    q = torch.randn((2, 8, T, D), generator=torch.Generator().manual_seed(43)).bfloat16().cuda()
    want, wl = fa.fa_fwd_paged(q, *args)
    big = torch.full((2, 8, T, D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    odd = torch.full((2, 8, T, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    for whole, o in ((big, big[..., 8:8 + D]), (odd, odd[..., :D])):  # base, strides at odd multiples of 16 bytes
        got, lse = fa.fa_fwd_paged(q, *args, o)
        assert got.data_ptr() == o.data_ptr() and torch.equal(o, want) and torch.equal(lse, wl)
        edge = torch.cat([whole[..., :o.storage_offset()], whole[..., o.storage_offset() + D:]], -1)
        assert bool((edge == 7.0).all())


@pytest.mark.parametrize("T", [1, 40])
def test_expanded_queries(T):
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(42, [60 + T] * 3, 2, 64, 16, "fp16")
    args = (kc.cuda(), vc.cuda(), table.cuda(), torch.tensor([60] * 3, dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 4, 1, 64).half().cuda()
    a, la = fa.fa_fwd_paged(q.expand(3, 4, T, 64), *args)
    b, lb = fa.fa_fwd_paged(q.expand(3, 4, T, 64).contiguous(), *args)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("T", [1, 40])
def test_side_stream_keeps_what_it_uses(T):
    # every tensor of the call, its workspace included, is dropped right after it; allocations on the
    # current stream must not reuse their memory while the side stream, held up first, still needs it
    import exact_attention_44_gb300 as fa
    kc, vc, table, k, v = pu.make_cache(43, [500 + T] * 4, 4, 128, 16, "bf16")
    q = torch.randn(4, 16, T, 128).bfloat16()
    lens = torch.tensor([500] * 4, dtype=torch.int32)
    want, wlse = fa.fa_fwd_paged(*[x.cuda() for x in (q, kc, vc, table, lens)])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = [x.cuda() for x in (q, kc, vc, table, lens)]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    o, lse = fa.fa_fwd_paged(*args, stream=s)
    sizes = [x.numel() * x.element_size() for x in args] + [fa.fa_fwd_paged_workspace_size(128)]
    del args
    junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes]
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wlse) and len(junk) == 6


def test_two_streams_at_once():
    import exact_attention_44_gb300 as fa
    jobs = []
    for n, (T, D, lens) in enumerate(((1, 128, [3000, 70, 900]), (60, 64, [40, 2000, 333]))):
        kc, vc, table, k, v = pu.make_cache(46 + n, [x + T for x in lens], 2, D, 16, "bf16")
        q = torch.randn((3, 8, T, D), generator=torch.Generator().manual_seed(n)).bfloat16().cuda()
        args = (q, kc.cuda(), vc.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
        ws = torch.empty(fa.fa_fwd_paged_workspace_size(D), dtype=torch.uint8, device="cuda")
        jobs.append((args, dict(workspace=ws), fa.fa_fwd_paged(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, (args, kw, _, stream) in enumerate(jobs):
            with torch.cuda.stream(stream):
                got[i].append(fa.fa_fwd_paged(*args, **kw))
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    for (_, _, (o, lse), _), runs in zip(jobs, got):
        assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in runs)


@pytest.mark.parametrize("T,G,D", [(1100, 1, 64), (520, 3, 128), (700, 2, 256)])
def test_prompts_from_scratch(T, G, D):
    # the tiles of a team have very different numbers of key blocks; groups of uneven sizes
    check(45, [0, 3, 130], 2 * G, 2, T, D, 16, "fp16", new=[T, T - 9, T // 3])


@pytest.mark.parametrize("T,G,tree", [(130, 4, True), (200, 3, False), (64, 8, True), (300, 2, True), (257, 5, False)])
def test_teams_of_tiles(T, G, tree):
    # several tiles of a kv head: teams of two to eight CTAs, the last tile ragged, sequences of all sizes
    lens, new = [0, 700, 33, 1500], [T, T // 2, 1, T - 3]
    seen = pu.random_tree(44, 4, T) if tree else None
    check(44, lens, 2 * G, 2, T, 64, 32, "bf16", new=new, seen=seen)


def test_many_sequences_of_all_lengths():
    r = np.random.RandomState(45)
    lens = np.concatenate([r.randint(0, 20, 200), r.randint(100, 900, 20), [2500]])
    r.shuffle(lens)
    check(45, list(lens), 4, 2, 1, 64, 16, "fp16")
    check(46, list(lens[:60]), 8, 1, 9, 64, 16, "fp16", new=list(r.randint(0, 10, 60)))


@pytest.mark.parametrize("T,G,D", [(6, 4, 64), (18, 1, 128), (9, 8, 128), (100, 1, 32), (5, 5, 256)])
def test_tiles_with_idle_warps_are_repeatable(T, G, D):
    # tiles whose last rows hold no token, over many blocks: the warps of those rows only keep the
    # barriers' counts; one that ran ahead would give the others a wrong row maximum now and then
    import exact_attention_44_gb300 as fa
    lens = [9000, 13, 4000, 700]
    kc, vc, table, k, v = pu.make_cache(47, [a + T for a in lens], 2, D, 32, "bf16")
    q = (4 * torch.randn(4, 2 * G, T, D)).bfloat16()
    args = [x.cuda() for x in (q, kc, vc, table, torch.tensor(lens, dtype=torch.int32))]
    first = [x.clone() for x in fa.fa_fwd_paged(*args)]
    for _ in range(40):
        o, lse = fa.fa_fwd_paged(*args)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    qd = q.double().numpy()
    want, wl = pu.attention(qd, k, v, lens, [T] * 4, None, 1 / math.sqrt(D))
    to, tl = pu.tolerances(qd, k, v, "bf16", 1 / math.sqrt(D))
    assert np.abs(first[0].double().cpu().numpy() - want).max() <= to
    assert np.abs(first[1].double().cpu().numpy() - wl).max() <= tl
