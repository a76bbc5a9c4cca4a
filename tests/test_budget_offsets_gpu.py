"""Offsets past 2^31 elements in the addresses of rotary positions and of the budgeted cache, bit by bit against the
same calls on compact tensors; and a wait of the score kernel that runs out is reported and leaves the device usable."""
import pytest
import torch

import paged_util as pu
from test_paged_offsets_gpu import FAR, far, i32, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def turns_of(R):
    import exact_attention_44_gb300 as fa
    return fa.fa_rope_turns(fa.fa_rope_frequencies(R))


@pytest.mark.parametrize("dim", [0, 1, 2])
def test_rope(dim):
    import exact_attention_44_gb300 as fa
    x = torch.randn(2, 2, 2, 64, generator=torch.Generator().manual_seed(1)).half()
    stride = list(x.stride())
    stride[dim] = FAR
    n = sum((a - 1) * b for a, b in zip(x.shape, stride)) + 1
    y = torch.empty(n, dtype=x.dtype, device="cuda").as_strided(x.shape, stride)
    y.copy_(x)
    want, _ = fa.fa_rope(x.cuda(), None, turns_of(32))
    fa.fa_rope(y, None, turns_of(32), q_out=y)
    assert same(y, want)


@pytest.mark.parametrize("dim", [0, 1])
def test_append_score_and_evict(dim):
    import exact_attention_44_gb300 as fa
    lens, T, L = [60, 25], 20, 3
    kc, vc, table, _, _ = pu.make_cache(2, [n + T for n in lens], 2, 64, 16, "bf16", layers=L, extra=3, garbage=1.0)
    refs = torch.bincount(table[table >= 0].flatten(), minlength=kc.shape[1]).int()
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(L, 2, h, T, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    results = []
    for place in (lambda c: c.cuda(), lambda c: far(c, dim)):
        kk, vv = place(kc), place(vc)
        t, n, r, missing = table.cuda(), i32(lens), refs.cuda(), i32([-1])
        scores = torch.ones(L, 2, 2, table.shape[1] * 16, device="cuda")
        for la in range(L):
            tq = fa.fa_cache_append_rope(q[la], k[la], v[la], kk[la], vv[la], t, n, turns_of(64))
            lse = torch.full((2, 4, T), 4.0, device="cuda")
            fa.fa_cache_score(tq, lse, kk[la], t, n, scores[la])                            # the tile kernel
            fa.fa_cache_score(tq[:, :, -1:], lse[:, :, -1:].contiguous(), kk[la], t, n + (T - 1), scores[la])  # the rows kernel
        n += T
        fa.fa_cache_evict(kk, vv, t, n, r, scores, 30, missing, first=2, recent=8)
        assert missing.item() == 0 and fa.fa_device_status()[0] == 0 and n.tolist() == [30, 30]
        results.append((kk, vv, t, r, scores))
    a, b = results
    assert same(a[0], b[0]) and same(a[1], b[1]) and all(torch.equal(x, y) for x, y in zip(a[2:], b[2:]))


def test_scores_far_apart():
    import exact_attention_44_gb300 as fa
    kc, _, table, _, _ = pu.make_cache(4, [90, 90], 2, 64, 16, "bf16", extra=0)
    q = torch.randn(2, 4, 30, 64, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    lse, n = torch.full((2, 4, 30), 4.0, device="cuda"), i32([60, 50])
    want = torch.ones(2, 2, 96, device="cuda")
    wide = torch.empty(FAR + 3 * 96, device="cuda").as_strided((2, 2, 96), (FAR, 96, 1))
    wide.copy_(want)
    for s in (want, wide):
        fa.fa_cache_score(q, lse, kc.cuda(), table.cuda(), n, s, decay=0.5)
        fa.fa_cache_score(q[:, :, :1], lse[:, :, :1].contiguous(), kc.cuda(), table.cuda(), n, s)
    assert torch.equal(want, wide)


def test_a_wait_that_runs_out_is_reported():
    import exact_attention_44_gb300 as fa
    kc, _, table, _, _ = pu.make_cache(6, [3000, 500], 2, 64, 16, "fp16", garbage=0.0)
    q = torch.randn(2, 8, 40, 64, generator=torch.Generator().manual_seed(7)).half().cuda()
    lse, n = torch.full((2, 8, 40), 5.0, device="cuda"), i32([2960, 460])
    call = lambda s: fa.fa_cache_score(q, lse, kc.cuda(), table.cuda(), n, s, decay=0.0)  # noqa: E731
    want, got = (torch.zeros(2, 2, table.shape[1] * 16, device="cuda") for _ in range(2))
    call(want)
    assert fa.fa_device_status() == (fa.FA_OK, 0)
    fa.fa_debug_set_wait_limit_ms(100)
    fa.fa_debug_inject_stall(True)
    try:
        call(got)
        code, word = fa.fa_device_status()
    finally:
        fa.fa_debug_inject_stall(False)
        fa.fa_debug_set_wait_limit_ms(0)
    assert code == fa.FA_ERR_DEVICE_TIMEOUT and word & 0xFF == fa.FA_ERR_DEVICE_TIMEOUT
    assert fa.fa_device_status() == (fa.FA_OK, 0)
    got.zero_()
    call(got)
    assert torch.equal(got, want) and fa.fa_device_status() == (fa.FA_OK, 0)
