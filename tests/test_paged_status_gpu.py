"""A recorded bad page does not hide a wait that runs out later, and the documented loop ends
sequences without recording one."""
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


def state(T):
    kc, vc, table, _, _ = pu.make_cache(1, [300 + T, 1000 + T], 2, 64, 16, "fp16")
    q = torch.randn((2, 8, T, 64), generator=torch.Generator().manual_seed(2)).half().cuda()
    return q, kc.cuda(), vc.cuda(), table, i32([300, 1000])


def bad_page(call, q, kc, vc, table, lens):
    """One call of a kind that meets a table entry outside the cache."""
    import exact_attention_44_gb300 as fa
    broken = table.clone()
    broken[0, -1], broken[1, 300 // 16] = 7, -1
    rows = torch.zeros(2, 2, 1, 64, dtype=torch.float16, device="cuda")
    if call == "attention":
        fa.fa_fwd_paged(q, kc, vc, broken.cuda(), lens)
    elif call == "append":
        fa.fa_cache_append(rows, rows, kc.clone(), vc.clone(), broken.cuda(), i32([5, 300]))
    elif call == "commit":
        fa.fa_cache_commit(kc.clone(), vc.clone(), broken.cuda(), i32([5, 300]), i32([[0], [3]]), i32([0, 1]))
    else:
        refs = torch.zeros(kc.shape[0], dtype=torch.int32, device="cuda")
        fa.fa_cache_fork(kc.clone(), vc.clone(), table.cuda(), lens.clone(), refs, i32([0, 5]))


@pytest.mark.parametrize("call", ["attention", "append", "commit", "fork"])
@pytest.mark.parametrize("T", [1, 40])
def test_a_wait_that_runs_out_is_reported_after_a_bad_page(call, T):
    import exact_attention_44_gb300 as fa
    q, kc, vc, table, lens = state(T)
    want = fa.fa_fwd_paged(q, kc, vc, table.cuda(), lens)
    assert fa.fa_device_status() == (fa.FA_OK, 0)
    bad_page(call, q, kc, vc, table, lens)
    fa.fa_debug_set_wait_limit_ms(100)
    fa.fa_debug_inject_stall(True)
    try:
        fa.fa_fwd_paged(q, kc, vc, table.cuda(), lens)
        first = fa.fa_device_status()
    finally:
        fa.fa_debug_inject_stall(False)
        fa.fa_debug_set_wait_limit_ms(0)
    second, third = fa.fa_device_status(), fa.fa_device_status()
    assert first[0] == fa.FA_ERR_DEVICE_TIMEOUT and first[1] & 0xFF == fa.FA_ERR_DEVICE_TIMEOUT
    assert second[0] == fa.FA_ERR_PAGE and 60 <= (second[1] >> 8) & 0xFF <= 63  # the other record, with its site
    assert third == (fa.FA_OK, 0)
    got = fa.fa_fwd_paged(q, kc, vc, table.cuda(), lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_steps_after_an_ended_sequence_record_nothing():
    # the loop of the documentation, with new_lens 0 for the sequences that have ended
    import exact_attention_44_gb300 as fa
    Z, T, page, P, M = 4, 6, 16, 40, 8
    k = torch.zeros(2, P, 2, page, 64, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    table, lens, refs = torch.full((Z, M), -1, dtype=torch.int32, device="cuda"), i32([0] * Z), i32([0] * P)
    missing, alive = i32([0]), i32([1] * Z)
    q = torch.randn((Z, 4, T, 64), generator=torch.Generator().manual_seed(3)).half().cuda()
    rows = torch.randn((Z, 2, T, 64), generator=torch.Generator().manual_seed(4)).half().cuda()
    for source in ([0, 1, 2, 3], [0, 0, -1, 3], [0, 1, 2, 3], [3, 1, 2, -1]):
        source = i32(source)
        alive = torch.where(source < 0, torch.zeros_like(alive), alive[source.clamp(min=0).long()])
        source = torch.where(alive > 0, source, torch.full_like(source, -1))
        new = alive * T
        fa.fa_cache_fork(k, v, table, lens, refs, source, room=T, missing=missing, all_or_nothing=True)
        for i in range(2):
            fa.fa_cache_append(rows, rows, k[i], v[i], table, lens, new_lens=new)
            o, lse = fa.fa_fwd_paged(q, k[i], v[i], table, lens, new_lens=new)
            assert bool((o[alive == 0] == 0).all()) and bool(torch.isneginf(lse[alive == 0]).all())
        kept = alive * 3
        fa.fa_cache_commit(k, v, table, lens, i32([[0, 2, 4]] * Z), kept)
        lens += kept
        assert missing.item() == 0 and fa.fa_device_status() == (fa.FA_OK, 0)
    assert lens.tolist() == [12, 12, 0, 0]
