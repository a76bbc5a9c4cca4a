"""Eviction where no page is free and sequences share some: cut in an order that gives pages back first."""
import torch

import pytest

import budget_util as bu
import paged_util as pu
from test_evict_gpu import bits, i32, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def test_sequences_of_a_full_pool_are_cut_in_turn():
    """Sequences 0 and 1 share a prefix, 2 is alone, and the pool is full.  All at once lacks pages, and changes nothing; 2
    alone gives pages back, 0 alone takes some of them for its copies, and then what 0 and 1 shared is 1's own."""
    import exact_attention_44_gb300 as fa
    lens, n, page = [150, 140, 130], 60, 16
    kc, vc, table, refs = state(31, lens, page, 2, 64, 2, extra=0, share=[(1, 0, 8)])
    refs = [max(c, 1) for c in refs]  # (pages that sequence 1 held before it shared belong to others)
    scores = torch.rand(2, 3, 2, table.shape[1] * page)
    kg, vg, tg, lg, rg, sg, missing = kc.cuda(), vc.cuda(), table.cuda(), i32(lens), i32(refs), scores.cuda(), i32([-1])
    t, books = table.tolist(), []
    for keep in (None, [-1, -1, n], [n, -1, -1], [-1, n, -1], None):
        before = [x.clone() for x in (kg, vg, sg)]
        was = t
        t, lens, refs, lack, kept = bu.evict(was, lens, refs, sg.cpu().double().numpy(), page, n, keep, 20, 10)
        fa.fa_cache_evict(kg, vg, tg, lg, rg, sg, n, missing, keep=None if keep is None else i32(keep), first=20, recent=10)
        assert missing.item() == lack and tg.tolist() == t and lg.tolist() == lens and rg.tolist() == refs
        books.append((lack, lens))
        for c, b in zip((kg, vg), before):
            assert torch.equal(bits(c), bits(bu.move(b.cpu(), was, t, kept, page)))
        want = before[2].cpu()
        for z, idx in enumerate(kept):
            if idx is not None:
                i = torch.from_numpy(idx)
                want[:, z, :, :n] = want[:, z].gather(2, i)
        assert torch.equal(sg.cpu(), want)
    assert [b[0] > 0 for b in books] == [True, False, False, False, False]
    assert books[0][1] == [150, 140, 130] and lens == [n, n, n] and fa.fa_device_status()[0] == 0
