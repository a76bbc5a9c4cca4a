"""fa_cache_fork when pages do not suffice: an all-or-nothing call leaves everything as it was and can
be retried once pages are free; without it what got lost is counted as missing until it is replaced."""
import numpy as np
import pytest
import torch

import fork_util as fu
import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """A cache on the GPU and its plain statement beside it."""

    def __init__(self, seed, lens, page, extra, cols, Hkv=2, D=64, L=2, layout="phnd"):
        kc, vc, table, k, v = pu.make_cache(seed, lens, Hkv, D, page, "fp16", layers=L, extra=extra, cols=cols,
                                            garbage=3.0, layout=layout)
        self.page, self.P = page, kc.shape[1]
        self.k, self.v, self.table, self.lens = pu.like(kc), pu.like(vc), table.cuda(), i32(lens)
        self.plain = [table.tolist(), list(lens), np.bincount(table[table >= 0].numpy(), minlength=self.P).tolist()]
        self.refs = i32(self.plain[2])
        self.rows = list(zip(k, v))  # what each sequence should hold

    def fork(self, source, room, whole):
        """One call, compared with the statement; returns the number of pages that lacked."""
        import exact_attention_44_gb300 as fa
        missing, before = i32([-1]), (self.k.clone(), self.v.clone())
        fa.fa_cache_fork(self.k, self.v, self.table, self.lens, self.refs, None if source is None else i32(source),
                         room=room, missing=missing, all_or_nothing=whole)
        table, lens, refs, lacks, tails = fu.fork(*self.plain, source, room, self.page, whole)
        assert missing.item() == lacks
        assert self.table.tolist() == table and self.lens.tolist() == lens and self.refs.tolist() == refs
        for c, was in zip((self.k, self.v), before):
            want = was.clone()
            for a, b, n in tails:
                want[:, b, :, :n] = was[:, a, :, :n]
            assert torch.equal(c.contiguous().view(torch.int16), want.contiguous().view(torch.int16))
        held = [p for r in table for p in r if p >= 0]
        assert np.bincount(held, minlength=self.P).tolist() == refs
        self.plain = [table, lens, refs]
        if not (whole and lacks) and source is not None:
            empty = np.zeros_like(self.rows[0][0][:, :, :0])
            self.rows = [self.rows[a] if a >= 0 else (empty, empty) for a in source]
        return lacks

    def check_rows(self, which=None):
        for z in range(len(self.rows)) if which is None else which:
            n = self.lens[z].item()
            ids = self.table[z, :pu.cdiv(n, self.page)].long()
            assert bool((ids >= 0).all())
            for c, want in zip((self.k, self.v), self.rows[z]):
                have = c[:, ids].transpose(1, 2).flatten(2, 3)[:, :, :n].double().cpu().numpy()
                assert np.array_equal(have, want)


LENS = [30, 20, 5, 64]


@pytest.mark.parametrize("layout", ["phnd", "pnhd"])
@pytest.mark.parametrize("extra,cols,source,room", [(3, 5, [0, 0, 0, 0], 40), (50, 4, [0, 3, 2, 3], 40),
                                                    (0, 6, [1, 0, 2, 1], 17), (0, 6, [1, 0, 2, 3], 0),
                                                    (0, 6, None, 30)])
def test_nothing_changes_when_pages_lack(extra, cols, source, room, layout):
    pool = Pool(1, LENS, 16, extra, cols, layout=layout)
    assert pool.fork(source, room, True) > 0  # (compared with the state before inside)
    pool.check_rows()


def test_short_then_freed_then_retried():
    # a swap of two beams with partly filled pages in a full pool, and room for all
    pool = Pool(2, [30, 20, 5, 64], 16, 0, 8)
    swap = [1, 0, 2, 3]
    assert pool.fork(swap, 1, True) == 3  # two tails, and a page for the 65th position
    assert pool.fork([0, 1, 2, -1], 0, True) == 0  # the last one ends: four pages
    assert pool.fork(swap[:3] + [-1], 1, True) == 0
    pool.check_rows()
    assert pool.lens.tolist() == [20, 30, 5, 0]


def test_captured_call_is_made_again_once_pages_are_free():
    import exact_attention_44_gb300 as fa
    pool = Pool(7, LENS, 16, 0, 8)
    source, missing = i32([1, 0, 2, 3]), i32([-1])
    ws = torch.empty(fa.fa_cache_fork_workspace_size(4, 8), dtype=torch.uint8, device="cuda")
    assert pool.fork([0, 1, 2, 3], 0, True) == 0  # (one call in the context before any capture)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            fa.fa_cache_fork(pool.k, pool.v, pool.table, pool.lens, pool.refs, source, room=1, missing=missing,
                             workspace=ws, all_or_nothing=True)
    torch.cuda.synchronize()
    state = [pool.table, pool.lens, pool.refs, pool.k, pool.v]
    before = [x.clone() for x in state]
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert missing.item() == 3 and all(torch.equal(a, b) for a, b in zip(state, before))
    assert pool.fork([0, 1, 2, -1], 0, True) == 0
    source.copy_(i32([1, 0, 2, -1]))
    want = fu.fork(*pool.plain, [1, 0, 2, -1], 1, 16, True)
    graph.replay()
    torch.cuda.synchronize()
    assert missing.item() == 0
    assert [pool.table.tolist(), pool.lens.tolist(), pool.refs.tolist()] == list(want[:3])
    pool.rows = [pool.rows[1], pool.rows[0], pool.rows[2], pool.rows[3]]
    pool.check_rows()
    assert fa.fa_device_status()[0] == 0


def test_enough_pages_all_or_nothing_is_the_same_call():
    for source in (None, [3, 0, 0, -1], [0, 1, 2, 3]):
        a, b = Pool(3, LENS, 16, 40, 8), Pool(3, LENS, 16, 40, 8)
        assert a.fork(source, 20, True) == b.fork(source, 20, False) == 0
        assert a.plain == b.plain
        a.check_rows()


def test_a_lost_tail_is_counted_until_it_is_replaced():
    pool = Pool(4, [30, 20, 5, 64], 16, 0, 8)
    assert pool.fork([1, 0, 2, 3], 0, False) == 2    # both tails are lost
    assert pool.fork([0, 1, 2, -1], 0, False) == 2   # pages are free again, but the rows are gone
    assert pool.fork([0, 1, 2, 3], 40, False) == 7   # no room behind a lost tail: 4 + 5 pages wanted, 1 + 1 held
    assert pool.fork([0, 0, 2, 3], 0, True) == 2     # a copy has lost it too
    assert pool.fork([-1, -1, 2, -1], 0, False) == 0
    assert pool.fork([2, 2, 2, -1], 17, True) == 0   # replaced
    pool.check_rows()
    assert pool.fork(None, 17, True) == 0


@pytest.mark.parametrize("whole", [True, False])
def test_many_calls_in_a_small_pool(whole):
    import exact_attention_44_gb300 as fa
    r = np.random.RandomState(5)
    pool = Pool(6, r.randint(0, 60, 9).tolist(), 16, 3, 7, Hkv=1, D=32, L=1)
    lacked = 0
    for step in range(40):
        source = [int(r.choice([z, z, z, r.randint(9), -1])) for z in range(9)]
        lacks = pool.fork(source if step % 3 else None, int(r.randint(0, 25)), whole)
        lacked += lacks > 0
        if whole:
            pool.check_rows()
    assert lacked > 0  # (the pool did run short)
    fa.fa_device_status()
