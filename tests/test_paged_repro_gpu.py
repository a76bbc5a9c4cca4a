"""fa_fwd_paged's bits depend on its arguments only: not on the queries of tokens that a sequence does
not have, and not on what earlier kernels left in shared memory behind the rows of a tile whose group
does not divide 128."""
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


def inputs(seed, lens, new, Hq, Hkv, T, D, page=32):
    kc, vc, table, _, _ = pu.make_cache(seed, [a + T for a in lens], Hkv, D, page, "bf16")
    q = torch.randn((len(lens), Hq, T, D), generator=torch.Generator().manual_seed(seed + 1)).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return q.cuda(), (kc.cuda(), vc.cuda(), table.cuda(), i32(lens)), i32(new)


@pytest.mark.parametrize("T,G,D", [(40, 4, 64), (64, 4, 128), (50, 3, 128), (21, 6, 64), (33, 1, 32), (9, 5, 256),
                                   (3, 4, 64)])
@pytest.mark.parametrize("tree", [False, True])
def test_queries_of_missing_tokens_do_not_enter(T, G, D, tree):
    lens, new = [3000, 40, 700, 1500], [T - 1, T // 2, max(1, T - 7), 1]
    q, args, news = inputs(1, lens, new, 2 * G, 2, T, D)
    words = pu.tree_words(pu.random_tree(2, 4, T)).cuda() if tree else None
    import exact_attention_44_gb300 as fa
    missing = torch.arange(T, device="cuda")[None] >= news[:, None]  # (Z, T)
    first = None
    for fill in (0.0, 30.0, 1000.0, float("inf"), float("nan")):
        x = fill * torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).to(q.dtype)
        got = fa.fa_fwd_paged(torch.where(missing[:, None, :, None], x.cuda(), q), *args, new_lens=news, tree_mask=words)
        if first is None:
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), fill
    assert fa.fa_device_status()[0] == 0


@pytest.mark.parametrize("T,G,D", [(42, 3, 128), (42, 3, 64), (21, 6, 128), (30, 12, 64), (25, 5, 256), (90, 3, 128)])
def test_other_kernels_before_do_not_enter(T, G, D):
    import exact_attention_44_gb300 as fa
    lens = [4000, 900, 2500]
    q, args, _ = inputs(4, lens, [T] * 3, 2 * G, 2, T, D)
    full, fargs, _ = inputs(5, [3000] * 8, [32] * 8, 8, 2, 32, D)  # tiles of all 128 rows
    first = None
    for scale in (0.0, 1.0, 10.0, 100.0, 1000.0):
        for sign in (1.0, -1.0):
            fa.fa_fwd_paged(sign * scale * full, *fargs)
            got = fa.fa_fwd_paged(q, *args)
            if first is None:
                first = got
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), (scale, sign)
    assert fa.fa_device_status()[0] == 0
    assert np.isfinite(first[0].float().cpu().numpy()).all()
