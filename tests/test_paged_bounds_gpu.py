"""fa_fwd_paged's O against bounds of each row's own weights: sharp for long contexts too, where O is
small beside the largest |v|."""
import math

import numpy as np
import pytest
import torch

import bounds_util as bu
import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page,tree", [
    ([5000, 17, 2500], 4, 1, 1, 64, 64, False), ([5000, 17, 2500], 4, 1, 3, 128, 16, True),
    ([4000, 300], 4, 1, 33, 64, 64, True), ([3000, 65], 4, 2, 20, 128, 32, True), ([2500, 700], 2, 1, 5, 256, 48, False),
    ([9000], 4, 2, 1, 128, 16, False), ([2000, 0], 3, 1, 42, 32, 16, False), ([0, 5], 2, 2, 300, 64, 16, False)])
def test_rows_own_bounds(dtype, lens, Hq, Hkv, T, D, page, tree):
    import exact_attention_44_gb300 as fa
    Z, scale = len(lens), 1 / math.sqrt(D)
    kc, vc, table, k, v = pu.make_cache(1, [n + T for n in lens], Hkv, D, page, dtype)
    q = torch.randn((Z, Hq, T, D), generator=torch.Generator().manual_seed(2)).to(pu.DT[dtype])
    seen = pu.random_tree(3, Z, T) if tree else None
    o, lse = fa.fa_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             tree_mask=pu.tree_words(seen).cuda() if tree else None)
    assert fa.fa_device_status()[0] == 0
    want, wl, bound = bu.attention(q.double().numpy(), k, v, lens, [T] * Z, seen, scale, dtype)
    over = np.abs(o.double().cpu().numpy() - want) / np.where(bound > 0, bound, 1)
    assert over.max() <= 1, over.max()
    tl = pu.tolerances(q.double().numpy(), k, v, dtype, scale)[1]
    assert np.abs(lse.double().cpu().numpy() - wl).max() <= tl
