"""The received attention weight where its kernels change their way: sequences without a new token, and unusual
magnitudes, among them in tiles that are full and seen whole (test_score_gpu.py has them in tiles that are not)."""
import math

import numpy as np
import pytest
import torch

import budget_util as bu
import paged_util as pu
from test_score_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T", [1, 64])
@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("Z", [4, 40])
def test_sequences_without_a_new_token_read_no_page(T, decay, Z):
    """An idle sequence's keys have no say: its table is not looked at, and its scores only decay, in both kernels."""
    import exact_attention_44_gb300 as fa
    lens = [100, 50, 70, 300] * (Z // 4)
    new = [T, 0, T, 0] * (Z // 4)
    kc, _, table, _, _ = pu.make_cache(23, [a + b for a, b in zip(lens, new)], 2, 64, 16, "fp16", garbage=0.0)
    bad = table.clone()
    bad[1::4] = -1
    bad[3::4, 1::2] = 9999
    q, lse = torch.randn(Z, 4, T, 64).half().cuda(), torch.full((Z, 4, T), 5.0, device="cuda")
    was = torch.rand(Z, 2, table.shape[1] * 16, device="cuda")
    out = []
    for t in (table, bad):
        s = was.clone()
        fa.fa_cache_score(q, lse, kc.cuda(), t.cuda(), i32(lens), s, new_lens=i32(new), decay=decay)
        assert fa.fa_device_status()[0] == 0
        out.append(s)
    assert torch.equal(*out)
    for z in range(1, Z, 2):
        assert torch.equal(s[z, :, :lens[z]], was[z, :, :lens[z]] * decay) and torch.equal(s[z, :, lens[z]:], was[z, :, lens[z]:])
    nobody = was.clone()
    fa.fa_cache_score(q, lse, kc.cuda(), torch.full_like(table, -1).cuda(), i32(lens), nobody, new_lens=i32([0] * Z), decay=decay)
    assert fa.fa_device_status()[0] == 0
    for z in range(Z):
        assert torch.equal(nobody[z, :, :lens[z]], was[z, :, :lens[z]] * decay)
        assert torch.equal(nobody[z, :, lens[z]:], was[z, :, lens[z]:])


def against_the_statement(q, lse, kc, k, table, lens, T, scale):
    """One call on empty scores, element by element."""
    import exact_attention_44_gb300 as fa
    Z, Hkv = len(lens), k[0].shape[0]
    s = torch.zeros(Z, Hkv, table.shape[1] * kc.shape[2], device="cuda")
    fa.fa_cache_score(q.cuda(), lse.cuda(), kc.cuda(), table.cuda(), i32(lens), s, scale=scale)
    assert fa.fa_device_status()[0] == 0
    want, bound = bu.score(q.double().numpy(), lse.double().numpy(), k, lens, [T] * Z, np.zeros(s.shape), 1.0, scale)
    got = s.cpu().double().numpy()
    for z in range(Z):
        n = lens[z] + T
        off = np.abs(got[z, :, :n] - want[z, :, :n])
        assert (off <= bound[z, :, :n]).all(), (z, np.nanmax(off / bound[z, :, :n]))


def sums(q, k, lens, scale):
    """lse of each row over the positions that it sees."""
    Z, Hq, T, _ = q.shape
    lse = np.empty((Z, Hq, T))
    for z in range(Z):
        for h in range(Hq):
            x = scale * (q[z, h].double().numpy() @ k[z][h * k[z].shape[0] // Hq].T)
            x[np.arange(lens[z] + T)[None] > lens[z] + np.arange(T)[:, None]] = -math.inf
            top = x.max(1)
            lse[z, h] = top + np.log(np.exp(x - top[:, None]).sum(1))
    return torch.from_numpy(lse).float()


@pytest.mark.parametrize("dtype,scale", [("fp16", 2.0 ** 28), ("fp16", -2.0 ** 38), ("bf16", 2.0 ** 100)])
@pytest.mark.parametrize("T", [2, 40, 200])
def test_large_scales(T, dtype, scale):
    """Queries and keys nearly as small as the type has them under a scale that makes up for it: lse / scale may be too
    small for pieces of 16 bits."""
    lens, D, small = [3, 700], 64, 2.0 * abs(scale) ** -0.5
    kc, _, table, k, _ = pu.make_cache(21, [n + T for n in lens], 1, D, 16, dtype, garbage=0.0)
    kc = (kc.float() * small).to(pu.DT[dtype])
    k = [(torch.from_numpy(x) * small).to(pu.DT[dtype]).double().numpy() for x in k]
    q = (small * torch.randn(2, 2, T, D, generator=torch.Generator().manual_seed(22))).to(pu.DT[dtype])
    against_the_statement(q, sums(q, k, lens, scale), kc, k, table, lens, T, scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-30])
def test_scales_of_full_tiles(scale, dtype):
    check(24, [3, 200, 700], [200] * 3, 200, 2, 1, 64, 16, dtype, scale=scale, spread=0.5)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_sharp_attention_of_full_tiles(dtype):
    check(25, [700, 663], [200, 200], 200, 2, 1, 128, 16, dtype, spread=40.0)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_single_rows_of_full_tiles(dtype):
    """A full tile seen whole, one of whose rows has no sum, one an lse / scale just within fp16's pieces and one just
    outside: the tile's other rows are as they are without them."""
    T, D, lens = 256, 64, [700]
    scale = 0.125
    kc, _, table, k, _ = pu.make_cache(26, [lens[0] + T], 1, D, 16, dtype, garbage=0.0)
    q = torch.randn(1, 2, T, D, generator=torch.Generator().manual_seed(27))
    for t, target in ((5, 59000.0), (70, 61000.0), (130, -59000.0)):  # lse is proportional to so sharp a row
        q[0, 1, t] *= 1000
        for _ in range(3):
            rows = q.to(pu.DT[dtype])
            q[0, 1, t] *= abs(target) / (sums(rows, k, lens, scale)[0, 1, t].item() / scale)
        if target < 0:
            q[0, 1, t] *= -1
    q = q.to(pu.DT[dtype])
    lse = sums(q, k, lens, scale)
    ratio = lse / scale
    assert 55000 < ratio[0, 1, 5] < 60000 < ratio[0, 1, 70] < 65000
    lse[0, 0, 3] = lse[0, 1, 200] = -math.inf
    against_the_statement(q, lse, kc, k, table, lens, T, scale)
