"""The received attention weight where its kernels change their way."""
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
