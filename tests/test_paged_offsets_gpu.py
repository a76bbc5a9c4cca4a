"""Offsets past 2^31 elements in every hand-written address of the paged cache: append, commit and fork
(and attention's V) on caches whose pages, or whose layers, lie 4.3 GB apart, bit by bit against the same
calls on a compact cache."""
import pytest
import torch

import paged_util as pu

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 + 2048  # elements


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def far(c, dim):
    """The same (layers, pages, Hkv, page, D) values with dimension `dim` (0: layer, 1: page) FAR apart."""
    stride = list(c.contiguous().stride())
    stride[dim] = FAR
    if dim == 1:
        stride[0] = 16 * 64 * c.shape[2]  # the layers of a page side by side
    n = sum((a - 1) * b for a, b in zip(c.shape, stride)) + 1
    out = torch.empty(n, dtype=c.dtype, device="cuda").as_strided(c.shape, stride)
    out.copy_(c)
    return out


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("dim", [0, 1])
def test_append_commit_and_fork(dim):
    import exact_attention_44_gb300 as fa
    lens, T, L = [20, 5], 10, 3
    kc, vc, table, _, _ = pu.make_cache(1, lens, 2, 64, 16, "bf16", layers=L, extra=4, cols=4, garbage=1.0)
    refs = torch.bincount(table[table >= 0].flatten(), minlength=kc.shape[1]).int()
    rows = [torch.randn((L, 2, 2, T, 64), generator=torch.Generator().manual_seed(s)).bfloat16().cuda() for s in (2, 3)]
    results = []
    for place in (lambda c: c.cuda(), lambda c: far(c, dim)):
        k, v = place(kc), place(vc)
        t, n, r = table.cuda(), i32(lens), refs.cuda()
        missing = i32([-1])
        fa.fa_cache_fork(k, v, t, n, r, i32([0, 0]), room=T, missing=missing)  # the second becomes the first's copy
        for la in range(L):
            fa.fa_cache_append(rows[0][la], rows[1][la], k[la], v[la], t, n)
        fa.fa_cache_commit(k, v, t, n, i32([[1, 4, 9], [0, 7, 8]]), i32([3, 3]))
        assert missing.item() == 0 and fa.fa_device_status()[0] == 0
        results.append((k, v, t, n, r))
    assert all(torch.equal(a, b) for a, b in zip(results[0][2:], results[1][2:]))
    assert same(results[0][0], results[1][0]) and same(results[0][1], results[1][1])
    t = results[0][2]
    assert t.max().item() >= 1  # (a page that is far away, dim 1)
    # the second sequence holds the first one's rows, then its own committed ones
    k = results[1][0]
    for i, j in enumerate((0, 7, 8)):
        p, s = divmod(20 + i, 16)
        assert same(k[:, t[1, p], :, s], rows[0][:, 1, :, j])
    assert same(k[:, t[1, 1], :, :4], k[:, t[0, 1], :, :4])


@pytest.mark.parametrize("T", [1, 39])
def test_attention_with_both_caches_far_apart(T):
    import exact_attention_44_gb300 as fa
    kc, vc, table, _, _ = pu.make_cache(4, [40], 1, 64, 16, "bf16", extra=0)
    q = torch.randn((1, 4, T, 64), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    lens = i32([40 - T])
    a = fa.fa_fwd_paged(q, far(kc[None], 1)[0], far(vc[None], 1)[0], table.cuda(), lens)
    b = fa.fa_fwd_paged(q, kc.cuda(), vc.cuda(), table.cuda(), lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and fa.fa_device_status()[0] == 0
