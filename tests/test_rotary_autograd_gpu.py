"""rotary as a node of autograd's graph: which side it turns back, what it refuses, and tensors that calls write in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def rows(seed=1):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(2, h, 33, 64, generator=g).half().cuda() for h in (4, 2)]


def turns_of(R):
    import exact_attention_44_gb300 as fa
    return fa.fa_rope_turns(fa.fa_rope_frequencies(R))


def test_forward_mode_is_refused():
    """A tangent would be lost; on either side, and of a gradient that comes back."""
    import torch.autograd.forward_ad as fwd

    import exact_attention_44_gb300 as fa
    (q, k), turns = rows(), turns_of(64)
    with fwd.dual_level():
        dual = [fwd.make_dual(t, torch.ones_like(t)) for t in (q, k)]
        for args in ((dual[0], k), (q, dual[1]), (dual[0], None)):
            with pytest.raises(NotImplementedError, match="tangent"):
                fa.rotary(*args, turns)
        with pytest.raises(NotImplementedError, match="tangent"):
            fa.rotary(dual[0][:, :, 0], None, turns, torch.zeros(2, dtype=torch.int32, device="cuda"))
        x = q.detach().requires_grad_()
        y, _ = fa.rotary(x, None, turns)
        with pytest.raises(NotImplementedError, match="tangent"):
            torch.autograd.grad(y, x, dual[0])
        fa.rotary(q, k, turns)  # (no tangent, no refusal)
    fa.rotary(fwd.unpack_dual(dual[0]).primal, k, turns)


@pytest.mark.parametrize("needed", [(True, False), (False, True), (True, True), (False, False)])
def test_only_what_needs_a_gradient_is_in_the_graph(needed):
    import exact_attention_44_gb300 as fa
    turns, grads = turns_of(32), rows(2)
    both = [t.clone().requires_grad_() for t in rows()]
    want = torch.autograd.grad(fa.rotary(*both, turns), both, grads)
    some = [t.clone().requires_grad_(n) for t, n in zip(rows(), needed)]
    y = fa.rotary(*some, turns)
    assert tuple(t.requires_grad for t in y) == needed
    for t, u, g, n, w in zip(y, some, grads, needed, want):
        if n:
            assert torch.equal(torch.autograd.grad(t, u, g, retain_graph=True)[0], w)
    for t, u in zip(y, fa.fa_rope(*rows(), turns)):
        assert torch.equal(t, u)


@pytest.mark.parametrize("side", [0, 1])
def test_only_what_is_asked_for_is_turned_back(side):
    """Both sides need gradients and both come back, but only one leaf's is asked for: one tensor is made, as where there
    is only that side."""
    import exact_attention_44_gb300 as fa
    turns, grads = turns_of(64), rows(3)
    leaves = [t.requires_grad_() for t in rows()]

    def made(outs, leaf, up):
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        g, = torch.autograd.grad(outs, leaf, up, retain_graph=True)
        return torch.cuda.memory_stats()["allocation.all.allocated"] - before, g

    alone, want = made(fa.rotary(leaves[side], None, turns)[0], leaves[side], grads[side])
    n, g = made(fa.rotary(*leaves, turns), leaves[side], grads)
    assert torch.equal(g, want) and n == alone == 1


def test_tensors_written_in_place_are_noticed():
    """Autograd saved q for its square; turned in place, it is no longer what was squared."""
    import exact_attention_44_gb300 as fa
    q, k = rows()
    turns = turns_of(64)
    page = torch.zeros(8, 2, 16, 64, dtype=torch.half, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    calls = (lambda x: fa.fa_rope(x, None, turns, q_out=x), lambda x: fa.fa_rope(q.clone(), x[:, :2], turns, k_out=x[:, :2]),
             lambda x: fa.fa_cache_append_rope(x, k, k, page, page.clone(), table, lens, turns, q_out=x))
    for call in calls:
        x = (q.detach().clone().requires_grad_() * 1.0)
        y = x * x
        call(x.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_what_a_call_writes_has_a_new_version():
    import exact_attention_44_gb300 as fa
    i32 = dict(dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(2, 8, 2, 16, 64, dtype=torch.half, device="cuda") for _ in range(2))
    table, lens, refs = torch.arange(8, **i32).view(2, 4), torch.full((2,), 30, **i32), torch.ones(8, **i32)
    scores, missing, turns = torch.zeros(2, 2, 2, 64, device="cuda"), torch.zeros(1, **i32), turns_of(64)
    q, k = (torch.randn(2, h, 1, 64, device="cuda").half() for h in (4, 2))
    out = torch.empty_like(q)

    def moved(call, written, read):
        before = [t._version for t in (*written, *read)]
        call()
        after = [t._version for t in (*written, *read)]
        n = len(written)
        assert all(a > b for a, b in zip(after[:n], before[:n])) and after[n:] == before[n:]

    moved(lambda: fa.fa_rope(q, k, turns, q_out=out), [out], [q, k])
    moved(lambda: fa.fa_cache_append_rope(q, k, k, kc[0], vc[0], table, lens, turns, q_out=out), [out, kc, vc], [q, k, table, lens])
    lse = torch.zeros(2, 4, 1, device="cuda")
    moved(lambda: fa.fa_cache_score(q, lse, kc[0], table, lens, scores[0]), [scores], [q, lse, kc, table, lens])
    moved(lambda: fa.fa_cache_evict(kc, vc, table, lens, refs, scores, 20, missing),
          [kc, vc, table, lens, refs, scores, missing], [])
    with torch.inference_mode():  # (tensors without versions)
        x = torch.randn(2, 4, 3, 64, device="cuda").half()
    with torch.inference_mode():
        fa.fa_rope(x, None, turns, q_out=x)
    fa.fa_rope(x, None, turns, q_out=x)
