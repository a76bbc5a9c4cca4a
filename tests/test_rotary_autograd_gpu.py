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
