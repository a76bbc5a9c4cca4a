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
