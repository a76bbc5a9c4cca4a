"""Rotary positions against a statement in complex 64-bit numbers, element by element, and their gradients."""
import math

import numpy as np
import pytest
import torch

import budget_util as bu
import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import exact_attention_44_gb300 as fa
    fa.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def turns_of(R):
    import exact_attention_44_gb300 as fa
    return fa.fa_rope_turns(fa.fa_rope_frequencies(R))


def check(y, x, pos, R, dtype, interleaved, factor=1.0, inverse=False, far=0):
    want, size = bu.turn(x.double().cpu().numpy(), pos, bu.frequencies(R), interleaved, factor, inverse)
    off = np.abs(y.double().cpu().numpy() - want)
    assert (off <= bu.turn_bound(want, size, dtype, factor, far)).all(), off.max()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(16, 16), (16, 4), (32, 32), (32, 6), (64, 64), (64, 32), (64, 2), (128, 128),
                                 (128, 64), (128, 16), (128, 48), (128, 126), (256, 256), (256, 64), (256, 100)])
def test_every_width(dtype, interleaved, D, R):
    import exact_attention_44_gb300 as fa
    g = torch.Generator().manual_seed(D + R)
    q = torch.randn(2, 3, 37, D, generator=g).to(pu.DT[dtype])
    k = torch.randn(2, 37, 2, D, generator=g).to(pu.DT[dtype]).transpose(1, 2)  # a projection's layout
    yq, yk = fa.fa_rope(q.cuda(), k.transpose(1, 2).cuda().transpose(1, 2), turns_of(R), interleaved=interleaved)
    assert yk.stride() == k.stride() and yq.stride() == q.stride()
    pos = np.arange(37)[None].repeat(2, 0)
    check(yq, q, pos, R, dtype, interleaved)
    check(yk, k, pos, R, dtype, interleaved)
    assert torch.equal(yq[..., R:].cpu(), q[..., R:]) and torch.equal(yk[..., R:].cpu(), k[..., R:])


@pytest.mark.parametrize("N,Hq,Hk,Z", [(1, 1, 1, 1), (1, 8, 1, 1), (1, 32, 8, 64), (7, 5, 3, 2), (513, 12, 2, 1), (4099, 3, 0, 1)])
@pytest.mark.parametrize("where", ["new", "in place", "strided"])
def test_sizes_and_places(N, Hq, Hk, Z, where):
    import exact_attention_44_gb300 as fa
    D, R = 128, 64
    g = torch.Generator().manual_seed(N)
    q, k = (torch.randn(Z, h, N, D, generator=g).half() for h in (Hq, Hk))
    at = torch.randint(0, 5000, (Z, N), generator=g, dtype=torch.int32)
    pos = at.numpy()
    qg, kg = q.cuda(), k.cuda()
    if where == "in place":
        yq, yk = fa.fa_rope(qg, kg, turns_of(R), at.cuda(), factor=1.25, q_out=qg, k_out=kg)
        assert yq is qg or yq.data_ptr() == qg.data_ptr()
    elif where == "strided":  # padded rows, and what lies between them stays
        pad = [torch.full((Z, N, h + 1, D + 8), 9.0, dtype=torch.half, device="cuda") for h in (Hq, Hk)]
        outs = [p[:, :, :h, :D].transpose(1, 2) for p, h in zip(pad, (Hq, Hk))]
        yq, yk = fa.fa_rope(qg, kg, turns_of(R), at.cuda(), factor=1.25, q_out=outs[0], k_out=outs[1])
        for p, h in zip(pad, (Hq, Hk)):
            assert (p[:, :, h:] == 9).all() and (p[..., D:] == 9).all()
    else:
        yq, yk = fa.fa_rope(qg, kg, turns_of(R), at.cuda(), factor=1.25)
    check(yq, q, pos, R, "fp16", False, 1.25, far=5000)
    if Hk:
        check(yk, k, pos, R, "fp16", False, 1.25, far=5000)
    alone = fa.fa_rope(q.cuda(), None, turns_of(R), at.cuda(), factor=1.25)
    assert alone[1] is None and torch.equal(alone[0], yq)


@pytest.mark.parametrize("at", [-5, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_far_positions(at):
    import exact_attention_44_gb300 as fa
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 2, 1, 128, generator=g).half()
    y, _ = fa.fa_rope(q.cuda(), None, turns_of(128), i32([at]))
    check(y, q, np.array([[at]]), 128, "fp16", False, far=at)


def test_positions_shared_by_sequences_and_broadcast_rows():
    import exact_attention_44_gb300 as fa
    q = torch.randn(1, 1, 9, 64).half().cuda()
    pos = i32([4, 4, 0, 1, 2, 100, 7, 7, 8])
    y, k = fa.fa_rope(q.expand(3, 2, 9, 64), q.expand(3, 1, 9, 64), turns_of(64), pos)
    one, _ = fa.fa_rope(q, None, turns_of(64), pos[None])
    assert torch.equal(y, one.expand(3, 2, 9, 64)) and torch.equal(k, one.expand(3, 1, 9, 64))
    assert fa.fa_rope(q[:0], None, turns_of(64))[0].shape == (0, 1, 9, 64)
    assert fa.fa_rope(q[:, :, :0], q[:, :, :0], turns_of(64))[1].shape == (1, 1, 0, 64)


def test_special_values_stay_in_their_pair():
    import exact_attention_44_gb300 as fa
    q = torch.randn(1, 1, 2, 64).half()
    q[0, 0, 1, 3], q[0, 0, 1, 40] = float("nan"), float("inf")  # pairs 3 and 8 of row 1; 40 = 32 + 8
    y, _ = fa.fa_rope(q.cuda(), None, turns_of(64))
    bad = ~torch.isfinite(y.cpu())
    assert sorted(np.argwhere(bad[0, 0].numpy())[:, 1].tolist()) == [3, 8, 35, 40] and not bad[0, 0, 0].any()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_are_the_turn_back(dtype, interleaved):
    import exact_attention_44_gb300 as fa
    D, R, N = 64, 32, 21
    g = torch.Generator().manual_seed(5)
    q, k, dq, dk = (torch.randn(2, h, N, D, generator=g).to(pu.DT[dtype]) for h in (4, 2, 4, 2))
    pos = torch.randint(0, 3000, (2, N), generator=g, dtype=torch.int32)
    leaves = [t.cuda().requires_grad_() for t in (q, k)]
    y = fa.rotary(*leaves, turns_of(R), pos.cuda(), interleaved=interleaved, factor=0.75)
    check(y[0].detach(), q, pos.numpy(), R, dtype, interleaved, 0.75, far=3000)
    # gradients as they come: transposed, of one value, or for one output only
    gq, gk = torch.autograd.grad(y, leaves, (dq.cuda().transpose(1, 2).contiguous().transpose(1, 2), dk.cuda()), retain_graph=True)
    check(gq, dq, pos.numpy(), R, dtype, interleaved, 0.75, True, far=3000)
    check(gk, dk, pos.numpy(), R, dtype, interleaved, 0.75, True, far=3000)
    ones, = torch.autograd.grad(y[0].sum(), leaves[:1], retain_graph=True)
    check(ones, torch.ones_like(q), pos.numpy(), R, dtype, interleaved, 0.75, True, far=3000)
    only, = torch.autograd.grad(y[1], leaves[1:], dk.cuda())
    assert torch.equal(only, gk)


def test_gradient_against_differences():
    """Turning is linear: <dy, turn(x + h v) - turn(x)> / h is <grad, v>, up to both roundings to fp16."""
    import exact_attention_44_gb300 as fa
    g = torch.Generator().manual_seed(6)
    x, v, dy = (torch.randn(1, 2, 50, 64, generator=g).half() for _ in range(3))
    x2 = (x.float() + 0.5 * v.float()).half()
    leaf = x.cuda().requires_grad_()
    turns = turns_of(64)
    y, _ = fa.rotary(leaf, None, turns)
    grad, = torch.autograd.grad(y, leaf, dy.cuda())
    y2, _ = fa.fa_rope(x2.cuda(), None, turns)
    step = (x2.double() - x.double())
    got = (dy.double() * (y2.double() - y.detach().double()).cpu()).sum()
    want = (grad.double().cpu() * step).sum()
    # each output is off by 2^-11 of itself (its rounding) and 2^-21 of its pair
    bound = (dy.double().abs() * (y2.double().abs() + y.detach().double().abs()).cpu()).sum() * (2.0 ** -11 + 2.0 ** -19)
    bound += (grad.double().abs().cpu() * step.abs()).sum() * (2.0 ** -11 + 2.0 ** -19)
    assert abs(got - want) <= bound


def test_shared_and_broadcast_leaves():
    """A leaf that is both q and k, and one expanded over heads, get the sums of their gradients."""
    import exact_attention_44_gb300 as fa
    x = torch.randn(2, 1, 9, 64, device="cuda").half().requires_grad_()
    turns = turns_of(64)
    q, k = fa.rotary(x.expand(2, 3, 9, 64), x, turns)
    w = torch.randn(2, 4, 9, 64, device="cuda").half()
    (gx,) = torch.autograd.grad((q, k), x, (w[:, :3], w[:, 3:]))
    parts = fa.fa_rope(w, None, turns, inverse=True)[0]
    # three heads summed by torch in fp32 and rounded, and the fourth added and rounded: 2^-10 of the sizes
    assert ((gx.double() - parts.double().sum(1, keepdim=True)).abs() <= parts.double().abs().sum(1, keepdim=True) * 2.0 ** -10 + 2.0 ** -24).all()


def test_packed_sequences_with_attention():
    """Packed (total, H, D) rows, their positions from 0 in each sequence: attention_varlen of turned rows equals
    each sequence turned and attended to alone, bit by bit; and gradients flow through both."""
    import exact_attention_44_gb300 as fa
    lens, D = [5, 1, 130, 64], 64
    total = sum(lens)
    q, k, v = (torch.randn(total, h, D, device="cuda").half().requires_grad_() for h in (4, 2, 2))
    pos = i32([p for n in lens for p in range(n)])
    cu = i32([0] + np.cumsum(lens).tolist())
    turns = turns_of(D)
    tq, tk = fa.rotary(q, k, turns, pos)
    o = fa.attention_varlen(tq, tk, v, cu, cu, max(lens), max(lens), causal=True)
    do = torch.randn_like(o)
    grads = torch.autograd.grad(o, (q, k, v), do)
    at = 0
    for n in lens:
        s = [t.detach()[at:at + n][None].transpose(1, 2).contiguous().requires_grad_() for t in (q, k, v)]
        yq, yk = fa.rotary(s[0], s[1], turns)
        assert torch.equal(yq[0].transpose(0, 1), tq[at:at + n]) and torch.equal(yk[0].transpose(0, 1), tk[at:at + n])
        at += n
    # the gradient of the turned rows, turned back
    leaves = [t.detach().requires_grad_() for t in (tq, tk)]
    mid = torch.autograd.grad(fa.attention_varlen(*leaves, v, cu, cu, max(lens), max(lens), causal=True), leaves, do)
    back = fa.fa_rope(*(g[None].transpose(1, 2) for g in mid), turns, pos, inverse=True)
    assert torch.equal(grads[0], back[0][0].transpose(0, 1)) and torch.equal(grads[1], back[1][0].transpose(0, 1))
    with pytest.raises(ValueError, match="packed"):
        fa.rotary(q, k, turns)


def test_scores_depend_on_distance_only():
    """q at p against k at p' depends on p - p': the same pair of rows 10^9 positions further on."""
    import exact_attention_44_gb300 as fa
    g = torch.Generator().manual_seed(8)
    x = torch.randn(1, 2, 1, 128, generator=g).half().cuda()
    freq = fa.fa_rope_frequencies(128)
    # frequencies that are whole parts of a turn in 2^-40: no rounding at any position
    turns = (fa.fa_rope_turns(freq) >> 24) << 24
    pairs = []
    for at in (0, 10 ** 9):
        q, _ = fa.fa_rope(x, None, turns, i32([at + 700]))
        k, _ = fa.fa_rope(x, None, turns, i32([at]))
        pairs.append((q.double() * k.double()).sum(-1))
    # each element is off by 2^-11 of itself, in both factors and both places
    bound = 4 * 2.0 ** -11 * 1.01 * (x.double() ** 2).sum(-1) * 2
    assert ((pairs[0] - pairs[1]).abs() <= bound).all()


def test_another_stream_and_graph():
    import exact_attention_44_gb300 as fa
    q, k = torch.randn(2, 8, 300, 128, device="cuda").half(), torch.randn(2, 2, 300, 128, device="cuda").half()
    turns = turns_of(128)
    want = fa.fa_rope(q, k, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.fa_rope(q, k, turns, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.zeros_like(t) for t in (q, k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(q, k, turns, q_out=out[0], k_out=out[1])
    q.copy_(torch.randn_like(q))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], fa.fa_rope(q, k, turns)[0]) and torch.equal(out[1], want[1])


# ------------------------------------------------------------- into the cache

@pytest.mark.parametrize("D,R,interleaved", [(16, 16, False), (32, 10, True), (64, 32, False), (128, 128, True), (256, 64, False)])
@pytest.mark.parametrize("T,page", [(1, 16), (5, 48), (70, 32)])
@pytest.mark.parametrize("layout", ["phnd", "pnhd", "padded"])
def test_append(D, R, interleaved, T, page, layout):
    """Bit by bit fa_rope, then fa_cache_append."""
    import exact_attention_44_gb300 as fa
    lens, new = [0, 1, page - 1, page, 100], [T, 0, T, 1, max(0, T - 2)]
    kc, vc, table, _, _ = pu.make_cache(1, [a + T for a in lens], 3, D, page, "fp16", layout=layout, garbage=7.0)
    q = torch.randn(5, T, 6, D).half().cuda().transpose(1, 2)
    k, v = (torch.randn(5, T, 3, D).half().cuda().transpose(1, 2) for _ in range(2))
    turns, kw = turns_of(R), dict(interleaved=interleaved, factor=1.125)
    for pos in (None, torch.randint(0, 10 ** 6, (5, T), dtype=torch.int32, device="cuda")):
        at = i32(lens)[:, None] + torch.arange(T, dtype=torch.int32, device="cuda") if pos is None else pos
        tq, tk = fa.fa_rope(q, k, turns, at, **kw)
        want = pu.like(kc), pu.like(vc)
        fa.fa_cache_append(tk, v, *want, table.cuda(), i32(lens), new_lens=i32(new))
        got = pu.like(kc), pu.like(vc)
        out = torch.full_like(q, 5.0)
        assert fa.fa_cache_append_rope(q, k, v, *got, table.cuda(), i32(lens), turns, positions=pos, new_lens=i32(new),
                                       q_out=out, **kw).data_ptr() == out.data_ptr()
        assert fa.fa_device_status()[0] == 0
        for a, b in zip(got, want):
            assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))
        for z in range(5):
            assert torch.equal(out[z, :, :new[z]], tq[z, :, :new[z]]) and (out[z, :, new[z]:] == 5).all()
        # in place
        q2 = q.clone()
        fa.fa_cache_append_rope(q2, k, v, *got, table.cuda(), i32(lens), turns, positions=pos, new_lens=i32(new), q_out=q2, **kw)
        for z in range(5):
            assert torch.equal(q2[z, :, :new[z]], tq[z, :, :new[z]]) and torch.equal(q2[z, :, new[z]:], q[z, :, new[z]:])


def test_append_bad_pages():
    import exact_attention_44_gb300 as fa
    kc, vc, table, _, _ = pu.make_cache(2, [40, 40, 40], 2, 64, 16, "bf16", garbage=1.0)
    table[0, 1], table[1, 1] = -1, 5000
    q, k, v = (torch.randn(3, h, 20, 64).bfloat16().cuda() for h in (4, 2, 2))
    turns, lens = turns_of(64), i32([16, 10, 45])  # the third's table ends at 48
    want = kc.cuda(), vc.cuda()
    tq, tk = fa.fa_rope(q, k, turns, lens[:, None] + torch.arange(20, dtype=torch.int32, device="cuda"))
    fa.fa_cache_append(tk, v, *want, table.cuda(), lens)
    assert fa.fa_device_status()[0] == fa.FA_ERR_PAGE
    got = kc.cuda(), vc.cuda()
    out = fa.fa_cache_append_rope(q, k, v, *got, table.cuda(), lens, turns)
    assert fa.fa_device_status()[0] == fa.FA_ERR_PAGE
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(out, tq)


def test_gradient_of_the_gradient():
    """The gradient is a turn too: differentiated by what came in, it is the turn itself."""
    import exact_attention_44_gb300 as fa
    x = torch.randn(1, 2, 9, 64, device="cuda").half().requires_grad_()
    up = torch.randn(1, 2, 9, 64, device="cuda").half().requires_grad_()
    w = torch.randn(1, 2, 9, 64, device="cuda").half()
    turns = turns_of(32)
    y, none = fa.rotary(x, None, turns, factor=0.5)
    assert none is None
    grad, = torch.autograd.grad(y, x, up, create_graph=True)
    second, = torch.autograd.grad(grad, up, w)
    assert torch.equal(second, fa.fa_rope(w, None, turns, factor=0.5)[0])


def test_positions_changed_between_the_directions_are_noticed():
    import exact_attention_44_gb300 as fa
    x = torch.randn(1, 2, 9, 64, device="cuda").half().requires_grad_()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    y, _ = fa.rotary(x, None, turns_of(64), pos)
    pos += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_turns_changed_between_the_directions_are_noticed():
    import exact_attention_44_gb300 as fa
    x = torch.randn(1, 2, 9, 64, device="cuda").half().requires_grad_()
    turns = turns_of(64)
    y, _ = fa.rotary(x, None, turns)
    turns += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_backward_in_a_graph_and_on_another_stream():
    """Forward and backward of a layer (rotary, then attention) captured in a CUDA graph replay to the eager bits; and
    a side stream's gradients are that stream's."""
    import exact_attention_44_gb300 as fa
    turns = turns_of(64)
    q, k, v = (torch.randn(1, h, 130, 64, device="cuda").half() for h in (4, 2, 2))
    do = torch.randn(1, 4, 130, 64, device="cuda").half()

    def layer(a, b, c):
        x, y = fa.rotary(a, b, turns)
        return fa.attention(x, y, c, causal=True)

    def grads():
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        return torch.autograd.grad(layer(*leaves), leaves, do)

    want = grads()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = grads()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grads()
    keep = [t.clone() for t in (q, k, v)]
    for t in (q, k, v):
        t.zero_()
    graph.replay()
    for t, c in zip((q, k, v), keep):
        t.copy_(c)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
