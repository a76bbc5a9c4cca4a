"""Rotary positions and the budgeted cache on the host: frequencies and turns, refusals before anything is enqueued
(no GPU needed), and invariants of the plain statements."""
import ctypes
import math

import numpy as np
import pytest
import torch

import budget_util as bu
import exact_attention_44_gb300 as fa
import paged_util as pu


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


# ------------------------------------------------------------- frequencies

def test_frequencies(lib):
    R, s, ctx = 64, 4.0, 2048.0
    plain = 10000.0 ** (-2 * np.arange(32) / R)
    f = {k: fa.fa_rope_frequencies(R, scaling=k, stretch=s, context=ctx).numpy() for k in ("none", "linear", "base", "ramp")}
    assert np.allclose(f["none"], plain, rtol=1e-14) and np.allclose(f["linear"], plain / s, rtol=1e-14)
    # base: the fastest pair stays, the slowest is stretched in full
    assert f["base"][0] == 1.0 and np.isclose(f["base"][-1], plain[-1] / s, rtol=1e-13)
    turns = ctx * plain / (2 * math.pi)
    assert np.allclose(f["ramp"][turns >= 32], plain[turns >= 32], rtol=1e-14)
    assert np.allclose(f["ramp"][turns <= 1], plain[turns <= 1] / s, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((f["ramp"][mid] < plain[mid]) & (f["ramp"][mid] > plain[mid] / s)).all()
    assert fa.fa_rope_frequencies(2, scaling="base", stretch=8.0).tolist() == [1.0]
    assert np.allclose(fa.fa_rope_frequencies(8, base=500000.0).numpy(), 500000.0 ** (-np.arange(4) / 4), rtol=1e-14)


def test_turns_are_exact_fractions(lib):
    f = torch.tensor([2 * math.pi / 4, 2 * math.pi, -2 * math.pi / 8, 0.0, 2 * math.pi * 5.5, 1.0, 1e-4], dtype=torch.float64)
    t = fa.fa_rope_turns(f).tolist()
    assert t[:4] == [1 << 62, 0, -(1 << 61), 0]
    # 5.5 turns in 53 bits, in radians and then in turns: half a turn but for 5.5 x 2^-52 of one
    assert abs(abs(t[4]) - (1 << 63)) <= 5.5 * 2.0 ** (64 - 52)
    assert fa.fa_rope_turns(torch.tensor([math.pi], dtype=torch.float64)).item() == -(1 << 63)  # (half a turn either way)
    # the product with any position wraps to the same fraction, off by p 2^-65 turns and the frequency's rounding
    from fractions import Fraction
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    for p in (1, 4097, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        for i in (5, 6):
            got = Fraction((t[i] * p) % (1 << 64), 1 << 64)
            d = (got - Fraction(f[i].item()) * p / two_pi) % 1
            assert min(d, 1 - d) <= abs(p) * (Fraction(1, 2 ** 65) + Fraction(f[i].item()) * Fraction(1, 2 ** 54))
    assert fa.fa_rope_turns(torch.tensor([0.5])).dtype == torch.int64  # float32 frequencies too


def test_frequency_refusals(lib):
    for bad in (dict(base=0.0), dict(base=-1.0), dict(base=math.nan), dict(scaling="linear", stretch=0.0),
                dict(scaling="base", stretch=math.inf), dict(scaling="ramp", stretch=2.0),
                dict(scaling="ramp", stretch=2.0, context=100.0, slow=4.0, fast=4.0)):
        with pytest.raises(fa.FaError):
            fa.fa_rope_frequencies(64, **bad)
    for R in (0, 3, -2):
        with pytest.raises(ValueError):
            fa.fa_rope_frequencies(R)
    with pytest.raises(ValueError, match="scaling"):
        fa.fa_rope_frequencies(64, scaling="other")
    for bad in (math.nan, math.inf):
        with pytest.raises(fa.FaError):
            fa.fa_rope_turns(torch.tensor([1.0, bad]))
    with pytest.raises(ValueError):
        fa.fa_rope_turns(torch.ones(2, 2))
    x = (ctypes.c_double * 1)(1.0)
    y = (ctypes.c_int64 * 1)()
    assert lib.fa_rope_turns(-1, x, y) == lib.fa_rope_turns(1, None, y) == lib.fa_rope_turns(1, x, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_rope_turns(0, None, None) == fa.FA_OK
    assert lib.fa_rope_frequencies(64, None, None) == fa.FA_ERR_INVALID_ARG


# ------------------------------------------------------------- C arguments

PTR = 0x10000


class Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("b", "h", "n", "d")]


def _st(b, h, n, d=1):
    return Strides(b, h, n, d)


class Cache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v")] + [("sk", Strides), ("sv", Strides)] +
                [(n, ctypes.c_int64) for n in ("k_layer", "v_layer")] +
                [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p)] +
                [(n, ctypes.c_int) for n in ("Z", "L", "P", "Hkv", "page", "D", "M")])


class Rope(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "qo", "ko")] + [(n, Strides) for n in ("sq", "sk", "sqo", "sko")] +
                [("pos", ctypes.c_void_p), ("pos_stride", ctypes.c_int64), ("turns", ctypes.c_void_p)] +
                [(n, ctypes.c_int) for n in ("Z", "Hq", "Hk", "N", "D", "R", "inter", "inverse")] +
                [("factor", ctypes.c_float), ("dtype", ctypes.c_int)])


class AppendRope(ctypes.Structure):
    _fields_ = ([("cache", Cache)] + [(n, ctypes.c_void_p) for n in ("q", "qo", "k", "v")] +
                [(n, Strides) for n in ("sq", "sqo", "sk", "sv")] + [("new", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("pos_stride", ctypes.c_int64), ("turns", ctypes.c_void_p)] +
                [(n, ctypes.c_int) for n in ("Hq", "T", "R", "inter")] + [("factor", ctypes.c_float), ("dtype", ctypes.c_int)])


class Score(ctypes.Structure):
    _fields_ = ([("cache", Cache)] + [(n, ctypes.c_void_p) for n in ("q", "lse", "scores")] +
                [(n, ctypes.c_int64) for n in ("ss", "sh")] + [("sq", Strides), ("new", ctypes.c_void_p), ("ws", ctypes.c_void_p),
                ("wsb", ctypes.c_size_t), ("Hq", ctypes.c_int), ("T", ctypes.c_int), ("scale", ctypes.c_float),
                ("decay", ctypes.c_float), ("dtype", ctypes.c_int)])


class Evict(ctypes.Structure):
    _fields_ = ([("cache", Cache), ("refs", ctypes.c_void_p), ("scores", ctypes.c_void_p)] +
                [(n, ctypes.c_int64) for n in ("sl", "ss", "sh")] + [(n, ctypes.c_void_p) for n in ("keep", "missing", "ws")] +
                [("wsb", ctypes.c_size_t)] + [(n, ctypes.c_int) for n in ("budget", "first", "recent")])


def _cache(kc=PTR, vc=PTR, table=PTR, lens=PTR, Z=2, L=1, P=9, H=2, page=16, D=64, M=4, ts=4, kl=1 << 16, sc=None):
    sc = sc or _st(H * page * D, page * D, D)
    return Cache(kc, vc, sc, sc, kl, kl, table, ts, lens, Z, L, P, H, page, D, M)


I, U, A, W, OK = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_ALIGNMENT, fa.FA_ERR_WORKSPACE, fa.FA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(Z=-1), I), (dict(Hq=-1), I), (dict(N=-1), I), (dict(R=0), I), (dict(R=7), I), (dict(R=66), I), (dict(inter=2), I),
    (dict(inverse=-1), I), (dict(factor=math.nan), I), (dict(factor=math.inf), I), (dict(q=None), I), (dict(ko=None), I),
    (dict(turns=None), I), (dict(ps=-1), I), (dict(so=_st(0, 192, 64)), I), (dict(D=96), U), (dict(dtype=2), U),
    (dict(Z=65536), U), (dict(Hq=65535), U), (dict(N=(1 << 30) + 1), U), (dict(q=PTR + 8), A), 
    (dict(pos=PTR + 2), A), (dict(so=_st(768, 190, 64)), A), (dict(so=_st(768, 192, 64, 2)), A),
    (dict(ko=PTR), I), (dict(qo=PTR + 4096), I), (dict(ko=PTR, k=PTR + 64), I),
    (dict(so=_st(1536, 384, 128)), I), (dict(so=_st(8, 192, 64), Z=1, N=0), OK),
    (dict(Z=0), OK), (dict(N=0), OK), (dict(Hq=0, Hk=0), OK),
])
def test_rope_arguments(lib, kw, code):
    # q in place at PTR, k in place at PTR + 4096
    k = dict(q=PTR, qo=PTR, k=PTR + 4096, ko=PTR + 4096, turns=PTR, pos=None, ps=0, so=None, Z=2, Hq=4, Hk=2, N=3, D=64, R=32, inter=0, inverse=0,
             factor=1.0, dtype=0) | kw
    st = _st(k["Hq"] * k["N"] * k["D"], k["N"] * k["D"], k["D"])
    a = Rope(k["q"], k["k"], k["qo"], k["ko"], st, st, k["so"] or st, st, k["pos"], k["ps"], k["turns"], k["Z"], k["Hq"], k["Hk"],
             k["N"], k["D"], k["R"], k["inter"], k["inverse"], k["factor"], k["dtype"])
    assert lib.fa_rope(ctypes.addressof(a), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), I), (dict(Hq=-1), I), (dict(L=2), I), (dict(R=80), I), (dict(inter=3), I), (dict(factor=-math.inf), I),
    (dict(q=None), I), (dict(v=None), I), (dict(kc=None), I), (dict(turns=None), I), (dict(lens=None), I),
    (dict(sc=_st(0, 1024, 64)), I), (dict(dtype=-1), U), (dict(D=40), U), (dict(page=24), U), (dict(T=(1 << 30) + 1), U),
    (dict(k=PTR + 2), A), (dict(new=PTR + 1), A), (dict(pos=PTR + 1), A), (dict(qo=PTR + 4096), I),
    (dict(so=_st(1536, 384, 128)), I), (dict(Z=0), OK), (dict(T=0), OK),
])
def test_append_rope_arguments(lib, kw, code):
    k = dict(q=PTR, qo=PTR, k=PTR + 4096, v=PTR + 4096, turns=PTR, pos=None, new=None, T=3, Hq=4, R=32, inter=0, factor=1.0, dtype=1, so=None) | kw
    c = _cache(**{n: k.pop(n) for n in list(k) if n in ("kc", "lens", "L", "sc", "D", "page", "Z")})
    st = _st(4 * k["T"] * c.D, k["T"] * c.D, c.D)
    a = AppendRope(c, k["q"], k["qo"], k["k"], k["v"], st, k["so"] or st, st, st, k["new"], k["pos"], 0, k["turns"], k["Hq"], k["T"], k["R"],
                   k["inter"], k["factor"], k["dtype"])
    assert lib.fa_cache_append_rope(ctypes.addressof(a), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3), I), (dict(H=0), I), (dict(T=-1), I), (dict(L=2), I), (dict(ss=-1), I), (dict(sh=63), I), (dict(ss=63), I),
    (dict(scale=math.nan), I), (dict(decay=math.inf), I), (dict(q=None), I), (dict(lse=None), I), (dict(scores=None), I),
    (dict(kc=None), I), (dict(lens=None), I), (dict(table=None), I), (dict(D=24), U), (dict(dtype=3), U), (dict(T=1 << 30), U),
    (dict(M=1 << 27), U), (dict(scores=PTR + 2), A), (dict(lse=PTR + 1), A), (dict(new=PTR + 2), A), (dict(q=PTR + 4), A),
    (dict(ws=None), W), (dict(ws=PTR + 16), W), (dict(Z=0), OK), (dict(P=0), OK), (dict(M=0, ts=0), OK),
])
def test_score_arguments(lib, kw, code):
    k = dict(q=PTR, lse=PTR, scores=PTR, ss=128, sh=64, new=None, ws=PTR, wsb=1 << 40, Hq=4, T=3, scale=0.1, decay=1.0,
             dtype=0) | kw
    c = _cache(vc=None, **{n: k.pop(n) for n in list(k) if n in ("kc", "lens", "L", "D", "page", "Z", "P", "M", "H", "table", "ts")})
    a = Score(c, k["q"], k["lse"], k["scores"], k["ss"], k["sh"], _st(4 * 3 * c.D, 3 * c.D, c.D), k["new"], k["ws"], k["wsb"],
              k["Hq"], k["T"], k["scale"], k["decay"], k["dtype"])
    assert lib.fa_cache_score(ctypes.addressof(a), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(budget=-1), I), (dict(first=-1), I), (dict(recent=-1), I), (dict(missing=None), I), (dict(refs=None), I),
    (dict(scores=None), I), (dict(lens=None), I), (dict(kc=None), I), (dict(ts=3), I), (dict(sh=60), I), (dict(sl=60), I),
    (dict(sc=_st(0, 1024, 64)), I), (dict(D=24), U), (dict(page=20), U), (dict(L=65536), U), (dict(P=(1 << 30) + 1), U),
    (dict(Z=65535, M=1 << 16, ts=1 << 16), U), (dict(L=4096, H=65536), U),
    (dict(scores=PTR + 2), A), (dict(keep=PTR + 1), A), (dict(missing=PTR + 2), A), (dict(kl=12), A),
    (dict(ws=None), W), (dict(ws=PTR + 8), W), (dict(wsb=64), W),
])
def test_evict_arguments(lib, kw, code):
    k = dict(refs=PTR, scores=PTR, sl=256, ss=128, sh=64, keep=None, missing=PTR, ws=PTR, wsb=1 << 50, budget=20, first=0,
             recent=0, L=2) | kw
    c = _cache(**{n: k.pop(n) for n in list(k) if n in ("kc", "lens", "L", "D", "page", "Z", "P", "M", "H", "ts", "sc", "kl")})
    a = Evict(c, k["refs"], k["scores"], k["sl"], k["ss"], k["sh"], k["keep"], k["missing"], k["ws"], k["wsb"], k["budget"],
              k["first"], k["recent"])
    assert lib.fa_cache_evict(ctypes.addressof(a), None) == code


def test_null_and_sizes(lib):
    for call in (lib.fa_rope, lib.fa_cache_append_rope, lib.fa_cache_score, lib.fa_cache_evict):
        assert call(None, None) == I
    n = ctypes.c_size_t()
    assert lib.fa_cache_evict_workspace_size(1, -1, 1, 1, 1, ctypes.byref(n)) == I
    assert lib.fa_cache_evict_workspace_size(1, 1, 1, 1, 1, None) == I
    big = 2 ** 31 - 1
    assert lib.fa_cache_evict_workspace_size(big, big, big, big, big, ctypes.byref(n)) == U
    assert fa.fa_cache_evict_workspace_size(2, 3, 4, 5, 6) >= 4 * (2 * 3 * 4 * 7 + 3 * 3 * 5)
    assert lib.fa_cache_score_workspace_size(None) == I


# ------------------------------------------------------------- Python arguments

def test_python_rope_checks(lib):
    turns = torch.zeros(16, dtype=torch.int64)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.half)
    for change, error in [(dict(q=q[0]), ValueError), (dict(q=q.float()), TypeError), (dict(k=q.bfloat16()), TypeError),
                          (dict(k=q[:1]), ValueError), (dict(k=q[:, :, :2]), ValueError), (dict(turns=turns.int()), ValueError),
                          (dict(turns=turns[None]), ValueError), (dict(positions=torch.zeros(4, dtype=torch.int32)), ValueError),
                          (dict(positions=torch.zeros(3)), TypeError), (dict(q_out=q[:1]), ValueError),
                          (dict(q_out=q.float()), ValueError), (dict(k=None, k_out=q), ValueError), (dict(factor="x"), TypeError),
                          (dict(), ValueError)]:  # (tensors of the CPU)
        with pytest.raises(error):
            fa.fa_rope(**{**dict(q=q, k=q, turns=turns), **change})


def test_python_cache_checks(lib):
    i32 = dict(dtype=torch.int32)
    c = torch.zeros(9, 2, 16, 64, dtype=torch.half)
    t, n = torch.zeros(2, 4, **i32), torch.zeros(2, **i32)
    q, k = torch.zeros(2, 4, 3, 64, dtype=torch.half), torch.zeros(2, 2, 3, 64, dtype=torch.half)
    turns, s, lse = torch.zeros(16, dtype=torch.int64), torch.zeros(2, 2, 64), torch.zeros(2, 4, 3)
    good = dict(q=q, k=k, v=k, k_cache=c, v_cache=c, block_table=t, seq_lens=n, turns=turns)
    for change, error in [(dict(q=q[:, :, :2]), ValueError), (dict(k=q), ValueError), (dict(v=k[:, :1]), ValueError),
                          (dict(q=q.bfloat16()), TypeError), (dict(q=q.float()), TypeError), (dict(new_lens=n[:1]), ValueError),
                          (dict(positions=n), ValueError), (dict(q_out=k), ValueError), (dict(turns=t), ValueError), (dict(), ValueError)]:
        with pytest.raises(error):
            fa.fa_cache_append_rope(**{**good, **change})
    good = dict(q=q, lse=lse, k_cache=c, block_table=t, seq_lens=n, scores=s)
    for change, error in [(dict(lse=lse.double()), ValueError), (dict(lse=lse[:, :2]), ValueError), (dict(scores=s.half()), TypeError),
                          (dict(scores=s[..., :63]), ValueError), (dict(scores=s[None]), ValueError), (dict(scores=s[:1]), ValueError),
                          (dict(scores=torch.zeros(2, 2, 128)[..., ::2]), ValueError), (dict(k_cache=c[None]), ValueError),
                          (dict(k_cache=c.bfloat16()), TypeError), (dict(decay=None), TypeError), (dict(), ValueError)]:
        with pytest.raises(error):
            fa.fa_cache_score(**{**good, **change})
    good = dict(k_cache=c, v_cache=c, block_table=t, seq_lens=n, ref_counts=torch.zeros(9, **i32), scores=s, budget=3,
                missing=torch.zeros(1, **i32))
    for change, error in [(dict(ref_counts=n), ValueError), (dict(scores=s[None]), ValueError), (dict(missing=n), ValueError),
                          (dict(missing=None), TypeError), (dict(keep=n[:1]), ValueError), (dict(keep=s), TypeError),
                          (dict(k_cache=c[None], v_cache=c[None]), ValueError), (dict(budget=1 << 40), ValueError),
                          (dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 20)), ValueError), (dict(), ValueError)]:
        with pytest.raises(error):
            fa.fa_cache_evict(**{**good, **change})


def test_rotary_refuses_forward_mode(lib):
    """A tangent is refused before anything else is looked at: it would be lost, and read as a derivative of zero."""
    import torch.autograd.forward_ad as fwd

    turns = torch.zeros(32, dtype=torch.int64)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.half)
    with fwd.dual_level():
        dual = fwd.make_dual(q, torch.ones_like(q))
        for args in ((dual, None), (dual, q), (q, dual)):
            with pytest.raises(NotImplementedError, match="tangent"):
                fa.rotary(*args, turns)
        with pytest.raises(ValueError, match="CUDA"):
            fa.rotary(q, q, turns)


# ------------------------------------------------------------- the plain statements

def test_turn_statement():
    r = np.random.RandomState(0)
    x, pos, f = r.randn(1, 1, 3, 8), np.array([[0, 1, 5]]), bu.frequencies(4)
    y, _ = bu.turn(x, pos, f, True)
    assert np.array_equal(y[0, 0, 0], x[0, 0, 0]) and np.array_equal(y[..., 4:], x[..., 4:])
    a = 5 * f[1]
    assert np.allclose(y[0, 0, 2, 2:4], [x[0, 0, 2, 2] * math.cos(a) - x[0, 0, 2, 3] * math.sin(a),
                                         x[0, 0, 2, 2] * math.sin(a) + x[0, 0, 2, 3] * math.cos(a)])
    assert np.allclose(bu.turn(y, pos, f, True, inverse=True)[0], x)
    perm = [0, 2, 1, 3, 4, 5, 6, 7]  # the half layout is the interleaved one of reordered elements
    assert np.allclose(bu.turn(x[..., perm], pos, f, False)[0], y[..., perm])


def test_score_statement_sums_to_the_rows():
    r = np.random.RandomState(1)
    q, k = r.randn(1, 4, 3, 8), [r.randn(2, 8, 8)]
    _, lse = pu.attention(q, k, k, [5], [3], None, 0.3)
    s, _ = bu.score(q, lse, k, [5], [3], np.zeros((1, 2, 10)), 1.0, 0.3)
    assert np.allclose(s[0].sum(1), 2 * 3) and (s[0, :, 8:] == 0).all() and (s[0, :, :8] > 0).all()


def test_evict_statement_keeps_the_counts():
    r = np.random.RandomState(2)
    page, P, Z, M = 16, 40, 4, 6
    for _ in range(50):
        lens = r.randint(0, 96, Z).tolist()
        ids = r.permutation(P).tolist()
        table = [[ids.pop() if c * page < n else -1 for c in range(M)] for n in lens]
        for c in range(min(lens[0], lens[1]) // page // 2):
            table[1][c] = table[0][c]
        refs = np.bincount([p for row in table for p in row if p >= 0], minlength=P).tolist()
        t, n, refs2, missing, kept = bu.evict(table, lens, refs, r.rand(2, Z, 1, 96), page, 30, None, 2, 5)
        assert np.bincount([p for row in t for p in row if p >= 0], minlength=P).tolist() == refs2
        for z in range(Z):
            assert n[z] == (min(lens[z], 30) if not missing else lens[z])
            if kept[z] is not None:
                assert sum(p >= 0 for p in t[z]) == 2
