"""The paged-cache entry points refuse bad arguments on the host, before anything is enqueued (no
GPU needed), and the plain statement of fork's bookkeeping keeps its invariants."""
import ctypes
import importlib

import numpy as np
import pytest
import torch

import exact_attention_44_gb300 as fa
import paged_util as pu


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


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


class Attend(ctypes.Structure):
    _fields_ = [("cache", Cache), ("q", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("sq", Strides), ("so", Strides), ("new", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_stride", ctypes.c_int64), ("ws", ctypes.c_void_p), ("wsb", ctypes.c_size_t), ("Hq", ctypes.c_int),
                ("T", ctypes.c_int), ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class Append(ctypes.Structure):
    _fields_ = [("cache", Cache), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("sk", Strides), ("sv", Strides),
                ("new", ctypes.c_void_p), ("T", ctypes.c_int)]


class Commit(ctypes.Structure):
    _fields_ = [("cache", Cache), ("path", ctypes.c_void_p), ("path_stride", ctypes.c_int64), ("kept", ctypes.c_void_p),
                ("A", ctypes.c_int)]


class Fork(ctypes.Structure):
    _fields_ = [("cache", Cache), ("refs", ctypes.c_void_p), ("src", ctypes.c_void_p), ("miss", ctypes.c_void_p),
                ("ws", ctypes.c_void_p), ("wsb", ctypes.c_size_t), ("room", ctypes.c_int)]


def _cache(kc=PTR, table=PTR, lens=PTR, Z=2, L=1, P=9, H=2, page=16, D=64, M=4, ts=4, kl=1 << 16, sc=None):
    sc = sc or _st(H * page * D, page * D, D)
    return Cache(kc, kc, sc, sc, kl, kl, table, ts, lens, Z, L, P, H, page, D, M)


def _attend(lib, *, q=PTR, k=PTR, o=PTR, lse=PTR, table=PTR, lens=PTR, new=None, mask=None, Z=2, Hq=4, Hkv=2, T=3,
            D=64, P=9, page=16, M=4, L=1, ts=4, ms=0, sq=None, sk=None, so=None, scale=0.1, dtype=0, ws=PTR,
            wsb=1 << 40):
    st = _st(Hq * T * D, T * D, D)
    a = Attend(_cache(k, table, lens, Z, L, P, Hkv, page, D, M, ts, 1 << 16, sk), q, o, lse, sq or st, so or st, new, mask,
               ms, ws, wsb, Hq, T, scale, dtype)
    return lib.fa_fwd_paged(ctypes.addressof(a), None)


@pytest.mark.parametrize("kw,code", [
    (dict(Z=-1), fa.FA_ERR_INVALID_ARG), (dict(T=-1), fa.FA_ERR_INVALID_ARG), (dict(Hq=3), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(L=2), fa.FA_ERR_INVALID_ARG), (dict(P=-1), fa.FA_ERR_INVALID_ARG), (dict(M=-1), fa.FA_ERR_INVALID_ARG),
    (dict(ts=-4), fa.FA_ERR_INVALID_ARG), (dict(ms=-1), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG), (dict(scale=3e38), fa.FA_ERR_INVALID_ARG),
    (dict(q=None), fa.FA_ERR_INVALID_ARG), (dict(k=None), fa.FA_ERR_INVALID_ARG), (dict(o=None), fa.FA_ERR_INVALID_ARG),
    (dict(table=None), fa.FA_ERR_INVALID_ARG), (dict(lens=None), fa.FA_ERR_INVALID_ARG),
    (dict(so=_st(0, 64, 64)), fa.FA_ERR_INVALID_ARG),  # batches of o folded together
    (dict(D=96), fa.FA_ERR_UNSUPPORTED), (dict(dtype=2), fa.FA_ERR_UNSUPPORTED), (dict(page=8), fa.FA_ERR_UNSUPPORTED),
    (dict(page=24), fa.FA_ERR_UNSUPPORTED), (dict(page=0), fa.FA_ERR_UNSUPPORTED),
    (dict(M=1 << 27), fa.FA_ERR_UNSUPPORTED), (dict(Z=65536), fa.FA_ERR_UNSUPPORTED),
    (dict(T=1 << 30), fa.FA_ERR_UNSUPPORTED),
    (dict(q=PTR + 8), fa.FA_ERR_ALIGNMENT), (dict(sk=_st(1024, 1028, 64)), fa.FA_ERR_ALIGNMENT),
    (dict(sk=_st(2048, 1024, 64, 2)), fa.FA_ERR_ALIGNMENT), (dict(sq=_st(-768, 192, 64)), fa.FA_ERR_ALIGNMENT),
    (dict(table=PTR + 2), fa.FA_ERR_ALIGNMENT), (dict(lens=PTR + 1), fa.FA_ERR_ALIGNMENT),
    (dict(new=PTR + 2), fa.FA_ERR_ALIGNMENT), (dict(mask=PTR + 2), fa.FA_ERR_ALIGNMENT),
    (dict(lse=PTR + 2), fa.FA_ERR_ALIGNMENT), (dict(ws=None), fa.FA_ERR_WORKSPACE),
    (dict(ws=PTR + 16), fa.FA_ERR_WORKSPACE),
    (dict(Z=0), fa.FA_OK), (dict(T=0), fa.FA_OK), (dict(Hq=0), fa.FA_OK),
])
def test_attention_arguments(lib, kw, code):
    assert _attend(lib, **kw) == code


def _append(lib, *, k=PTR, T=3, new=None, sk=None, **kw):
    c = _cache(**kw)
    st = sk or _st(c.Hkv * T * c.D, T * c.D, c.D)
    return lib.fa_cache_append(ctypes.addressof(Append(c, k, k, st, st, new, T)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=-1), fa.FA_ERR_INVALID_ARG), (dict(T=-2), fa.FA_ERR_INVALID_ARG), (dict(k=None), fa.FA_ERR_INVALID_ARG),
    (dict(kc=None), fa.FA_ERR_INVALID_ARG), (dict(lens=None), fa.FA_ERR_INVALID_ARG),
    (dict(table=None), fa.FA_ERR_INVALID_ARG), (dict(sc=_st(0, 1024, 64)), fa.FA_ERR_INVALID_ARG),
    (dict(D=40), fa.FA_ERR_UNSUPPORTED), (dict(page=20), fa.FA_ERR_UNSUPPORTED),
    (dict(T=1 << 28), fa.FA_ERR_UNSUPPORTED),
    (dict(kc=PTR + 2), fa.FA_ERR_ALIGNMENT), (dict(sk=_st(384, 192, 60)), fa.FA_ERR_ALIGNMENT),
    (dict(new=PTR + 3), fa.FA_ERR_ALIGNMENT), (dict(Z=0), fa.FA_OK), (dict(T=0), fa.FA_OK), (dict(H=0), fa.FA_OK),
])
def test_append_arguments(lib, kw, code):
    assert _append(lib, **kw) == code


def _commit(lib, *, path=PTR, kept=PTR, A=3, ps=3, L=2, **kw):
    return lib.fa_cache_commit(ctypes.addressof(Commit(_cache(L=L, **kw), path, ps, kept, A)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(L=-1), fa.FA_ERR_INVALID_ARG), (dict(A=-1), fa.FA_ERR_INVALID_ARG), (dict(ps=-3), fa.FA_ERR_INVALID_ARG),
    (dict(path=None), fa.FA_ERR_INVALID_ARG), (dict(kept=None), fa.FA_ERR_INVALID_ARG),
    (dict(kc=None), fa.FA_ERR_INVALID_ARG), (dict(D=8), fa.FA_ERR_UNSUPPORTED), (dict(page=17), fa.FA_ERR_UNSUPPORTED),
    (dict(kl=0), fa.FA_ERR_ALIGNMENT), (dict(kl=12), fa.FA_ERR_ALIGNMENT), (dict(path=PTR + 1), fa.FA_ERR_ALIGNMENT),
    (dict(Z=0), fa.FA_OK), (dict(L=0), fa.FA_OK), (dict(A=0), fa.FA_OK),
])
def test_commit_arguments(lib, kw, code):
    assert _commit(lib, **kw) == code


def _fork(lib, *, refs=PTR, src=PTR, miss=None, room=1, ws=PTR, wsb=1 << 40, L=2, **kw):
    return lib.fa_cache_fork(ctypes.addressof(Fork(_cache(L=L, **kw), refs, src, miss, ws, wsb, room)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(room=-1), fa.FA_ERR_INVALID_ARG), (dict(lens=None), fa.FA_ERR_INVALID_ARG),
    (dict(refs=None), fa.FA_ERR_INVALID_ARG), (dict(table=None), fa.FA_ERR_INVALID_ARG),
    (dict(ts=3), fa.FA_ERR_INVALID_ARG), (dict(sc=_st(0, 1024, 64)), fa.FA_ERR_INVALID_ARG),
    (dict(Z=8193), fa.FA_ERR_UNSUPPORTED), (dict(page=100), fa.FA_ERR_UNSUPPORTED), (dict(D=24), fa.FA_ERR_UNSUPPORTED),
    (dict(src=PTR + 2), fa.FA_ERR_ALIGNMENT), (dict(miss=PTR + 2), fa.FA_ERR_ALIGNMENT),
    (dict(kl=4), fa.FA_ERR_ALIGNMENT), (dict(ws=None), fa.FA_ERR_WORKSPACE), (dict(wsb=16), fa.FA_ERR_WORKSPACE),
    (dict(ws=PTR + 8), fa.FA_ERR_WORKSPACE), (dict(Z=0), fa.FA_OK),
    (dict(L=0, P=(1 << 30) + 1), fa.FA_ERR_UNSUPPORTED), (dict(room=(1 << 30) + 1), fa.FA_ERR_UNSUPPORTED),
])
def test_fork_arguments(lib, kw, code):
    assert _fork(lib, **kw) == code


def test_workspace_sizes(lib):
    assert fa.fa_cache_fork_workspace_size(0, 0) >= 0
    assert fa.fa_cache_fork_workspace_size(10, 100) >= 4 * 10 * 108
    n = ctypes.c_size_t()
    assert lib.fa_cache_fork_workspace_size(-1, 3, ctypes.byref(n)) == fa.FA_ERR_INVALID_ARG
    for call in (lib.fa_fwd_paged, lib.fa_cache_append, lib.fa_cache_commit, lib.fa_cache_fork):
        assert call(None, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_fwd_paged_workspace_size(20, ctypes.byref(n)) == fa.FA_ERR_UNSUPPORTED
    assert lib.fa_fwd_paged_workspace_size(64, None) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_status_string(fa.FA_ERR_PAGE) == "FA_ERR_PAGE"


# ------------------------------------------------------------- Python checks -

def _tensors(Z=2, Hq=4, Hkv=2, T=3, D=64, P=9, page=16, M=4, dt=torch.float16):
    return dict(q=torch.zeros(Z, Hq, T, D, dtype=dt), k_cache=torch.zeros(P, Hkv, page, D, dtype=dt),
                v_cache=torch.zeros(P, Hkv, page, D, dtype=dt), block_table=torch.zeros(Z, M, dtype=torch.int32),
                seq_lens=torch.zeros(Z, dtype=torch.int32))


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros(2, 4, 64, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(2, 4, 3, 32, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(2, 4, 3, 64)), TypeError),
    (dict(q=torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16)), TypeError),
    (dict(v_cache=torch.zeros(8, 2, 16, 64, dtype=torch.float16)), ValueError),
    (dict(block_table=torch.zeros(3, 4, dtype=torch.int32)), ValueError),
    (dict(block_table=torch.zeros(2, 4, dtype=torch.int64)), TypeError),
    (dict(block_table=torch.zeros(4, 2, dtype=torch.int32).t()), ValueError),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(new_lens=torch.zeros(1, dtype=torch.int32)), ValueError),
    (dict(tree_mask=torch.zeros(2, 3, 2, dtype=torch.int32)), ValueError),
    (dict(tree_mask=torch.zeros(2, 3, 1, dtype=torch.uint8)), TypeError),
    (dict(o=torch.zeros(2, 4, 3, 64)), ValueError),
    (dict(lse=torch.zeros(2, 4, 3, dtype=torch.float16)), ValueError),
    (dict(), ValueError),  # tensors of the CPU
])
def test_python_attention_checks(change, error):
    with pytest.raises(error):
        fa.fa_fwd_paged(**{**_tensors(), **change})


def test_python_cache_checks():
    t = _tensors()
    kc, vc, tb, ln = t["k_cache"], t["v_cache"], t["block_table"], t["seq_lens"]
    rows = torch.zeros(2, 2, 3, 64, dtype=torch.float16)
    i32 = dict(dtype=torch.int32)
    for bad, error in [(lambda: fa.fa_cache_append(rows[:, :1], rows[:, :1], kc, vc, tb, ln), ValueError),
                       (lambda: fa.fa_cache_append(rows.bfloat16(), rows.bfloat16(), kc, vc, tb, ln), TypeError),
                       (lambda: fa.fa_cache_append(rows, rows, kc[None], vc[None], tb, ln), ValueError),
                       (lambda: fa.fa_cache_append(rows, rows, kc, vc, tb, ln[:1]), ValueError),
                       (lambda: fa.fa_cache_commit(kc, vc, tb, ln, torch.zeros(2, 3, **i32), torch.zeros(1, **i32)), ValueError),
                       (lambda: fa.fa_cache_commit(kc, vc, tb, ln, torch.zeros(2, 3), torch.zeros(2, **i32)), TypeError),
                       (lambda: fa.fa_cache_commit(kc.float(), vc.float(), tb, ln, torch.zeros(2, 3, **i32), torch.zeros(2, **i32)), TypeError),
                       (lambda: fa.fa_cache_fork(kc, vc, tb, ln, torch.zeros(8, **i32)), ValueError),
                       (lambda: fa.fa_cache_fork(kc, vc, tb, ln, torch.zeros(9, **i32), torch.zeros(3, **i32)), ValueError),
                       (lambda: fa.fa_cache_fork(kc, vc, tb, ln, torch.zeros(9, **i32), missing=torch.zeros(2, **i32)), ValueError),
                       (lambda: fa.fa_cache_fork(kc, vc, tb, ln, torch.zeros(9, **i32)), ValueError)]:
        with pytest.raises(error):
            bad()


def test_python_workspace_must_be_contiguous():
    t, ws = _tensors(), torch.zeros(1, dtype=torch.uint8).expand(1 << 30)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        fa.fa_fwd_paged(**t, workspace=ws)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        fa.fa_cache_fork(t["k_cache"], t["v_cache"], t["block_table"], t["seq_lens"], torch.zeros(9, dtype=torch.int32),
                         workspace=ws)


def test_binding_is_built_for_torch_with_cuda_only(tmp_path, monkeypatch):
    from types import SimpleNamespace

    b = importlib.import_module("exact_attention_44_gb300.build")
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    assert b._torch_dir() is None
    spec = SimpleNamespace(submodule_search_locations=[str(tmp_path)])
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: spec)
    assert b._torch_dir() is None
    (tmp_path / "lib").mkdir()
    (tmp_path / "lib" / "libc10_cuda.so").touch()
    assert b._torch_dir() == str(tmp_path)


# ------------------------------------------------------------- the plain statements

def test_fork_statement_keeps_the_counts():
    r = np.random.RandomState(3)
    page, P, Z, M = 16, 60, 7, 9
    table, lens, refs = [[-1] * M for _ in range(Z)], [0] * Z, [0] * P
    for step in range(200):
        source = [int(r.choice([z, z, r.randint(Z), -1])) for z in range(Z)] if step % 2 else None
        room = int(r.randint(0, 40))
        table, lens, refs, missing, tails = pu.fork(table, lens, refs, source, room, page)
        counted = np.bincount([p for row in table for p in row if p >= 0], minlength=P)
        assert counted.tolist() == refs
        for z in range(Z):
            have = sum(p >= 0 for p in table[z])
            assert missing or have * page >= lens[z] + (room if source is None or source[z] >= 0 else 0)
            lens[z] = max(min(have * page, lens[z] + int(r.randint(0, room + 1))) if lens[z] or have else 0,
                          min(lens[z], have * page))


def test_attention_statement_against_softmax():
    r = np.random.RandomState(0)
    q, k, v = r.randn(1, 2, 2, 8), [r.randn(1, 7, 8)], [r.randn(1, 7, 8)]
    o, lse = pu.attention(q, k, v, [5], [2], None, 0.3)
    s = torch.from_numpy(0.3 * q[0, 1, 0] @ k[0][0][:6].T)
    assert np.allclose(o[0, 1, 0], torch.softmax(s, -1).numpy() @ v[0][0][:6])
    assert np.isclose(lse[0, 1, 0], torch.logsumexp(s, -1).item())
