"""libfa.so does not depend on its optional Python binding: a binding that cannot be compiled leaves the
library built and is not left behind stale, and a new torch or interpreter rebuilds the binding only."""
import importlib
import os

import pytest

import exact_attention_44_gb300 as fa


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build of a library of one small unit, with a binding that compiles without torch."""
    b = importlib.import_module("exact_attention_44_gb300.build")
    csrc, torch = tmp_path / "csrc", tmp_path / "torch"
    (torch / "lib").mkdir(parents=True)
    csrc.mkdir()
    (csrc / "a.cu").write_text('extern "C" int fa_answer() { return 42; }\n')
    (csrc / "paged_ext.cpp").write_text("int answer() { return 42; }\n")
    (torch / "version.py").write_text("one")
    monkeypatch.setattr(b, "CSRC", str(csrc))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "build" / "libfa.so"))
    monkeypatch.setattr(b, "EXT", str(tmp_path / "build" / "_paged_ext.so"))
    monkeypatch.setattr(b, "UNITS", [("a.cu", "a.o", [])])
    monkeypatch.setattr(b, "_torch_dir", lambda: str(torch))
    monkeypatch.setattr(b, "_ext_command", lambda torch, cc, out: ["g++", "-shared", "-fPIC", str(csrc / "paged_ext.cpp"),
                                                                   "-o", out])
    return b, csrc, torch


def test_library_is_built_without_its_binding(small, capfd):
    b, csrc, _ = small
    (csrc / "paged_ext.cpp").write_text("#error no headers\n")
    lib = b.build()
    assert os.path.exists(lib) and not os.path.exists(b.EXT)
    err = capfd.readouterr().err
    assert "no headers" in err and "g++ failed on paged_ext.cpp" in err and "nvcc failed" not in err
    first = os.stat(lib).st_mtime_ns
    (csrc / "paged_ext.cpp").write_text("int answer() { return 1; }\n")
    assert b.build() == lib and os.path.exists(b.EXT)  # tried again, and the library left alone
    assert os.stat(lib).st_mtime_ns == first


def test_stale_binding_does_not_stay(small):
    b, csrc, _ = small
    b.build()
    assert os.path.exists(b.EXT)
    (csrc / "paged_ext.cpp").write_text("#error broken\n")
    b.build()
    assert not os.path.exists(b.EXT)


def test_new_torch_rebuilds_the_binding_only(small):
    b, csrc, torch = small
    lib = b.build()
    at = {p: os.stat(p).st_mtime_ns for p in (lib, b.EXT)}
    with pytest.MonkeyPatch.context() as m:
        m.setattr(b, "nvcc", lambda: pytest.fail("nothing is to be compiled"))
        b.build()
    assert all(os.stat(p).st_mtime_ns == t for p, t in at.items())
    (torch / "version.py").write_text("two")
    b.build()
    assert os.stat(lib).st_mtime_ns == at[lib] and os.stat(b.EXT).st_mtime_ns > at[b.EXT]


def test_failing_library_still_raises(small):
    b, csrc, _ = small
    (csrc / "a.cu").write_text("#error broken\n")
    with pytest.raises(RuntimeError, match="libfa build failed"):
        b.build()
    assert not os.path.exists(b.LIB)


def test_missing_binding_is_named_by_the_calls(monkeypatch, tmp_path):
    import torch
    paged = importlib.import_module("exact_attention_44_gb300.paged")
    fa.build()
    monkeypatch.setattr(paged, "_EXT", str(tmp_path / "_paged_ext.so"))
    monkeypatch.setattr(paged, "_ext", None)
    monkeypatch.setattr(paged, "_bound", None)
    x = torch.zeros(1)
    for call, args in ((paged.fa_fwd_paged, 5), (paged.fa_cache_append, 6), (paged.fa_cache_commit, 6), (paged.fa_cache_fork, 5)):
        with pytest.raises(ImportError, match="paged-cache binding is not built"):
            call(*[x] * args)
