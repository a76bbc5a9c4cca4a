"""Build libfa.so in-tree with nvcc for sm_103a (one -gencode, parallel TUs).

    python -m exact_attention_44_gb300.build [--force] [--verbose] [--debug-checks]

Objects and the shared library go to exact_attention_44_gb300/_build/ (git
ignored).  A content hash of the sources, headers and flags is stored next to
the library; an unchanged tree is not rebuilt.  --debug-checks builds a
second library, _build/checks/libfa.so, whose forward kernels check every
unit they decode against the launch's sizes (FA_DEBUG_CHECKS=1).  Where torch
with CUDA is installed, the binding of the paged-cache and rotary calls (_paged_ext.so,
a CPython extension over torch's headers) is built beside libfa.so with g++, under a
hash of its own.  The library does not need it: if it cannot be compiled, the
compiler's output is printed, the library is built all the same, and those calls of the
package raise ImportError.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libfa.so")
EXT = os.path.join(BUILD, "_paged_ext.so")

# (source, object, extra flags): the per-head-dim launchers are one source
# each, compiled once per supported head dim
FWD_DIMS = (16, 32, 64, 128, 256)
BWD_DIMS = (16, 32, 64, 128, 256)
UNITS = ([(src, src.replace(".cu", ".o"), []) for src in ("fa_api.cu", "fa_lse_merge.cu", "fa_noalloc.cu",
                                                           "fa_paged_api.cu", "fa_cache.cu", "fa_budget_api.cu",
                                                           "fa_rope.cu", "fa_evict.cu")] +
         [("fa_fwd_dim.cu", f"fa_fwd_d{d}.o", [f"-DFA_HEAD_DIM={d}"]) for d in FWD_DIMS] +
         [("fa_bwd_dim.cu", f"fa_bwd_d{d}.o", [f"-DFA_HEAD_DIM={d}"]) for d in BWD_DIMS] +
         [("fa_paged_dim.cu", f"fa_paged_d{d}.o", [f"-DFA_HEAD_DIM={d}"]) for d in FWD_DIMS] +
         [("fa_score_dim.cu", f"fa_score_d{d}.o", [f"-DFA_HEAD_DIM={d}"]) for d in FWD_DIMS])
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libfa needs the CUDA 13 toolkit to build")


def _hash(files: list[str], flags: list[str]) -> str:
    h = hashlib.sha256()
    for path in files:
        with open(path, "rb") as f:
            h.update(os.path.basename(path).encode() + b"\0" + f.read())
    h.update(" ".join(flags).encode())
    return h.hexdigest()


def _sources(folder: str, *endings: str) -> list[str]:
    return [os.path.join(folder, name) for name in sorted(os.listdir(folder)) if name.endswith(endings)]


def _tree_hash(extra_flags: list[str]) -> str:
    """Of what libfa.so is made of."""
    return _hash(_sources(CSRC, ".cu", ".cuh", ".h") + _sources(INCLUDE, ".h"), FLAGS + extra_flags)


def _ext_hash(torch: str) -> str:
    """Of what the binding is made of and tied to."""
    return _hash([os.path.join(CSRC, "paged_ext.cpp")] + _sources(INCLUDE, ".h"),
                 [*_ext_command(torch, "nvcc", EXT), _ext_stamp(torch)])


def _fresh(product: str, digest: str) -> bool:
    """Whether the product is there, and was made from what has this hash."""
    stamp = product + ".hash"
    if not (os.path.exists(product) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        return f.read() == digest


def _install(tmp: str, product: str, digest: str) -> None:
    os.replace(tmp, product)
    with open(product + ".hash", "w") as f:
        f.write(digest)


def _torch_dir() -> str | None:
    """Where torch with CUDA is installed (it is not imported), or None."""
    spec = importlib.util.find_spec("torch")
    for d in spec.submodule_search_locations or [] if spec is not None else []:
        if os.path.exists(os.path.join(d, "lib", "libc10_cuda.so")):
            return d
    return None


def _ext_stamp(torch: str) -> str:
    """What the binding is tied to: this interpreter, and the torch whose headers it was built over."""
    with open(os.path.join(torch, "version.py")) as f:
        return sys.version + "\n" + torch + "\n" + f.read()


def _ext_command(torch: str, cc: str, out: str) -> list[str]:
    """The command that builds the paged-cache binding."""
    inc = os.path.join(torch, "include")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", os.path.join(CSRC, "paged_ext.cpp"), "-o", out,
            f"-I{INCLUDE}", f"-I{sysconfig.get_paths()['include']}", f"-isystem{inc}",
            f"-isystem{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
            f"-I{os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), 'include')}",
            f"-L{os.path.join(torch, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
          debug_checks: bool = False) -> str:
    """Compile every translation unit (in parallel) and link libfa.so; returns its path.

    debug_checks: build the index-checking variant into _build/checks/ instead."""
    extra_flags = list(extra_flags or [])
    build_dir, lib_path = BUILD, LIB
    if debug_checks:
        extra_flags.append("-DFA_DEBUG_CHECKS=1")
        build_dir = os.path.join(BUILD, "checks")
        lib_path = os.path.join(build_dir, "libfa.so")
    os.makedirs(build_dir, exist_ok=True)
    digest = _tree_hash(extra_flags)
    need_lib = force or not _fresh(lib_path, digest)
    torch = None if debug_checks else _torch_dir()
    ext_digest = "" if torch is None else _ext_hash(torch)
    need_ext = torch is not None and (force or not _fresh(EXT, ext_digest))
    if not need_lib and not need_ext:
        return lib_path
    cc = nvcc()
    jobs = []  # (compiler, source, output, command)
    for src, obj_name, unit_flags in UNITS if need_lib else []:
        obj = os.path.join(build_dir, obj_name)
        cmd = [cc, *FLAGS, *unit_flags, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append(("nvcc", src, obj, cmd))
    objects = [obj for _, _, obj, _ in jobs]
    ext_tmp = EXT + f".tmp{os.getpid()}"
    if need_ext:
        jobs.append(("g++", "paged_ext.cpp", ext_tmp, _ext_command(torch, cc, ext_tmp)))

    def run(job):
        try:
            r = subprocess.run(job[3], capture_output=True, text=True)
            return r.returncode == 0, r.stdout + r.stderr
        except OSError as e:  # no such compiler
            return False, f"{e}\n"

    with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
        results = list(ex.map(run, jobs))
    failed = set()
    for (compiler, src, out, _), (ok, text) in zip(jobs, results):
        if not ok:
            failed.add(out)
            sys.stderr.write(f"--- {compiler} failed on {src}\n{text}\n")
        elif verbose and text:
            sys.stderr.write(f"--- {os.path.basename(out)}\n{text}\n")
    if ext_tmp in failed:
        sys.stderr.write("the paged-cache binding was not built: fa_fwd_paged and the fa_cache_* calls will raise ImportError\n")
        if os.path.exists(EXT):  # of other sources, or of another torch
            os.remove(EXT)
    elif need_ext:
        _install(ext_tmp, EXT, ext_digest)
    if failed.intersection(objects):
        raise RuntimeError("libfa build failed")
    if need_lib:
        tmp = lib_path + f".tmp{os.getpid()}"
        r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objects], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"libfa link failed:\n{r.stdout}{r.stderr}")
        _install(tmp, lib_path, digest)
    return lib_path


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/spill/smem usage")
    ap.add_argument("--debug-checks", action="store_true",
                    help="build the variant whose kernels check every unit against the launch's sizes")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose, debug_checks=a.debug_checks))


if __name__ == "__main__":
    main()
