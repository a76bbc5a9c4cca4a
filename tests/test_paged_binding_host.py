"""The paged-cache extension called before it is bound to a library raises; it does not end the process."""
import os
import subprocess
import sys

import pytest

import exact_attention_44_gb300 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("call,count", [("fwd_paged", 13), ("cache_append", 8), ("cache_commit", 7), ("cache_fork", 11)])
def test_unbound_extension_raises(call, count):
    fa.build()
    code = f"""
import importlib.util, torch
from exact_attention_44_gb300.build import EXT
spec = importlib.util.spec_from_file_location("_paged_ext", EXT)
ext = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ext)
try:
    ext.{call}(*[None] * {count})
except ImportError as e:
    assert "libfa is not loaded" in str(e)
    print("raised")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "raised", (r.returncode, r.stderr[-300:])
