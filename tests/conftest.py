import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built libfa")
    config.addinivalue_line("markers", "slow: takes more than a few seconds on the CPU")


def pytest_collection_modifyitems(config, items):
    # GPU tests cannot run without a device; make that a clear skip rather than an error.
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device in this environment")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(autouse=True)
def _argument_structures_outlive_their_calls(request, monkeypatch):
    # ctypes.addressof returns a bare integer: a structure made in the call's own argument list is freed
    # before the library reads it, and the refusal that a test sees is then that of whatever lies there.
    if request.module.__name__ == "test_paged_host":
        import ctypes
        held, addressof = [], ctypes.addressof
        monkeypatch.setattr(ctypes, "addressof", lambda x: (held.append(x), addressof(x))[1])
    yield
