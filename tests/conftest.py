import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a) and the built libplsh.so")
    config.addinivalue_line("markers", "slow: takes more than a few seconds on the CPU")


def pytest_collection_modifyitems(config, items):
    # GPU tests run only where a device exists; on a CPU-only host they are
    # deselected by -m "not gpu" and skipped otherwise.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device on this host")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)


def pytest_runtest_setup(item):
    # test_zz_no_alloc compares allocated bytes before and after calls: tensors that earlier tests left in reference cycles (a caught
    # exception's frames) go first, or a garbage collection between the two counts frees them
    if item.path.name == "test_zz_no_alloc.py":
        gc.collect()
