import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


# Tests whose calls pass every check of the arguments, with addresses that are no
# memory: only the missing device stops them.  Where there is one they would launch.
ONLY_WITHOUT_A_DEVICE = {"test_head_cpu.py": {"test_sizes", "test_pointers", "test_without_a_device"}}


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


def pytest_collection_modifyitems(config, items):
    # GPU tests need a device; on a CPU-only host they are skipped, not failed.
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        skip = pytest.mark.skip(reason="launches on invented addresses where there is a GPU")
        for it in items:
            if getattr(it, "originalname", None) in ONLY_WITHOUT_A_DEVICE.get(os.path.basename(it.path), ()):
                it.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no GPU on this host")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
