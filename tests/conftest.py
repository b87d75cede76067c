import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built libspc.so")


def pytest_collection_modifyitems(config, items):
    # GPU tests are skipped, not failed, where no GPU is present; the CPU suite
    # is selected with -m "not gpu".
    try:
        import torch

        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)


@pytest.fixture(scope="module", autouse=True)
def _collected():
    """What earlier tests left in reference cycles (an exception holds its frames' tensors) is freed
    before a module begins, not while one of its tests counts memory."""
    gc.collect()
    yield
