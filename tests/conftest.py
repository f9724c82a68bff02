import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


def pytest_collection_modifyitems(config, items):
    if _has_gpu():
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(autouse=True)
def _former_tests_graphs_are_gone(request):
    """A CUDA graph that a former test left in a reference cycle (a caught exception's frame holds it) is destroyed when
    the collector happens to run.  Within a later test's capture that ends the capture, so it runs before."""
    if "gpu" in request.keywords:
        gc.collect()


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.lib()
    return oracle
