import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
HERE = os.path.dirname(os.path.abspath(__file__))
if HERE not in sys.path:
    sys.path.insert(0, HERE)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


@pytest.fixture(autouse=True)
def own_memory(request):
    """A GPU test begins with nothing in torch's cache.  A segment that an earlier test left there
    would be cut up for this one's tensors: it then stays, whole, for as long as they live, and a
    test that limits the process to what is reserved has all of its rest to allocate from."""
    if request.node.get_closest_marker("gpu") is not None:
        import torch
        if torch.cuda.is_available():
            if torch.cuda.memory_allocated() > 0:
                gc.collect(1)  # tensors in reference cycles (of the latest tests: quick)
            torch.cuda.empty_cache()
    yield
