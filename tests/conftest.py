import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


def pytest_collection_modifyitems(items):
    """The decode operators' GPU tests last. They use second streams and captured graphs, and work on
    another queue moves the XCD that the default queue's workgroup 0 goes to by one or two for the
    rest of the process (measured; any kernel does it). test_gpu_robustness pins the dispatch of a
    process that has used one queue."""
    items.sort(key=lambda i: i.path.name.startswith("test_gpu_decode_"))


def gpu_available() -> bool:
    try:
        import torch
    except Exception:
        return False
    return torch.cuda.is_available()


@pytest.fixture(scope="session")
def oracle_mod():
    from oracle import oracle

    oracle.lib()
    return oracle
