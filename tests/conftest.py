import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long CPU test")


@pytest.fixture(autouse=True)
def seeded():
    """What a test draws from torch's own generator is the same whatever ran before it."""
    import torch

    torch.manual_seed(0)


@pytest.fixture(scope="session")
def ctwin():
    from oracle.ctwin import LIB, build_ctwin, load_ctwin

    if not os.path.exists(LIB):
        build_ctwin()
    return load_ctwin()
