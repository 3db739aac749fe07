import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built CUDA library")
    config.addinivalue_line("markers", "slow: long-running GPU parity case at full benchmark size")


# Host tests with a call that is sound but for its addresses, which only the want of a device keeps from a launch.
NEEDS_NO_GPU = ("test_rope_calls_are_refused",)


def pytest_collection_modifyitems(items):
    import torch
    if torch.cuda.is_available():
        for item in items:
            if item.name in NEEDS_NO_GPU:
                item.add_marker(pytest.mark.skip(reason="made-up addresses: only where no GPU would read them"))


@pytest.fixture(scope="session")
def golden():
    import json
    with open(os.path.join(ROOT, "tests", "golden", "worked_examples.json")) as f:
        return json.load(f)
