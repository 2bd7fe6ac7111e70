import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a GB300 (runs through the C-ABI library)")
    config.addinivalue_line("markers", "slow: full-size case (minutes)")


# Their calls have made-up pointers, and some pass the checks: where there is a GPU, kernels would run
# on those.
MADE_UP_POINTERS = ("test_operators_refusals.py", "test_serving_refusals.py")


def pytest_collection_modifyitems(items):
    made_up = [i for i in items if i.path.name in MADE_UP_POINTERS]
    if not made_up:
        return
    import torch
    if torch.cuda.is_available():
        for i in made_up:
            i.add_marker(pytest.mark.skip(reason="made-up pointers: only where no launch can follow"))
