import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Tests that hold a value the definition does not give; they stay as they are, and must go on failing.
WRONG_VALUES = {
    "test_layer_equals_its_parts_on_host_splits":
        "its layer has an FC2 bias and its reference adds that bias without the router's weight, sum_j (w_j W2 a_j + "
        "b2): the definition is sum_j w_j (W2 a_j + b2) (tests/test_gpu_moe_layer.py, against 64 bits)",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG_VALUES.get(getattr(item, "originalname", None))
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))
