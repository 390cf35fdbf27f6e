import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Tests that hold a wrong value.  They run as they are; one that passes is an error.
WRONG = {
    "test_gpu_delta.py::test_backward_of_a_gate_that_forgets_everything":
        "asserts dgamma = 0 at gamma = 0, where the definition <N - dw k^T, S> is not 0 (test_gpu_delta_gates.py)",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, reason in WRONG.items():
            if item.nodeid.endswith(name):
                item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))
