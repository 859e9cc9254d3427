import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: CPU test that takes more than a few seconds")


@pytest.fixture(scope="session")
def oracle():
    import oracle as _oracle
    return _oracle.default()


# Tests that hold a wrong value, and why.
WRONG = {
    "test_w4_router_refusals.py::test_balance_loss_records_its_gradient":
        "asserts that the backward pass reads the counts that the caller got: written into by a collective "
        "they give a wrong gradient (test_balance_recorded.py has its other assertions and the right one)",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, reason in WRONG.items():
            if item.nodeid.endswith(name):
                item.add_marker(pytest.mark.xfail(reason=reason, strict=True))
