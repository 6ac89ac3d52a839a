import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle._load()
    return oracle


# Tests that stay as they are though a value that they ask for is wrong. They run, and have to fail, at that value.
WRONG_VALUES = {
    "test_gpu_expert_layer_f8.py::test_gradients_against_64_bits":
        "asks for the router's gradient at the tokens' 8-bit values, but the layer's logits are formed from the tokens "
        "themselves: 2.9e-2 of the norm off by differences in 64 bits. test_gpu_expert_layer_f8_forms.py asks for all of "
        "its values, this one from the loss",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, reason in WRONG_VALUES.items():
            if item.nodeid.split("/")[-1].split("[")[0] == name:
                item.add_marker(pytest.mark.xfail(strict=True, raises=AssertionError, reason=reason))
