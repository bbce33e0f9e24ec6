"""pytest configuration: the `gpu` marker and import paths.

Tests marked `gpu` need an MI355X (gfx950) and the built GPU library; everything
else runs on a CPU-only host. Run the CPU suite with `pytest -m "not gpu"`.
"""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
TESTS = os.path.dirname(os.path.abspath(__file__))
if TESTS not in sys.path:
    sys.path.insert(0, TESTS)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X GPU and the built HIP library")


# Tests whose expected values are wrong; they run, and have to fail.
WRONG = {
    # 12 experts in 12 groups, a group's value the sum of its two best: their reference gives a group of one
    # expert -inf, so that all groups are equal and experts 0 to 3 are chosen whatever the logits are. The sum
    # over the one that there is is its value (test_groups_of_one_expert)
    f"test_experts_gpu.py::test_route[11-{biased}-{dtype}]": "a group of one expert has that expert's value, not -inf"
    for biased in (False, True) for dtype in ("bf16", "f16", "f32")
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG.get(item.nodeid.rsplit("/", 1)[-1])
        if reason:
            item.add_marker(pytest.mark.xfail(strict=True, raises=AssertionError, reason=reason))
