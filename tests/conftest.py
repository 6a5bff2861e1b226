import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


# Tests that hand complete lists of arguments with made-up addresses to the library: without a GPU
# such a call ends at the device's check; with one its kernels would read and write there.
MADE_UP_ADDRESSES = {("test_dense_abi", "test_refusals"), ("test_dense_abi", "test_what_may_be_left_out"),
                     ("test_experts_args", "test_a_join_without_rows_needs_no_rows"),
                     ("test_experts_args", "test_counts_beside_the_end_of_32_bits")}


def gpu_is_here():
    """Whether the library would find a device (any that the driver shows)."""
    import torch
    return torch.cuda.device_count() > 0


def pytest_runtest_setup(item):
    name = getattr(item, "originalname", item.name)
    if (item.module.__name__, name) in MADE_UP_ADDRESSES and gpu_is_here():
        pytest.skip("made-up addresses: for machines without a GPU")


def read_golden(name):
    """Rows of a golden fixture, comments and blank lines removed."""
    rows = []
    with open(os.path.join(GOLDEN, name)) as f:
        for line in f:
            line = line.strip()
            if not line or line.startswith("#"):
                continue
            rows.append(line.split())
    return rows


@pytest.fixture(scope="session")
def oracle_mod():
    import oracle
    oracle.build()
    return oracle
