import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200)")
    config.addinivalue_line("markers", "slow: long-running parity case")


@pytest.fixture(autouse=True)
def _same_numbers_every_run(request):
    """Seeds torch's generators, which are seeded by chance in every process: rows that a
    test draws without a generator of its own may have equal logits at the top in one run
    of twenty, whose order is another one than of different logits."""
    if request.node.get_closest_marker("gpu"):
        import torch
        torch.manual_seed(0)


def load_golden(name):
    """Parses a tests/golden/*.txt fixture into a dict of whitespace-split
    value lists (comments start with '#')."""
    out = {}
    with open(os.path.join(ROOT, "tests", "golden", name)) as f:
        for line in f:
            line = line.strip()
            if not line or line.startswith("#"):
                continue
            key, _, val = line.partition(":")
            out[key.strip()] = val.split()
    return out


@pytest.fixture(scope="session")
def golden():
    return load_golden
