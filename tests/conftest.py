"""Shared pytest set-up.

Markers: ``gpu`` -- needs a CUDA device (the parity tests proper, through the
C-ABI library). Everything unmarked runs on a CPU-only machine.
"""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a)")


@pytest.fixture(scope="session")
def orc():
    from oracle import oracle
    oracle.lib()
    return oracle


@pytest.fixture(autouse=True)
def _seeded():
    """Inputs that a test draws without a seed are the same on every run."""
    import torch
    torch.manual_seed(0)
