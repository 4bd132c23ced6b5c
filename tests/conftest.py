"""Shared pytest configuration: the ``gpu`` marker, the repository root on sys.path, and the tests that must not
meet a GPU."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# Tests that call an entry point with arguments it accepts and made-up addresses, to see that every check on the host
# lets them through: without a B200 the call ends there (MLA_ERR_CUDA or MLA_ERR_UNSUPPORTED), with one it would launch
# a kernel on those addresses. They run only where no GPU is visible (tests/test_no_gpu_calls.py keeps the list whole).
NO_GPU_ONLY = {
    ("test_serving_cpu.py", "test_shared_decode_refuses_a_small_workspace"),
    ("test_serving_cpu.py", "test_rope_q_refuses"),
    ("test_serving_cpu.py", "test_append_refuses"),
}


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU; runs the CUDA path")


def no_gpu_only(item) -> bool:
    return (os.path.basename(str(item.path)), getattr(item, "originalname", None) or item.name) in NO_GPU_ONLY


def pytest_runtest_setup(item):
    if no_gpu_only(item):
        import torch
        if torch.cuda.is_available():
            pytest.skip("calls entry points with made-up addresses: only where there is no GPU")
