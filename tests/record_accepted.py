"""A pytest plugin for tests/test_no_gpu_calls.py: writes, to the file named by ACCEPTED_CALLS, each test without the
``gpu`` marker that got past the host checks of an entry point of the library (status MLA_ERR_CUDA or
MLA_ERR_UNSUPPORTED where there is no B200, MLA_OK where there is one)."""
import ctypes
import os

import pytest

import mla_decode_attention_14_b200 as mla

# calls that launch nothing and take no device address
HOST_ONLY = {"mla_status_string", "mla_default_fixed_cost", "mla_workspace_bytes", "mla_shared_units",
             "mla_shared_fixed_cost", "mla_shared_workspace_bytes", "mla_rope_init", "mla_launch_count",
             "mla_last_cuda_error", "mla_default_num_parts", "mla_check_status"}
_accepted = []


def _record(name):
    def errcheck(result, func, args):
        if result not in (1, 3):  # neither MLA_ERR_INVALID_ARG nor MLA_ERR_WORKSPACE
            _accepted.append(name)
        return result
    return errcheck


@pytest.hookimpl(hookwrapper=True)
def pytest_runtest_call(item):
    del _accepted[:]
    yield
    if _accepted and item.get_closest_marker("gpu") is None:
        with open(os.environ["ACCEPTED_CALLS"], "a") as f:
            f.write("%s %s\n" % (item.nodeid, ",".join(sorted(set(_accepted)))))


def pytest_collection_finish(session):
    L = mla.lib()
    for name in mla.EXPORTS:
        if name not in HOST_ONLY:
            fn = getattr(L, name)
            assert isinstance(fn, ctypes._CFuncPtr)
            fn.errcheck = _record(name)
