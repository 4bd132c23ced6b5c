"""No test without the ``gpu`` marker may reach a launch with made-up addresses where there is a GPU: on a CPU-only
machine such a call shows by its status, so it is found there."""
import os
import subprocess
import sys

import pytest
import torch

from mla_decode_attention_14_b200 import build as mla_build
from tests import conftest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_tests_whose_calls_are_accepted_stay_off_gpus(tmp_path):
    """Every CPU test file that calls the library, run without a visible GPU: the tests whose calls pass the host
    checks are those that conftest keeps off GPUs."""
    mla_build.build()
    files = [f for f in sorted(os.listdir(HERE)) if f.startswith("test_") and f != os.path.basename(__file__)
             and not f.endswith("_gpu.py") and "mla_decode_attention_14_b200 as mla" in open(os.path.join(HERE, f)).read()]
    assert {"test_abi.py", "test_serving_cpu.py"} <= set(files)
    log = tmp_path / "accepted"
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", ACCEPTED_CALLS=str(log))
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-p", "tests.record_accepted", "-m",
                          "not gpu"] + [os.path.join(HERE, f) for f in files], cwd=conftest.ROOT, env=env,
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-2000:]
    found = {(os.path.basename(line.split("::")[0]), line.split("::")[1].split(" ")[0].split("[")[0])
             for line in log.read_text().splitlines()}
    assert found == conftest.NO_GPU_ONLY


def test_they_are_skipped_where_there_is_a_gpu(monkeypatch):
    class Item:
        name = originalname = "test_rope_q_refuses"
        path = os.path.join(HERE, "test_serving_cpu.py")
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    with pytest.raises(pytest.skip.Exception):
        conftest.pytest_runtest_setup(Item)
    Item.name = Item.originalname = "test_shared_units_and_workspace"
    conftest.pytest_runtest_setup(Item)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    Item.name = Item.originalname = "test_rope_q_refuses"
    conftest.pytest_runtest_setup(Item)
