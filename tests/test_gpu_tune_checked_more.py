"""More of the fine-tuning operators in the checked build (-DLP_CHECKED) on a GB300: the check word stays 0 and every
output has the normal build's bits."""

import os
import subprocess
import sys

import pytest
import torch

from invariant_token_logprobs_gb300 import _build_lib, tune
from _tune_checked_more import run_cases

pytestmark = pytest.mark.gpu


def test_checked_build_clean_and_bitwise_equal(tmp_path):
    ref = run_cases(tune)
    path = str(tmp_path / "checked.pt")
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_tune_checked_more.py")
    env = dict(os.environ, LP_LIBRARY=_build_lib.build(checked=True))
    res = subprocess.run([sys.executable, child, path], capture_output=True, text=True, env=env, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    got = torch.load(path)
    assert got["backend"].endswith("+checked") and got["word"] == 0, f"check word {got['word']:#x}"
    assert set(got["out"]) == set(ref)
    for k in ref:
        assert torch.equal(got["out"][k], ref[k]), k
