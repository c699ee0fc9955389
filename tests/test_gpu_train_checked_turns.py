"""The checked build (-DLP_CHECKED) over several turns of a CTA on a GB300: the check word stays 0
and every output has the normal build's bits."""

import os
import subprocess
import sys

import pytest
import torch

from invariant_token_logprobs_gb300 import _build_lib, train
import _train_turn_cases as cases

pytestmark = pytest.mark.gpu


def test_checked_build_clean_and_bitwise_equal(tmp_path):
    ref = cases.run_cases(train)
    path = str(tmp_path / "checked.pt")
    env = dict(os.environ, LP_LIBRARY=_build_lib.build(checked=True))
    res = subprocess.run([sys.executable, cases.__file__, path], capture_output=True, text=True, env=env,
                         timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    got = torch.load(path, map_location=cases.DEV)
    assert got["backend"].endswith("+checked") and got["word"] == 0, f"check word {got['word']:#x}"
    assert set(got["out"]) == set(ref)
    for k in ref:
        # a kept element may be NaN in both
        assert torch.equal(got["out"][k].nan_to_num(7), ref[k].nan_to_num(7)), k
