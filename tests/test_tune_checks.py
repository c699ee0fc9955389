"""The checked build's promise for the fine-tuning operators: every kernel tests the indexes of its accesses."""

import os

import pytest

from invariant_token_logprobs_gb300 import _build_lib
from test_train_checks import KERNEL, bodies


@pytest.mark.parametrize("source,kernels", [("lp_layer_norm.cu", 2), ("lp_layer_norm_backward.cu", 2),
                                            ("lp_preference.cu", 4), ("lp_muon.cu", 3)])
def test_every_kernel_tests_its_indexes(source, kernels):
    with open(os.path.join(_build_lib.CSRC, source)) as f:
        found = dict(bodies(f.read(), KERNEL))
    assert len(found) == kernels
    for name, body in found.items():
        assert "LP_CHECK(" in body, f"{source}: {name}"


def test_parameters_and_tiles_test_theirs():
    """The accesses that Muon's product kernel makes through its parts."""
    with open(os.path.join(_build_lib.CSRC, "lp_muon.cu")) as f:
        found = dict(bodies(f.read(), r"__device__ __forceinline__ void (write_params|write_split)\("))
    assert set(found) == {"write_params", "write_split"}
    assert all("LP_CHECK(" in body for body in found.values())
