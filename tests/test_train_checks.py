"""The checked build's promise: every kernel tests the indexes of its accesses."""

import os
import re

import pytest

from invariant_token_logprobs_gb300 import _build_lib


def bodies(text, pattern):
    """(name, body) of every function that `pattern` finds the head of, its braces matched."""
    for m in re.finditer(pattern, text):
        at = text.index("{", m.end())
        depth, i = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[at:i]


KERNEL = r"__global__[^;{]*?\b(lp_\w+)\s*\("


@pytest.mark.parametrize("source", ["lp_norm.cu", "lp_norm_backward.cu", "lp_policy.cu", "lp_adamw.cu"])
def test_every_kernel_tests_its_indexes(source):
    with open(os.path.join(_build_lib.CSRC, source)) as f:
        found = dict(bodies(f.read(), KERNEL))
    assert found
    for name, body in found.items():
        assert "LP_CHECK(" in body, f"{source}: {name}"


def test_row_copies_and_stores_test_theirs():
    """The accesses that the norm's kernels make through their shared parts."""
    with open(os.path.join(_build_lib.CSRC, "lp_norm.cuh")) as f:
        text = f.read()
    wanted = {"fetch": 5, "put": 3, "read_weight": 1}  # the ways that an operand is reached
    found = dict(bodies(text, r"__device__ __forceinline__ void (fetch|put|read_weight)\("))
    assert set(found) == set(wanted)
    for name, body in found.items():
        assert body.count("LP_CHECK(") >= wanted[name], name
