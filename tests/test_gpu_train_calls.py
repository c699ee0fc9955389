"""What the calls of train.py and their autograd forms owe their caller besides the numbers:
what they return where these are not finite, streams, lifetimes, versions, serialisation."""

import pytest
import torch

from invariant_token_logprobs_gb300 import autograd, train  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value,want", [("inf", "inf"), ("-inf", "inf"), ("1e30", "inf"), ("nan", "nan")])
@pytest.mark.parametrize("at", [0, 4321])
def test_norm_of_gradients_that_are_not_finite(bits, value, want, at):
    """An infinite gradient, or squares past float32, have an infinite norm; only a NaN has a NaN."""
    p, g = torch.ones(5000, device=DEV), torch.ones(5000, device=DEV)
    g[at] = float(value)
    norm = train.AdamW([p], [g], state_bits=bits).step(max_norm=1.0)
    assert str(float(norm)) == want
    assert torch.equal(p, torch.ones_like(p))
