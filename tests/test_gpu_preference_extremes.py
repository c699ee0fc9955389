"""The preference loss at the ends of its arguments and of its sequences' lengths, on a GB300.

u = 2^-24.  Where a tolerance is named it is derived in the test."""

import math

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import tune
from oracle import tune as ot

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def host(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("scale", [1, 400])  # one CTA, and three launches
@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("side", [0, 1])
def test_a_term_without_a_weight_is_none(side, smoothing, scale):
    """z of both infinities: the term that is infinite counts by its weight, and not at all where that is 0.  Every
    finite value here is exact: weights of 1 / 2 of two pairs, and a slope of 0 or of a weight.

    The other pair's loss has 20 u of the terms' sizes, which are below 8 (|z| is)."""
    lengths = [8 * scale, 6 * scale, 5 * scale, 9 * scale]
    cu = torch.tensor([0, *lengths], device=DEV).cumsum(0)
    c = host(cu)
    logp = torch.full((int(c[-1]),), -2.0 ** -12, device=DEV)
    logp[c[side]] = -math.inf
    out = tune.preference_loss(logp, cu, beta=0.25, label_smoothing=smoothing)
    stats, rewards, grad = ot.preference_loss(host(logp), c, beta=0.25, label_smoothing=smoothing)
    weight = (1 - smoothing, smoothing)[side]
    assert math.isinf(stats[0]) == (weight != 0)
    assert float(out.stats[0]) == stats[0] or abs(float(out.stats[0]) - stats[0]) <= 20 * U * 8
    assert out.rewards[side] == -math.inf and rewards[side] == -math.inf
    got = host(out.grad_logp).astype(np.float64)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - grad) <= 16 * U * 0.25)
    assert np.all(got[:c[1]] == got[0]) and abs(got[0]) == np.float32(0.125 * np.float32(weight))


@pytest.mark.parametrize("scale", [1, 1200])  # one CTA, and three launches
@pytest.mark.parametrize("beta", [1e-37, 1e-25, 1e-3, 1.0, 1e25, 1e37])
def test_the_square_kinds_gradient_over_the_range_of_beta(beta, scale):
    """The loss is (gap - 1 / (2 beta))^2 with margin 0, and its gradient twice the base over the pairs' number, which is
    finite wherever the base is.  The base is a pair's product, settled (2 u), the rest 2 more; the gap is exact."""
    lengths = [2 * scale, 3 * scale, 4 * scale, scale]
    cu = torch.tensor([0, *lengths], device=DEV).cumsum(0)
    c = host(cu)
    logp = torch.zeros(int(c[-1]), device=DEV)
    logp[c[1]], logp[c[2]] = -2.0 ** -40, -3.0
    out = tune.preference_loss(logp, cu, kind="square", beta=beta)
    half = 0.5 / beta
    for i, base in enumerate((2.0 ** -40 - half, -3.0 - half)):
        for j, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
            got = host(out.grad_logp[c[j]:c[j + 1]]).astype(np.float64)
            assert np.all(np.abs(got - sign * base) <= 4 * U * abs(base)), (beta, got[0], base)


def test_means_of_more_rows_than_float32_counts():
    """Sequences of 2^24 + 1 and 2^24 + 3 rows of -1, whose means are -1 both: every sum is of integers that a pair holds,
    and the quotient's rest is 0, so that z is 0 without an error.  (A divisor in float32 made it -1/8.)"""
    lengths = [2 ** 24 + 1, 2 ** 24 + 3]
    cu = torch.tensor([0, *lengths], device=DEV).cumsum(0)
    logp = torch.full((sum(lengths),), -1.0, device=DEV)
    beta = 2.0 ** 20
    out = tune.preference_loss(logp, cu, beta=beta, average=True)
    stats = out.stats.tolist()
    assert abs(stats[0] - math.log(2.0)) <= 20 * U
    assert stats[3:] == [0.0, -beta, -beta] and out.rewards.tolist() == [-beta, -beta]
    for rows, n, sign in ((out.grad_logp[:lengths[0]], lengths[0], -1.0), (out.grad_logp[lengths[0]:], lengths[1], 1.0)):
        low, high = torch.aminmax(rows)
        want = sign * 0.5 * beta / n
        assert float(low) == float(high) and abs(float(low) - want) <= 16 * U * abs(want)
