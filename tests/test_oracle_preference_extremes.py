"""The oracle's preference loss where a term is infinite (CPU only)."""

import numpy as np
import pytest

from oracle import tune as ot


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("side", [0, 1])
def test_an_infinite_term_counts_by_its_weight(side, smoothing):
    logp = np.array([-1.0, -1.0])
    logp[side] = -np.inf
    stats, _, grad = ot.preference_loss(logp, np.array([0, 1, 2]), beta=0.5, label_smoothing=smoothing)
    weight = (1 - smoothing, smoothing)[side]  # of the term that is infinite
    assert stats[0] == (np.inf if weight else 0.0)
    np.testing.assert_array_equal(grad, 0.5 * weight * (np.array([-1.0, 1.0]) if side == 0 else np.array([1.0, -1.0])))


def test_a_score_that_is_no_number_shows():
    for smoothing in (0.0, 0.1, 1.0):
        stats, _, grad = ot.preference_loss(np.array([np.nan, -1.0]), np.array([0, 1, 2]), label_smoothing=smoothing)
        assert np.isnan(stats[0]) and np.isnan(grad).all()
