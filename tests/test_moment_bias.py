"""What holding the root of the second moment in 8 bits does to the second moment over many steps,
as include/lp_train.h states it: simulated with the oracle's codes (CPU)."""

import numpy as np
import pytest

from oracle import train as ot


@pytest.mark.parametrize("beta2", [0.99, 0.999, 0.9999])
def test_the_second_moment_settles_a_few_per_cent_high(beta2):
    """Noisy gradients of many sizes; each step rounds the root up or down a code by chance.  The
    mean over 5120 elements of ratios that spread by 10 to 15% is good to 0.2%."""
    rng = np.random.default_rng(0)
    values = ot.moment_values(False)
    size = np.exp(rng.normal(size=(20, 256)))
    u = np.zeros_like(size)
    v_exact = np.zeros_like(size)
    for _ in range(1000):
        g2 = (size * rng.normal(size=size.shape)) ** 2
        v_exact = beta2 * v_exact + (1 - beta2) * g2
        root = np.sqrt(beta2 * u * u + (1 - beta2) * g2)
        scale = root.max(axis=1, keepdims=True)
        low = np.searchsorted(values, root / scale, side="right") - 1
        high = np.minimum(low + 1, len(values) - 1)
        share = (root / scale - values[low]) / np.where(high > low, values[high] - values[low], 1)
        u = np.where(rng.random(size.shape) < share, values[high], values[low]) * scale
    assert 1.01 < np.mean(u * u / v_exact) < 1.035
    assert np.mean(u / np.sqrt(v_exact)) < 1.012
