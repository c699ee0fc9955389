"""Pins for the fp64 oracle of the fine-tuning operators (CPU only): gradients against central differences of
the definitions, closed forms, and the Newton-Schulz steps as products of matrices."""

import numpy as np
import pytest

from oracle import tune as ot

STEP = 1e-5  # central differences in float64: truncation ~1e-10, rounding ~1e-11


def _difference(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        kept = x[i]
        x[i] = kept + STEP
        up = f()
        x[i] = kept - STEP
        down = f()
        x[i] = kept
        g[i] = (up - down) / (2 * STEP)
    return g


@pytest.mark.parametrize("branch", [False, True])
@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm_gradients(branch, affine):
    rng = np.random.default_rng(3)
    T, d = 3, 6
    r, y = rng.normal(size=(T, d)), rng.normal(size=(T, d)) if branch else None
    w, b = (rng.normal(size=d), rng.normal(size=d)) if affine else (None, None)
    gh, gr = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss():
        n, new, _, _ = ot.layer_norm(r, branch=y, weight=w, bias=b, eps=1e-2)
        return (gh * n).sum() + (gr * new).sum()

    _, new, mean, rstd = ot.layer_norm(r, branch=y, weight=w, bias=b, eps=1e-2)
    D, gw, gb = ot.layer_norm_backward(gh, gr, new, mean, rstd, weight=w)
    np.testing.assert_allclose(D, _difference(loss, r), atol=1e-8)
    if branch:
        np.testing.assert_allclose(D, _difference(loss, y), atol=1e-8)
    if affine:
        np.testing.assert_allclose(gw, _difference(loss, w), atol=1e-8)
        np.testing.assert_allclose(gb, _difference(loss, b), atol=1e-8)


def test_layer_norm_closed_form():
    n, new, mean, rstd = ot.layer_norm(np.array([[1.0, 3.0]]), eps=0.0)
    np.testing.assert_allclose(n, [[-1.0, 1.0]])
    np.testing.assert_allclose([mean[0], rstd[0]], [2.0, 1.0])
    n, _, _, _ = ot.layer_norm(np.array([[5.0, 5.0]]), eps=1.0, weight=np.array([2.0, 2.0]), bias=np.array([0.5, 1.5]))
    np.testing.assert_allclose(n, [[0.5, 1.5]])


@pytest.mark.parametrize("kw", [dict(), dict(label_smoothing=0.2, nll_coef=0.3), dict(kind="square", beta=0.7),
                                dict(kind="hinge", beta=0.3, margin=0.4), dict(average=True, beta=2.0),
                                dict(halves=True, average=True, nll_coef=0.1, margin=-0.2)])
@pytest.mark.parametrize("ref", [False, True])
def test_preference_gradients(kw, ref):
    rng = np.random.default_rng(7)
    cu = np.array([1, 4, 4, 9, 12, 13, 16])
    logp = -rng.exponential(size=18)
    x = {"ref_logp": logp + 0.3 * rng.normal(size=18) if ref else None, "mask": rng.random(18) > 0.2}
    f = lambda: ot.preference_loss(logp, cu, **x, **kw)[0][0]  # noqa: E731
    _, _, grad = ot.preference_loss(logp, cu, **x, **kw)
    np.testing.assert_allclose(grad, _difference(f, logp), atol=1e-7)


def test_preference_closed_forms():
    cu, logp = np.array([0, 2, 3]), np.array([-1.0, -2.0, -5.0])
    z = 0.5 * 2.0
    stats, rewards, grad = ot.preference_loss(logp, cu, beta=0.5)
    np.testing.assert_allclose(stats, [np.log1p(np.exp(-z)), np.log1p(np.exp(-z)), 1.5, 1.0, -1.5, -2.5])
    np.testing.assert_allclose(rewards, [-1.5, -2.5])
    s = 0.5 / (1 + np.exp(z))
    np.testing.assert_allclose(grad, [-s, -s, s])
    stats, _, _ = ot.preference_loss(logp, cu, kind="square", beta=0.5, average=True)
    np.testing.assert_allclose(stats[1], (3.5 - 1.0) ** 2)
    stats, _, grad = ot.preference_loss(logp, cu, kind="hinge", beta=0.5, margin=0.25)
    np.testing.assert_allclose(stats[1], 0.25)
    # a pair without a counted row on one side is none
    stats, rewards, grad = ot.preference_loss(logp, np.array([0, 3, 3]))
    assert not stats.any() and not grad.any()


@pytest.mark.parametrize("shape", [(5, 8), (8, 5), (6, 6), (1, 4)])
def test_newton_schulz_is_the_products(shape):
    u = np.random.default_rng(1).normal(size=shape)
    x = u / (np.linalg.norm(u) + 1e-7)
    for _ in range(5):
        g = x @ x.T
        x = ot.A * x + (ot.B * g + ot.C * (g @ g)) @ x
    np.testing.assert_allclose(ot.newton_schulz(u, 5, 1e-7), x, atol=1e-10)


def test_newton_schulz_takes_singular_values_towards_one():
    """What the kernels' range rests on: on [0, 1] the polynomial stays below 1.21, and below 1.21 on [0, 1.21]; five
    steps take 0.01 and more into (0.6, 1.21)."""
    p = lambda s: s * (ot.A + s * s * (ot.B + ot.C * s * s))  # noqa: E731
    s = np.linspace(0, 1.21, 100001)
    assert p(s).max() < 1.21 and p(s).min() >= 0
    t = np.linspace(0.01, 1, 100001)
    for _ in range(5):
        t = p(t)
    assert t.min() > 0.6 and t.max() < 1.21
    # no element of P = a I + b G + c G G passes a
    g = s * s
    assert np.abs(ot.A + ot.B * g + ot.C * g * g).max() <= ot.A


def test_muon_step():
    rng = np.random.default_rng(2)
    p, g, m = rng.normal(size=(4, 6)), rng.normal(size=(4, 6)), rng.normal(size=(4, 6))
    new, buffer = ot.muon_step(p, g, m, lr=0.1, momentum=0.9, weight_decay=0.5, lr_scale=2.0, scaling="rms")
    np.testing.assert_allclose(buffer, 0.9 * m + g)
    x = ot.newton_schulz(g + 0.9 * buffer, 5, 1e-7)
    np.testing.assert_allclose(new, p * (1 - 0.1) - 0.2 * 0.2 * np.sqrt(6) * x)
    assert ot.muon_scale(8, 2, "spectral") == 2.0 and ot.muon_scale(2, 8, "spectral") == 1.0
