"""Pins for the fp64 oracle of the training-step operators (CPU only): gradients against
central differences of the definitions, closed forms, and a published Philox vector."""

import numpy as np
import pytest

from oracle import train as ot

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


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("weight", [False, True])
def test_residual_norm_gradients(post, gate, weight):
    rng = np.random.default_rng(5)
    T, d = 3, 5
    r, y = rng.normal(size=(T, d)), rng.normal(size=(T, d))
    wb = rng.normal(size=d) if post else None
    w = rng.normal(size=d) if weight else None
    g = {None: None, "channel": rng.normal(size=d), "token": rng.normal(size=(T, d))}[gate]
    gh, gr = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def forward():
        return ot.residual_norm(r, y, w, wb, g, 0.9, 0.7, 1e-3)

    def loss():
        h, new, _, _ = forward()
        return np.sum(new * gr) + (np.sum(h * gh) if weight else 0.0)

    _, new, rstd, branch_rstd = forward()
    got = ot.residual_norm_backward(gh if weight else None, gr, new, rstd, y, w, wb, branch_rstd,
                                    g, 0.9, 0.7)
    for x, grad in zip((r, y, w, wb, g), got):
        assert (x is None) == (grad is None)
        if x is not None:
            assert np.max(np.abs(_difference(loss, x) - grad)) < 1e-8


def test_residual_norm_closed_forms():
    # a row of equal entries norms to 1 (eps 0), and any multiple of it to the same
    r = np.full((2, 4), 3.0) * np.array([[1.0], [-5.0]])
    h, new, rstd, _ = ot.residual_norm(r, weight=np.arange(1.0, 5.0), eps=0.0)
    assert np.allclose(h, np.array([[1.0], [-1.0]]) * np.arange(1.0, 5.0))
    assert np.array_equal(new, r) and np.allclose(rstd, [1 / 3, 1 / 15])


@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_loss_gradients(reduction):
    rng = np.random.default_rng(7)
    cu, T = [0, 4, 4, 9, 12], 12
    logp, old = -rng.random(T), -rng.random(T)
    # float32 values, so that the clip's decision is that of the float64 difference
    logp, old = (x.astype(np.float32).astype(np.float64) for x in (logp, old))
    ref, ent, mask = -rng.random(T), rng.random(T), rng.random(T) < 0.7
    mask[:4] = False
    A = np.array([1.0, -2.0, 1.5, -0.5])
    kw = dict(mask=mask, ref_logp=ref, entropy=ent, cu_seqlens=cu, reduction=reduction,
              per_sequence=True, kl_coef=0.3, entropy_coef=0.2)
    stats, g_logp, g_ent = ot.policy_loss(logp, old, A, **kw)
    f = lambda: ot.policy_loss(logp, old, A, **kw)[0][0]  # noqa: E731
    assert np.max(np.abs(_difference(f, logp) - g_logp)) < 1e-8
    assert np.max(np.abs(_difference(f, ent) - g_ent)) < 1e-8
    assert np.all(g_logp[:4] == 0) and stats[4] > 0


def test_policy_loss_weights():
    # equal old and new policies: the loss is minus the mean advantage, each way of averaging
    logp, A = np.zeros(5), np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    assert np.isclose(ot.policy_loss(logp, logp, A)[0][0], -3.0)
    by = ot.policy_loss(logp, logp, A, cu_seqlens=[0, 1, 5], reduction="sequence")[0][0]
    assert np.isclose(by, -(1.0 + 3.5) / 2)
    assert np.all(ot.policy_loss(logp, logp, A, mask=np.zeros(5))[0] == 0)


def test_adamw_first_step_is_the_sign():
    p, m, v = ot.adamw_step([1.0, 1.0], [0.5, -3.0], [0.0, 0.0], [0.0, 0.0], 1, 0.1, (0.9, 0.999),
                            1e-12, 0.5)
    assert np.allclose(p, [1 - 0.05 - 0.1, 1 - 0.05 + 0.1]) and np.allclose(m, [0.05, -0.3])


def test_moment_codes():
    m, u = ot.moment_values(True), ot.moment_values(False)
    assert len(m) == 128 and len(u) == 256 and m[-1] == u[-1] == 1.0
    assert m[1] == 1.25 * 2.0 ** -16 and u[1] == 1.125 * 2.0 ** -16
    # the codes are the leading bits of the float
    for values, shift, first in ((m, 20, 889), (u, 19, 1777)):
        bits = ((np.arange(1, len(values)) + first) << shift).astype(np.uint32)
        assert np.array_equal(bits.view(np.float32).astype(np.float64), values[1:])
    low, high, part = ot.moment_neighbours(np.array([0.53, 1.0, 0.0]), 1.0, True)
    assert np.allclose(low, [0.5, 1.0, 0.0]) and np.allclose(high, [0.5625, 1.0, m[1]])
    assert np.allclose(part, [0.48, 0.0, 0.0])


def test_philox_published_vector():
    assert ot.philox_4x32_7((0, 0, 0, 0), (0, 0)) == [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]
