"""The fine-tuning operators past 2^31 elements, on a GB300.

What the last rows hold is known without a 64-bit pass over all of them: a row of the layer norm has the
bits that it has alone, the preference loss is of sums of a few ones, and Muon's gradient has one element
in each row and no two in a column, so that its singular values are all equal and X stays in those places."""

import math

import pytest
import torch

from invariant_token_logprobs_gb300 import tune
from oracle import tune as ot

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def test_layer_norm():
    T, d = 131200, 16384
    assert T * d > 2 ** 31
    r = torch.empty(T, d, device=DEV, dtype=torch.bfloat16).normal_()
    y = torch.empty(T, d, device=DEV, dtype=torch.bfloat16).normal_()
    w, b = torch.randn(d, device=DEV), torch.randn(d, device=DEV)
    out = tune.layer_norm(r, y, weight=w, bias=b)
    back = tune.layer_norm_backward(out.normed, None, out.residual, out.mean, out.rstd, weight=w, bias=b,
                                    branch=True, weight_grads=False)
    for at in (0, 65535, 131071, T - 3):
        rows = slice(at, at + 3)
        alone = tune.layer_norm(r[rows].clone(), y[rows].clone(), weight=w, bias=b)
        for got, want in zip(out, alone):
            assert torch.equal(got[rows], want)
        grad = tune.layer_norm_backward(alone.normed, None, alone.residual, alone.mean, alone.rstd, weight=w,
                                        bias=b, branch=True, weight_grads=False)
        assert torch.equal(back.residual[rows], grad.residual)


def test_preference_loss():
    """Scores -1, -3, -2 and 0 with beta 1, exact in float32; z = 2 and -2."""
    T = 2 ** 31 - 1
    logp = torch.zeros(T, device=DEV)
    logp[[2, 5, T // 2, T - 9, T - 8, T - 7]] = -1.0
    cu = torch.tensor([0, 5, T - 8, T - 6, T], device=DEV)
    out = tune.preference_loss(logp, cu, beta=1.0)
    assert out.rewards.tolist() == [-1.0, -3.0, -2.0, 0.0]
    loss = 0.5 * (math.log1p(math.exp(-2.0)) + math.log1p(math.exp(2.0)))
    assert abs(float(out.stats[0]) - loss) <= 20 * U * (loss + 1)
    slopes = [-0.5 / (1 + math.exp(2.0)), -0.5 / (1 + math.exp(-2.0))]
    bounds = cu.tolist()
    for i, want in enumerate((slopes[0], -slopes[0], slopes[1], -slopes[1])):
        rows = out.grad_logp[bounds[i]:bounds[i + 1]]
        low, high = torch.aminmax(rows)
        assert float(low) == float(high) and abs(float(low) - want) <= 16 * U * abs(want)


@pytest.mark.parametrize("tall", [False, True])
def test_muon(tall):
    """Tolerance: each step's three products have one term that is not zero, with three products of float16
    pairs of 2^-22 each and the polynomial's roundings, 16 at most: 13 times that in all, and the steps after
    multiply it by 450 at the most (as for dense matrices)."""
    m, n, steps = 33000, 65536, 5
    assert m * n > 2 ** 31
    rows = torch.arange(m, device=DEV)
    cols = (rows * 40503 + 7) % n  # an odd factor: no two are the same
    at = (cols, rows) if tall else (rows, cols)
    grad = torch.zeros((n, m) if tall else (m, n), device=DEV, dtype=torch.bfloat16)
    grad[at] = 2.0
    p = torch.zeros(grad.shape, device=DEV)
    tune.Muon([p], [grad], lr=1.0, momentum=0.0, scaling=1.0, steps=steps).step()
    s = 1 / math.sqrt(m)
    for _ in range(steps):
        s = ot.A * s + ot.B * s ** 3 + ot.C * s ** 5
    assert float((p[at] + s).abs().max()) <= 450 * 13 * (3 * 2.0 ** -22 + 16 * U) * s
    p[at] = 0.0
    low, high = torch.aminmax(p)
    assert float(low) == 0.0 and float(high) == 0.0
