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


def rows(lengths, seed=0):
    """logp, offsets and a reference of sequences of these lengths."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    cu = torch.tensor([0, *lengths], device=DEV).cumsum(0)
    logp = -torch.empty(int(cu[-1]), device=DEV).exponential_(1.0, generator=g)
    return logp, cu, logp + 0.1 * torch.randn(logp.shape, generator=g, device=DEV)


LONG = {"one": [16] * 1001 + [1 << 20] + [16] * 2998, "side by side": [20] * 1002 + [70000, 131072, 5, 90001] + [3] * 1994,
        "at the end": [40] * 4999 + [300000],
        "empty ones between": [700, 5, 0, 0, 3] + [0] * 5001 + [31, 0, 900, 40] + [0] * 70 + [3000, 9],
        "runs of empty ones": ([90, 90] + [0] * 100) * 60, "empty ones around": [0] * 3000 + [9000, 800, 7, 1] + [0] * 2000,
        "every other one empty": [3, 2, 0, 0] * 900, "32 and 33 empty ones": ([5, 6] + [0] * 32 + [7, 8, 9] + [0] * 33) * 100,
        "a few chunks": [1] * 3000 + [512 * 8, 512 * 8 + 1, 512 * 9, 7] + [1] * 3000}


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("lengths", LONG.values(), ids=LONG.keys())
def test_long_sequences_among_many_short_ones(lengths, average, halves):
    """The longest chain of additions is a lane's 16 rows and 5 steps of its warp, then 2048 / 32 chunks a lane and 5
    more: n = 90, so that a sum is within n^2 u^2 < 2^-35 of its terms' size S (each of n two-sums leaves at most n u S in
    the low part, rounded n times).  A mean divides both.  The stats' sums add no chain that shows: 2 u of the largest reward and
    what the scores' errors make; a sigmoid's slope is 16 u and a quarter of z's error."""
    logp, cu, ref = rows(lengths)
    out = tune.preference_loss(logp, cu, ref_logp=ref, beta=0.05, average=average, halves=halves)
    stats, rewards, grad = ot.preference_loss(host(logp), host(cu), ref_logp=host(ref), beta=0.05, average=average,
                                              halves=halves)
    size = np.abs(host(logp).astype(np.float64)) + np.abs(host(ref).astype(np.float64))
    run = np.concatenate([[0.0], np.cumsum(size)])
    S = run[host(cu)[1:]] - run[host(cu)[:-1]]
    if average:
        S = S / np.maximum(lengths, 1)
    got = [host(t).astype(np.float64) for t in out]
    each = 0.05 * 2.0 ** -35 * S
    assert np.all(np.abs(got[1] - rewards) <= 1.01 * U * np.abs(rewards) + each)
    ez = 2 * each.max()
    assert np.all(np.abs(got[0][:3] - stats[:3]) <= 20 * U * (np.abs(stats[:3]).max() + 1) + ez)
    assert abs(got[0][3] - stats[3]) <= U
    assert np.all(np.abs(got[0][4:] - stats[4:]) <= 2 * U * np.abs(rewards).max() + ez)
    assert np.all(np.abs(got[2] - grad) <= 16 * U * np.abs(grad) + 0.05 * 0.25 * ez)
    for i in np.flatnonzero(np.array(lengths) == 0):
        assert got[1][i] == 0
    again = tune.preference_loss(logp, cu, ref_logp=ref, beta=0.05, average=average, halves=halves)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def microseconds(call):
    best = math.inf
    for _ in range(5):
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        call()
        start.record()
        for _ in range(10):
            call()
        stop.record()
        stop.synchronize()
        best = min(best, start.elapsed_time(stop) * 100)
    return best


def test_a_long_sequence_costs_what_it_costs_alone():
    """Among many short ones it is no chain of a single lane: the call takes 60 us, the long pair's and the short ones' own
    66 together, and a lane's chain took 564.  The bound is three times the calls apart."""
    short, long = [16] * 3998, [16, 1 << 20]

    def time_of(lengths):
        logp, cu, ref = rows(lengths)
        return microseconds(lambda: tune.preference_loss(logp, cu, ref_logp=ref))

    apart, together = time_of(short) + time_of(long), time_of(short[:2000] + long + short[2000:])
    print(f"apart {apart:.1f} us, together {together:.1f} us")
    assert together <= 3 * apart


def test_runs_of_empty_sequences_are_passed():
    """100000 of them between two answers: 19 us, and 1536 when they were gone through."""
    def time_of(lengths):
        logp, cu, ref = rows(lengths)
        return microseconds(lambda: tune.preference_loss(logp, cu, ref_logp=ref))

    without = time_of([5000] * 4)
    middle = time_of([5000, 5000] + [0] * 100000 + [5000, 5000])
    print(f"without {without:.1f} us, with {middle:.1f} us")
    assert middle <= 8 * without
