"""The policy loss at the ends of its range: sequences by the thousand million, differences whose
exponentials pass float32, coefficients of zero."""

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import train

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def milliseconds(call):
    """The fastest of three, on the GPU."""
    call()
    times = []
    for _ in range(3):
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        call()
        stop.record()
        stop.synchronize()
        times.append(start.elapsed_time(stop))
    return min(times)


@pytest.mark.parametrize("T,first,empty", [(9002, 4502, 300_000), (2_000_002, 4502, 300_000),
                                           (9002, 0, 300_000), (8002, 4001, 1900)])
@pytest.mark.parametrize("reduction", ["sequence", "token"])
def test_empty_sequences_are_passed_at_once(T, first, empty, reduction):
    """Two sequences on either side of many empty ones have the weights of the two alone, and the
    call takes no time for the others (walked one by one, 300 000 took 60 ms; they may take 2)."""
    g = torch.Generator(device=DEV).manual_seed(1)
    logp = -torch.rand(T, generator=g, device=DEV)
    old = logp + 0.1 * torch.randn(T, generator=g, device=DEV)
    A = torch.randn(T, generator=g, device=DEV)
    mask = torch.rand(T, generator=g, device=DEV) < 0.5
    mask[first - 4:first + 4] = True
    cu = torch.full((empty + 3,), first, dtype=torch.int64, device=DEV)
    cu[0], cu[-1] = 0, T
    small = torch.tensor([0, first, T], device=DEV)
    run = lambda c: train.policy_loss(logp, old, A, mask=mask, cu_seqlens=c, reduction=reduction,  # noqa: E731
                                      per_sequence=False)
    for a, b in zip(run(cu), run(small)):
        assert (a is None and b is None) or torch.equal(a, b)
    advantages = torch.zeros(empty + 2, device=DEV)
    advantages[0], advantages[-1] = 1.5, -0.5
    with_each = lambda c, v: train.policy_loss(logp, old, v, mask=mask, cu_seqlens=c, reduction=reduction,  # noqa: E731
                                               per_sequence=True)
    for a, b in zip(with_each(cu, advantages), with_each(small, advantages[[0, -1]])):
        assert (a is None and b is None) or torch.equal(a, b)
    assert milliseconds(lambda: with_each(cu, advantages)) < 2.0


def test_offsets_padded_to_a_capacity():
    """Offsets that repeat the last one, as for a fixed capacity of sequences."""
    T = 61
    logp = -torch.rand(T, device=DEV)
    cu = torch.tensor([0, 20, 61], device=DEV)
    padded = torch.cat([cu, torch.full((2000,), T, device=DEV)])
    for reduction in ("sequence", "token"):
        run = lambda c: train.policy_loss(logp, logp * 1.1, -logp, cu_seqlens=c, reduction=reduction)  # noqa: E731
        for a, b in zip(run(padded), run(cu)):
            assert (a is None and b is None) or torch.equal(a, b)


def test_more_than_2_to_30_sequences_in_a_chunk():
    """The search for a row's sequence among n has sums of up to 2 n.  Two sequences lie on either
    side of 1.2e9 empty ones: the weights are those of the two alone."""
    empty, first, T = 1_200_000_000, 4502, 9002
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    g = torch.Generator(device=DEV).manual_seed(1)
    logp = -torch.rand(T, generator=g, device=DEV)
    old = logp + 0.1 * torch.randn(T, generator=g, device=DEV)
    A = torch.randn(T, generator=g, device=DEV)
    cu = torch.full((empty + 3,), first, dtype=torch.int64, device=DEV)
    cu[0], cu[-1] = 0, T
    small = torch.tensor([0, first, T], device=DEV)
    for reduction in ("sequence", "token"):
        got = train.policy_loss(logp, old, A, cu_seqlens=cu, reduction=reduction)
        ref = train.policy_loss(logp, old, A, cu_seqlens=small, reduction=reduction)
        for a, b in zip(got, ref):
            assert (a is None and b is None) or torch.equal(a, b)


def test_exponentials_are_good_to_the_last_places():
    """The gradient of a row with advantage -1 is its weight, a power of two here, times the ratio:
    the float32 exponential of an exact difference, whose error CUDA gives as at most 1 unit in the
    last place; 2 are asked.  An exponential by way of a rounded exponent is 14 off at 10."""
    n = 8192
    delta = torch.linspace(-13, 85, n, dtype=torch.float64).float()
    zero = torch.zeros(n, device=DEV)
    got = train.policy_loss(delta.to(DEV), zero, zero - 1, clip_low=1 - 1e-6).grad_logp
    want = np.exp(delta.double().numpy())
    assert np.all(np.abs(got.double().cpu().numpy() * n - want) <= 2 * 2.0 ** -23 * want)
    # and that of the divergence's, with no advantage: minus its coefficient times expm1
    got = train.policy_loss(zero, zero, zero, ref_logp=delta.to(DEV), kl_coef=1.0).grad_logp
    want = -np.expm1(delta.double().numpy())
    assert np.all(np.abs(got.double().cpu().numpy() * n - want) <= 2 * 2.0 ** -23 * np.abs(want))


@pytest.mark.parametrize("T", [4, 20000])
def test_a_row_without_advantage_adds_nothing(T):
    """exp(delta) passes float32 from 88.7 on; the product with an advantage of 0 is 0 in the
    definition, not NaN.  (T: one launch, two passes.)"""
    delta, A = torch.full((T,), 0.1, device=DEV), torch.ones(T, device=DEV)
    delta[1], A[1] = 100.0, 0.0
    delta[2], A[2] = 100.0, 2.0    # clipped: the value is that of the limit
    delta[3], A[3] = -100.0, -2.0  # clipped on the other side
    zero = torch.zeros(T, device=DEV)
    got = train.policy_loss(delta, zero, A)
    assert torch.isfinite(got.grad_logp).all() and not got.grad_logp[1:4].any()
    want = -((T - 3) * np.exp(np.float64(np.float32(0.1))) + 2 * 1.2 - 2 * 0.8) / T
    assert abs(float(got.stats[0]) - want) <= 4200 * 2.0 ** -24 * abs(want)
    # an infinite difference is one, and an advantage that is not zero loses that much
    delta[1] = float("inf")
    assert torch.isnan(train.policy_loss(delta, zero, A).grad_logp[1])
    delta[1], A[1] = 100.0, -1e3
    assert float(train.policy_loss(delta, zero, A).grad_logp[1]) == float("inf")


@pytest.mark.parametrize("T", [4, 20000])
def test_terms_with_a_coefficient_of_zero_are_only_watched(T):
    """An estimate of the divergence that passes float32, or an entropy that is none, shows in its
    statistic and nowhere else."""
    logp = torch.full((T,), -0.5, device=DEV)
    logp[1] = -100.0
    entropy = torch.ones(T, device=DEV)
    entropy[2] = float("nan")
    A = torch.ones(T, device=DEV)
    ref = train.policy_loss(logp, logp, A)
    got = train.policy_loss(logp, logp, A, ref_logp=torch.zeros(T, device=DEV), entropy=entropy)
    assert float(got.stats[2]) == float("inf") and torch.isnan(got.stats[3])
    assert torch.equal(got.stats[:2], ref.stats[:2]) and torch.equal(got.grad_logp, ref.grad_logp)
    assert not got.grad_entropy.any()
