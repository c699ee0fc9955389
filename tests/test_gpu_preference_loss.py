"""The preference loss and its gradient on a GB300 against the fp64 oracle.

Tolerances, with u = 2^-24.  A sum is a float pair: each two-sum is exact, its error of at most u S (S: the
sum of the magnitudes) goes into the low part, and what n of them make, n u S, is rounded at each of n
additions: n^2 u^2 S at most.  n is the longest chain: a lane's rows (16; with one CTA a sequence's rows over
its warps' lanes, at most 10 here), the lanes' tree (5), then chunks over a pair's lanes and their tree, or the
warps of a team (at most 16): n <= 45, 2^11 u^2 = 2^-37.  A score is rounded once to float32 for rewards: u.
z is beta times that, held as a pair, so its error is ez = beta 2^-37 S, far below u |z|.  In the sigmoid kind exp(-|z|)
is expf's 2 units and 2 roundings and is within 8 u relatively, as are log1p, the reciprocal and the product
after it: the slope is within 16 u of the terms' sizes and what ez changes (a slope of at most 1/4 of them).  A gradient is a slope times
factors held as pairs, rounded once."""

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import autograd, tune
from oracle import tune as ot

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def host(t):
    return None if t is None else t.cpu().numpy()


def make(lengths, ref=True, masked=0.3, seed=0, lead=0, trail=0, drift=0.1, empty=()):
    """Rows of sequences, `lead` rows before the first and `trail` behind the last.  empty: sequences
    whose mask leaves nothing."""
    g = torch.Generator(device=DEV).manual_seed(seed + sum(lengths))
    cu = torch.tensor([0, *lengths]).cumsum(0) + lead
    T = int(cu[-1]) + trail
    logp = -torch.empty(T, device=DEV).exponential_(1.0, generator=g)
    x = {"ref_logp": logp + drift * torch.randn(T, generator=g, device=DEV) if ref else None, "mask": None}
    if masked:
        mask = torch.rand(T, generator=g, device=DEV) >= masked
        for i in empty:
            mask[int(cu[i]):int(cu[i + 1])] = False
        x["mask"] = mask
        logp = torch.where(mask, logp, torch.full_like(logp, float("nan")))
    return logp, cu.to(DEV), x


def check(logp, cu, x, **kw):
    out = tune.preference_loss(logp, cu, **x, **kw)
    h = {k: host(v) for k, v in x.items()}
    stats, rewards, grad = ot.preference_loss(host(logp), host(cu), **h, **kw)
    beta, kind = kw.get("beta", 0.1), kw.get("kind", "sigmoid")
    keep = np.ones(logp.shape[0], bool) if h["mask"] is None else h["mask"]
    size = np.where(keep, np.abs(host(logp).astype(np.float64)), 0.0)
    if h["ref_logp"] is not None:
        size = size + np.where(keep, np.abs(h["ref_logp"]), 0.0)
    c = host(cu)
    S = np.array([size[c[i]:c[i + 1]].sum() for i in range(len(c) - 1)])
    n = np.array([max(1, keep[c[i]:c[i + 1]].sum()) for i in range(len(c) - 1)])
    if kw.get("average"):
        S = S / n
    ez = 2.0 ** -37 * beta * (S.max(initial=0.0) * 2)
    got = [host(t).astype(np.float64) for t in out]
    assert np.all(np.abs(got[1] - rewards) <= 1.01 * U * np.abs(rewards) + beta * 2.0 ** -37 * S)
    # a pair's slope in z, in size, and how it changes with z
    steep = {"sigmoid": 1.0, "hinge": 1.0, "square": 2 * np.abs(rewards).max(initial=0.0) * 2 / beta ** 2 + 1 / beta ** 2}[kind]
    bend = {"sigmoid": 0.25, "hinge": 0.0, "square": 2 / beta ** 2}[kind]
    pairs = max(1, len(c) // 2)
    counted = max(1, np.count_nonzero([keep[c[i]:c[i + 1]].any() for i in range(len(c) - 1)]) // 2)
    assert counted <= pairs
    loss_size = np.abs(stats[:3]).max() + steep * ez + 1.0
    assert np.all(np.abs(got[0][:3] - stats[:3]) <= 20 * U * loss_size + steep * ez)
    assert abs(got[0][3] - stats[3]) <= U
    assert np.all(np.abs(got[0][4:] - stats[4:]) <= 2 * U * np.abs(rewards).max(initial=0.0) + ez)
    # the smoothed slope is a difference of terms of up to 1; a row's share is beta / n of it
    least = 16 * U * (np.abs(grad) + (kw.get("label_smoothing", 0.0) > 0) * beta / 1.0) + beta * bend * ez
    if kw.get("nll_coef"):
        least = least + 4 * U * abs(kw["nll_coef"])
    assert np.all(np.abs(got[2] - grad) <= least)
    assert np.all(got[2][~keep] == 0)
    return out


KINDS = [dict(), dict(kind="hinge", beta=0.5, margin=0.25), dict(kind="square", beta=0.3, average=True),
         dict(label_smoothing=0.1, margin=-0.5, nll_coef=0.3), dict(average=True, beta=2.0, nll_coef=1.0),
         dict(kind="square", beta=0.2, nll_coef=0.1, margin=0.1)]
LENGTHS = [[5, 3], [1, 1], [0, 4, 3, 2], [60, 1, 64, 33, 20, 7, 9, 31], [4000, 4100], [1] * 64, [127, 129] * 16,
           [513, 2, 8000, 3], [1] * 66, [300, 0, 0, 700] * 20, [20000, 1, 511, 512], [512] * 40, [3] * 4000,
           [100001, 70000], [1, 0] * 40]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("lengths", LENGTHS)
def test_kinds_and_lengths(lengths, kw):
    check(*make(lengths), **kw)
    check(*make(lengths, ref=False, masked=0.0), halves=True, **kw)


@pytest.mark.parametrize("lead,trail", [(0, 37), (3, 0), (700, 1500), (5000, 9000)])
def test_rows_in_no_sequence(lead, trail):
    logp, cu, x = make([40, 9, 300, 301], lead=lead, trail=trail)
    out = check(logp, cu, x, beta=0.2)
    assert not out.grad_logp[:lead].any() and not out.grad_logp[logp.shape[0] - trail:].any()


@pytest.mark.parametrize("lengths", [[40, 30, 20, 10, 50, 60], [4000, 3000, 2000, 1000, 5000, 6000]])
def test_pairs_without_a_counted_row(lengths):
    """Pairs one or both of whose sequences the mask leaves empty: no gradient, no part of any mean."""
    logp, cu, x = make(lengths, empty=(1, 4, 5))
    out = check(logp, cu, x, beta=0.3, nll_coef=0.5)
    c = host(cu)
    for i in (0, 1, 4, 5):
        assert not out.grad_logp[c[i]:c[i + 1]].any()
    assert out.grad_logp[c[2]:c[4]].any()
    assert out.rewards[1] == 0 and out.rewards[4] == 0 and out.rewards[0] != 0
    x["mask"].zero_()
    out = tune.preference_loss(logp, cu, **x, nll_coef=0.5)
    assert not out.stats.any() and not out.rewards.any() and not out.grad_logp.any()


@pytest.mark.parametrize("T,n", [(0, 0), (0, 6), (0, 200), (700, 0), (9000, 0)])
def test_nothing_to_pair(T, n):
    logp = -torch.ones(T, device=DEV)
    out = tune.preference_loss(logp, torch.zeros(n + 1, dtype=torch.int64, device=DEV), kind="hinge")
    assert out.grad_logp.shape == (T,) and out.rewards.shape == (n,)
    assert not out.stats.any() and not out.rewards.any() and not out.grad_logp.any()


@pytest.mark.parametrize("scale", [1, 400])
def test_infinite_and_missing_values(scale):
    """A counted NaN or infinity shows in its own pair and the means, and in no other row's gradient's
    finiteness; a saturated pair has a slope of exactly 0 or -1."""
    lengths = [8 * scale, 6 * scale, 5 * scale, 9 * scale, 7 * scale, 4 * scale]
    logp, cu, x = make(lengths, masked=0.0)
    c = host(cu)
    bad = logp.clone()
    bad[c[2] + 1] = float("nan")
    out = tune.preference_loss(bad, cu, **x)
    assert torch.isnan(out.stats[0]) and torch.isnan(out.grad_logp[c[2]:c[4]]).all()
    assert torch.isfinite(out.grad_logp[:c[2]]).all() and torch.isfinite(out.grad_logp[c[4]:]).all()
    low = logp.clone()
    low[c[1]] = -float("inf")  # a rejected sequence that cannot occur: nothing more to gain
    out = tune.preference_loss(low, cu, **x)
    assert torch.isfinite(out.stats[0]) and not out.grad_logp[:c[2]].any() and out.rewards[1] == -float("inf")
    low = logp.clone()
    low[c[0] + 3] = -float("inf")  # a chosen sequence that cannot
    out = tune.preference_loss(low, cu, **x, beta=0.25)
    assert out.stats[0] == float("inf")
    want = torch.full((c[1] - c[0],), -0.25 / 3, device=DEV)
    assert torch.equal(out.grad_logp[:c[1]], want) and torch.equal(out.grad_logp[c[1]:c[2]], -want[:1].expand(c[2] - c[1]))


def test_long_sums_that_nearly_cancel():
    """Scores of -10^5 each whose difference is of order one: the loss keeps float32's precision."""
    logp, cu, x = make([100000, 100000], ref=False, masked=0.0)
    logp[100000:] = logp[:100000].flip(0)
    logp[-1] += 0.75
    check(logp, cu, x, beta=1.0)
    out = tune.preference_loss(logp, cu, beta=1.0)
    z = float(np.sum(host(logp[:100000]).astype(np.float64)) - np.sum(host(logp[100000:]).astype(np.float64)))
    assert abs(float(out.stats[1]) - np.log1p(np.exp(-z))) <= 1e-6


@pytest.mark.parametrize("lengths", [[30, 40, 3, 700], [3000, 900, 4000, 4500, 2, 7]])
def test_alignment_does_not_show(lengths):
    logp, cu, x = make(lengths)
    want = check(logp, cu, x)
    for shift in (1, 2, 3):
        def moved(t):
            base = torch.empty(t.shape[0] + shift, dtype=t.dtype, device=DEV)
            base[shift:] = t
            return base[shift:]
        got = tune.preference_loss(moved(logp), cu, **{k: moved(v) for k, v in x.items()})
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("lengths", [[30, 40, 3, 700], [3000, 900, 4000, 4500, 2, 7]])
def test_streams_graphs_and_repeats(lengths):
    logp, cu, x = make(lengths)
    want = tune.preference_loss(logp, cu, **x, nll_coef=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tune.preference_loss(logp, cu, **x, nll_coef=0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    size = tune.preference_loss_workspace_size(logp.shape[0], len(lengths))
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tune.preference_loss(logp, cu, **x, nll_coef=0.1, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(tune.LpError):
        tune.preference_loss(logp, cu, **x, workspace=ws[:size - 1])


@pytest.mark.parametrize("n", [6, 600])
def test_offsets_that_do_not_ascend(n):
    """Offsets that are no offsets: the call ends, whatever it gives."""
    rng = np.random.default_rng(n)
    for T in (50, 20000):
        cu = torch.from_numpy(rng.integers(-T, 2 * T, n + 1)).to(DEV)
        out = tune.preference_loss(-torch.ones(T, device=DEV), cu)
        torch.cuda.synchronize()
        assert out.grad_logp.shape == (T,)


def test_refusals():
    logp, cu, x = make([5, 3])
    call = lambda *a, **kw: tune.preference_loss(*(a or (logp, cu)), **{**x, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="kind"):
        call(kind="logistic")
    with pytest.raises(ValueError, match="pairs"):
        call(logp, cu[:2])
    with pytest.raises(ValueError, match="cu_seqlens"):
        call(logp, cu[:0])
    with pytest.raises(TypeError, match="cu_seqlens must be int64"):
        call(logp, cu.int())
    with pytest.raises(TypeError, match="logp must be float32"):
        call(logp.bfloat16(), cu)
    with pytest.raises(ValueError, match="ref_logp"):
        call(ref_logp=logp[:3])
    with pytest.raises(TypeError, match="mask must be bool"):
        call(mask=x["mask"].float())
    with pytest.raises(ValueError, match="CUDA"):
        call(logp, cu.cpu())
    for bad in (dict(beta=0.0), dict(beta=-1.0), dict(beta=float("nan")), dict(beta=1e-320),
                dict(margin=float("inf")), dict(label_smoothing=1.5), dict(label_smoothing=-0.1),
                dict(label_smoothing=0.1, kind="hinge"), dict(nll_coef=float("nan"))):
        with pytest.raises(tune.LpError):
            call(**bad)


def test_autograd():
    """The binding's gradient is the call's scaled, and that of differences of the oracle's loss."""
    logp, cu, x = make([6, 4, 3, 8], masked=0.0)
    kw = dict(beta=0.4, label_smoothing=0.05, nll_coef=0.2)
    leaf = logp.clone().requires_grad_()
    loss, stats, rewards = autograd.preference_loss(leaf, cu, ref_logp=x["ref_logp"], **kw)
    assert not stats.requires_grad and not rewards.requires_grad and torch.equal(loss, stats[0])
    (2.0 * loss).backward()
    want = tune.preference_loss(logp, cu, ref_logp=x["ref_logp"], **kw)
    assert torch.equal(leaf.grad, 2.0 * want.grad_logp)
    at, step = host(logp).astype(np.float64), 1e-6
    f = lambda v: ot.preference_loss(v, host(cu), ref_logp=host(x["ref_logp"]), **kw)[0][0]  # noqa: E731
    for t in range(at.shape[0]):
        e = np.zeros_like(at)
        e[t] = step
        slope = (f(at + e) - f(at - e)) / (2 * step)
        assert abs(float(want.grad_logp[t]) - slope) <= 1e-8 + 32 * U * abs(slope)
    g, = torch.autograd.grad(autograd.preference_loss(leaf, cu)[0], leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="gradient of a gradient"):
        g.sum().backward()
