"""The policy loss on a GB300 against the fp64 oracle.

Tolerances, with u = 2^-24: exp and expm1 are within 2 units in the last place, and delta and r
are rounded once, which moves their exponentials by u |delta| relatively; a row's gradient is
those and three products and a sum, (16 + |delta| + |r|) u of its terms' magnitude.  A weight is
two rounded operations.  A statistic is a sum over at most T rows of such terms, in chains of at
most 4096 additions: 4200 u of the terms' summed magnitude."""

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import train
from oracle import train as ot

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def make(lengths, masked=0.3, ref=True, entropy=True, per_sequence=True, seed=0, lead=0, tail=0):
    """Rows of ragged sequences; `lead` and `tail` rows belong to no sequence."""
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64) + lead
    T = int(cu[-1]) + tail
    f = lambda x: x.astype(np.float32)  # noqa: E731
    logp = f(-rng.exponential(size=T))
    x = {"logp": logp, "old_logp": f(logp + 0.2 * rng.normal(size=T)), "cu_seqlens": cu,
         "advantages": f(rng.normal(size=len(lengths) if per_sequence else T)),
         "mask": rng.random(T) >= masked if masked is not None else None,
         "ref_logp": f(logp + 0.5 * rng.normal(size=T)) if ref else None,
         "entropy": f(3 * rng.random(T)) if entropy else None, "per_sequence": per_sequence}
    return x


def run(x, **kw):
    dev = {k: torch.from_numpy(v).to(DEV) if isinstance(v, np.ndarray) else v for k, v in x.items()}
    return train.policy_loss(**dev, **kw)


def check(x, **kw):
    got = run(x, **kw)
    ref = ot.policy_loss(**x, **kw)
    # magnitudes: the oracle on the terms' absolute values, by the largest a row can have
    T = len(x["logp"])
    w = ot.policy_loss(x["logp"], x["logp"], -np.ones_like(x["advantages"]), x["mask"],
                       cu_seqlens=x["cu_seqlens"], per_sequence=x["per_sequence"],
                       reduction=kw.get("reduction", "token"))[1]
    with np.errstate(invalid="ignore"):
        delta = np.abs(np.where(w > 0, x["logp"].astype(float) - x["old_logp"], 0))
        r = np.zeros(T) if x["ref_logp"] is None else \
            np.abs(np.where(w > 0, x["ref_logp"].astype(float) - x["logp"], 0))
    seq = np.clip(np.searchsorted(x["cu_seqlens"][1:], np.arange(T), side="right"), 0,
                  max(0, len(x["cu_seqlens"]) - 2))
    A = np.zeros(T)
    if T and len(x["advantages"]):
        A = np.abs(x["advantages"][seq] if x["per_sequence"] else x["advantages"])
    ent = np.zeros(T) if x["entropy"] is None else np.abs(np.where(w > 0, x["entropy"], 0))
    kl = kw.get("kl_coef", 0.0)
    mag = w * (A * np.exp(delta) + kl * (np.exp(r) + 1))
    g = got.grad_logp.double().cpu().numpy()
    assert np.all(np.abs(g - ref[1]) <= (16 + delta + r) * U * mag)
    assert np.all(g[w == 0] == 0)
    if ref[2] is not None:
        e = got.grad_entropy.double().cpu().numpy()
        assert np.all(np.abs(e - ref[2]) <= 8 * U * np.abs(ref[2]))
    else:
        assert got.grad_entropy is None
    terms = [np.sum(w * A * np.exp(delta)), np.sum(w * (np.exp(r) + r + 1)), np.sum(w * ent), 1.0]
    limits = 4200 * U * np.array([terms[0] + kl * terms[1] + kw.get("entropy_coef", 0.0) * terms[2]]
                                 + terms)
    assert np.all(np.abs(got.stats.double().cpu().numpy() - ref[0]) <= limits)
    return got


KW = dict(kl_coef=0.1, entropy_coef=0.02, clip_low=0.2, clip_high=0.28)


@pytest.mark.parametrize("lengths", [[1], [3], [64] * 8, [5, 0, 9, 0, 0, 1], [2000, 1, 3000, 17], [1] * 300,
                                     [9000], [100, 4000, 0, 0, 12345, 7]])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("per_sequence", [False, True])
def test_lengths(lengths, reduction, per_sequence):
    check(make(lengths, per_sequence=per_sequence, seed=len(lengths)), reduction=reduction, **KW)


@pytest.mark.parametrize("masked", [None, 0.0, 0.9, 1.0])
@pytest.mark.parametrize("ref,entropy", [(False, False), (True, False), (False, True)])
def test_masks_and_parts(masked, ref, entropy):
    x = make([40, 7, 300, 0, 1], masked=masked, ref=ref, entropy=entropy)
    for reduction in ("token", "sequence"):
        got = check(x, reduction=reduction, **KW)
        if masked == 1.0:
            assert torch.equal(got.stats, torch.zeros(5, device=DEV))


def test_rows_outside_every_sequence_do_not_count():
    x = make([30, 0, 50], lead=13, tail=9, masked=None)
    for reduction in ("token", "sequence"):
        got = check(x, reduction=reduction, **KW)
        assert not got.grad_logp[:13].any() and not got.grad_logp[-9:].any()


def test_masked_rows_may_hold_anything():
    x = make([50, 20, 30], masked=0.5)
    ref = run(x, reduction="sequence", **KW)
    for value in (np.nan, np.inf, -np.inf):
        y = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in x.items()}
        for k in ("logp", "old_logp", "ref_logp", "entropy"):
            y[k][~x["mask"]] = value
        got = run(y, reduction="sequence", **KW)
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    # any byte but zero counts
    y = dict(x, mask=x["mask"].astype(np.uint8) * 170)
    for a, b in zip(run(y, reduction="sequence", **KW), ref):
        assert torch.equal(a, b)


def test_a_counted_nan_shows():
    x = make([50, 20, 30], masked=None)
    x["logp"][7] = np.nan
    got = run(x, reduction="token", **KW)
    assert torch.isnan(got.stats[0]) and torch.isnan(got.grad_logp[7])
    assert torch.isfinite(torch.cat([got.grad_logp[:7], got.grad_logp[8:]])).all()


def test_nothing():
    x = make([], masked=None)
    for reduction in ("token", "sequence"):
        got = check(x, reduction=reduction, **KW)
        assert torch.equal(got.stats, torch.zeros(5, device=DEV))
    # rows, but no sequence
    x = make([], masked=None, tail=5)
    got = check(x, reduction="sequence", **KW)
    assert not got.grad_logp.any()


def test_offsets_that_are_not_ascending_do_no_harm():
    """Offsets are device data: nonsense in them gives some weights, never an access elsewhere."""
    x = make([30, 10, 50])
    x["cu_seqlens"] = np.array([-5, 1 << 40, 3, -(1 << 40)], dtype=np.int64)
    for reduction in ("token", "sequence"):
        got = run(x, reduction=reduction, **KW)
        assert got.grad_logp.shape == (90,)
    torch.cuda.synchronize()


def test_limits_of_the_clip():
    """Rows exactly on a limit are not clipped, the next float32 beyond it is."""
    high, low = np.float32(np.log1p(0.28)), np.float32(np.log1p(-0.2))
    delta = np.array([high, np.nextafter(high, np.float32(1)), low, np.nextafter(low, np.float32(-1))] * 2,
                     dtype=np.float32)
    A = np.array([1, 1, 1, 1, -1, -1, -1, -1], dtype=np.float32)
    x = {"logp": delta, "old_logp": np.zeros(8, np.float32), "advantages": A, "mask": None,
         "cu_seqlens": np.array([0, 8]), "ref_logp": None, "entropy": None, "per_sequence": False}
    got = check(x, **KW)
    zero = (got.grad_logp == 0).cpu().numpy()
    assert zero.tolist() == [False, True, False, False, False, False, False, True]
    assert abs(float(got.stats[4]) - 0.25) < 1e-6


def test_gradient_against_differences():
    """Central differences of the loss in float32: a step of 1e-2 leaves ~1e-4 of curvature and
    ~20 u / 1e-2 = 1e-4 of rounding in the quotient, on gradients of up to 0.2."""
    x = make([6, 9], masked=0.2, seed=5)
    got = run(x, reduction="sequence", **KW)
    h = np.float32(1e-2)
    for name, grad in (("logp", got.grad_logp), ("entropy", got.grad_entropy)):
        for t in range(15):
            y = dict(x)
            ends = []
            for s in (h, -h):
                v = x[name].copy()
                v[t] += s
                y[name] = v
                ends.append((float(run(y, reduction="sequence", **KW).stats[0]), float(v[t])))
            slope = (ends[0][0] - ends[1][0]) / (ends[0][1] - ends[1][1])
            d = x["logp"][t] - x["old_logp"][t]
            if name == "logp" and min(abs(d - np.log1p(0.28)), abs(d - np.log1p(-0.2))) < 2e-2:
                continue  # the step crosses the clip
            assert abs(slope - float(grad[t])) < 5e-4


def test_streams_graphs_and_repeats():
    for lengths in ([64] * 8, [3000, 20000, 1, 40000]):
        x = make(lengths)
        dev = {k: torch.from_numpy(v).to(DEV) if isinstance(v, np.ndarray) else v for k, v in x.items()}
        f = lambda **kw: train.policy_loss(**dev, reduction="sequence", **KW, **kw)  # noqa: E731
        ref = f()
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(f(), ref))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = f(stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f()
        for _ in range(3):
            for t in out:
                t.fill_(7)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_refusals():
    z = torch.zeros(8, device=DEV)
    cu = torch.tensor([0, 8], device=DEV)
    with pytest.raises(ValueError, match="cu_seqlens"):
        train.policy_loss(z, z, z, reduction="sequence")
    with pytest.raises(ValueError, match="old_logp"):
        train.policy_loss(z, z[:7], z)
    with pytest.raises(ValueError, match="advantages"):
        train.policy_loss(z, z, z, cu_seqlens=cu, per_sequence=True)
    with pytest.raises(TypeError, match="logp"):
        train.policy_loss(z.half(), z, z)
    with pytest.raises(TypeError, match="mask"):
        train.policy_loss(z, z, z, mask=z)
    with pytest.raises(TypeError, match="cu_seqlens"):
        train.policy_loss(z, z, z, cu_seqlens=cu.int(), reduction="sequence")
    with pytest.raises(ValueError, match="contiguous"):
        train.policy_loss(torch.zeros(16, device=DEV)[::2], z, z)
    with pytest.raises(train.LpError, match="INVALID"):
        train.policy_loss(z, z, z, clip_low=1.5)
