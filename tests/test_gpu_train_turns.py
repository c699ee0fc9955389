"""The training-step operators where a CTA, a team or a warp takes several turns, the last of them
ragged: rings that wrap, sums and roots carried from one turn to the next, rows of a later turn
fetched ahead.  Against the fp64 definitions, with the bounds of the operators' other tests."""

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import train
from oracle import train as ot
from test_gpu_adamw import HYPER
from test_gpu_residual_norm import BF16, F32, check_backward, check_forward, make, split

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def same_alone(x, out, grads, at, a, b, eps):
    """The rows `at` on their own have the bits that they have in the batch."""
    residual, kw = split(x)
    T = residual.shape[0]
    cut = lambda t: t[at] if t.dim() == 2 and t.shape[0] == T else t  # noqa: E731
    k = {n: cut(v) for n, v in kw.items()}
    part = train.residual_norm(cut(residual), residual_scale=a, branch_scale=b, eps=eps, **k)
    for p, whole in zip(part, out):
        assert (p is None and whole is None) or torch.equal(p, whole[at])
    gh, gr = (cut(g) for g in x["grads"])
    g = train.residual_norm_backward(gh, gr, part.residual, part.rstd, branch_rstd=part.branch_rstd,
                                     residual_scale=a, branch_scale=b, **k)
    assert torch.equal(g.residual, grads.residual[at]) and torch.equal(g.branch, grads.branch[at])
    if "gate" in kw and kw["gate"].dim() == 2:
        assert torch.equal(g.gate, grads.gate[at])


@pytest.mark.parametrize("T,d", [
    (2001, 4096),   # one team a CTA: 6 or 7 rows each forward, 13 or 14 backward
    (9001, 264),    # four teams a CTA
    (1003, 6000),   # two groups of columns a thread
    (611, 12288),   # four groups a thread forward; backward row by row, sums in shared memory
])
@pytest.mark.parametrize("residual,act", [(BF16, BF16), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("post,gate", [(True, "token"), (False, None)])
def test_norm(T, d, residual, act, post, gate):
    x = make(T, d, residual, act, BF16, post, gate, seed=11)
    out = check_forward(x, 0.9, 0.5, 1e-6)
    grads = check_backward(x, out, 0.9, 0.5)
    for at in (slice(0, 1), slice(T - 1, T), slice(T // 2, T // 2 + 7)):
        same_alone(x, out, grads, at, 0.9, 0.5, 1e-6)


@pytest.mark.parametrize("T,d,pad,shift", [
    (2003, 2047, 0, 0),  # rows at every place in a word
    (2003, 2047, 3, 1),  # a pitch of whole words, all rows in the middle of one
    (2003, 2048, 2, 0),  # rows of whole words that are not whole groups
    (2003, 2044, 4, 0),  # aligned rows whose last group is not whole
    (4001, 263, 0, 1),   # several teams a CTA
    (801, 5001, 0, 1),   # two groups a thread
])
@pytest.mark.parametrize("residual,act", [(BF16, BF16), (F32, BF16), (F32, F32)])
def test_norm_of_rows_that_are_not_aligned(T, d, pad, shift, residual, act):
    x = make(T, d, residual, act, F32, True, "channel", pad=pad, shift=shift, seed=12)
    out = check_forward(x, 1.0, 0.5, 1e-6)
    grads = check_backward(x, out, 1.0, 0.5)
    for at in (slice(0, 1), slice(T - 1, T), slice(T // 2, T // 2 + 7)):
        same_alone(x, out, grads, at, 1.0, 0.5, 1e-6)


def test_norm_in_place_over_several_turns():
    x = make(2001, 4096, BF16, BF16, BF16, True, "channel", seed=13)
    residual, kw = split(x)
    ref = train.residual_norm(residual, **kw)
    again = residual.clone()
    out = train.residual_norm(again, **kw, in_place=True)
    assert torch.equal(again, ref.residual) and torch.equal(out.normed, ref.normed)


# ------------------------------------------------------------------------ policy loss

def policy_reference(x, reduction, clip_low, clip_high, kl_coef, entropy_coef):
    """oracle.train.policy_loss with arrays in place of its loop, and the magnitudes of its terms:
    (stats, grad_logp, grad_entropy, weights, gradients' terms, stats' terms, |delta| + |r|)."""
    T, cu, B = len(x["logp"]), x["cu_seqlens"], len(x["cu_seqlens"]) - 1
    rows = np.arange(T)
    seq = np.searchsorted(cu[1:], rows, side="right")
    inside = (seq < B) & (rows >= cu[0])
    seq = np.minimum(seq, B - 1)
    keep = np.ones(T, bool) if x["mask"] is None else x["mask"].copy()
    if reduction == "sequence" or x["per_sequence"]:
        keep &= inside
    if reduction == "sequence":
        n = np.bincount(seq[keep], minlength=B)
        w = keep / (np.maximum(n[seq], 1) * max(1, np.count_nonzero(n)))
    else:
        w = keep / max(1, np.count_nonzero(keep))
    A = np.where(keep, x["advantages"][seq] if x["per_sequence"] else x["advantages"], 0).astype(float)
    d32 = np.where(keep, x["logp"] - x["old_logp"], np.float32(0))
    delta = np.where(keep, x["logp"].astype(float) - x["old_logp"], 0.0)
    over = (A > 0) & (d32 > np.float32(np.log1p(clip_high)))
    under = (A < 0) & (d32 < np.float32(np.log1p(-clip_low)))
    ratio = np.exp(delta)
    value = -A * np.where(over, 1 + clip_high, np.where(under, 1 - clip_low, ratio))
    grad = np.where(over | under, 0.0, -A * ratio)
    r = np.where(keep, x["ref_logp"].astype(float) - x["logp"], 0.0)
    ent = np.where(keep, x["entropy"], 0.0).astype(float)
    grad = grad - kl_coef * np.expm1(r)
    stats = [0.0, np.sum(w * value), np.sum(w * (np.expm1(r) - r)), np.sum(w * ent), np.sum(w * (over | under))]
    stats[0] = stats[1] + kl_coef * stats[2] - entropy_coef * stats[3]
    terms = [np.sum(w * np.abs(A) * np.exp(np.abs(delta))), np.sum(w * (np.exp(np.abs(r)) + np.abs(r) + 1)),
             np.sum(w * np.abs(ent)), 1.0]
    mag = w * (np.abs(A) * np.exp(np.abs(delta)) + kl_coef * (np.exp(np.abs(r)) + 1))
    return np.array(stats), w * grad, -entropy_coef * w, w, mag, terms, np.abs(delta) + np.abs(r)


def policy_rows(lengths, per_sequence, masked, seed, lead=0, tail=0):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64) + lead
    T = int(cu[-1]) + tail
    f = lambda v: v.astype(np.float32)  # noqa: E731
    logp = f(-rng.exponential(size=T))
    return {"logp": logp, "old_logp": f(logp + 0.2 * rng.normal(size=T)), "cu_seqlens": cu,
            "advantages": f(rng.normal(size=len(lengths) if per_sequence else T)),
            "mask": rng.random(T) >= masked if masked is not None else None,
            "ref_logp": f(logp + 0.5 * rng.normal(size=T)), "entropy": f(3 * rng.random(T)),
            "per_sequence": per_sequence}


KW = dict(kl_coef=0.1, entropy_coef=0.02, clip_low=0.2, clip_high=0.28)


def check_policy(x, reduction):
    dev = {k: torch.from_numpy(v).to(DEV) if isinstance(v, np.ndarray) else v for k, v in x.items()}
    got = train.policy_loss(**dev, reduction=reduction, **KW)
    stats, g_logp, g_ent, w, mag, terms, far = policy_reference(x, reduction, **KW)
    g, e = got.grad_logp.double().cpu().numpy(), got.grad_entropy.double().cpu().numpy()
    assert np.all(np.abs(g - g_logp) <= (16 + far) * U * mag) and np.all(g[w == 0] == 0)
    assert np.all(np.abs(e - g_ent) <= 8 * U * np.abs(g_ent))
    limits = 4200 * U * np.array([terms[0] + KW["kl_coef"] * terms[1] + KW["entropy_coef"] * terms[2]] + terms)
    assert np.all(np.abs(got.stats.double().cpu().numpy() - stats) <= limits)


def test_policy_reference_is_the_oracle():
    for per_sequence in (False, True):
        x = policy_rows([5, 0, 9, 300, 1], per_sequence, 0.3, 1, lead=3, tail=2)
        for reduction in ("token", "sequence"):
            a = policy_reference(x, reduction, **KW)[:3]
            b = ot.policy_loss(**x, reduction=reduction, **KW)
            for u, v in zip(a, b):
                assert np.allclose(u, v, rtol=1e-12, atol=1e-15)


LENGTHS = {  # of some 1.6 M rows: a CTA of the second pass takes three turns of 1024
    "long": lambda rng: [700_001, 3, 900_000, 5],
    "ragged": lambda rng: rng.integers(1, 8192, 400),
    "short": lambda rng: rng.integers(1, 3, 1_060_000),  # more of a chunk than its shared memory holds
    "empty": lambda rng: rng.integers(1, 900, 9000) * (rng.random(9000) < 0.4),
}


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("per_sequence,masked", [(True, 0.3), (False, 0.9), (True, None)])
def test_policy_loss(lengths, reduction, per_sequence, masked):
    n = LENGTHS[lengths](np.random.default_rng(3))
    check_policy(policy_rows(n, per_sequence, masked, 4, lead=13, tail=9), reduction)


# ------------------------------------------------------------------------ AdamW

def check_codes(x, held, signed):
    """Every held value is one of the two code values around x, by blocks of 256; slack as in the
    other tests of the codes: a relative 2^-20."""
    n = -(-len(x) // 256) * 256
    part = np.abs(np.concatenate([x, np.zeros(n - len(x))]).reshape(-1, 256))
    got = np.abs(np.concatenate([held, np.zeros(n - len(x))]).reshape(-1, 256))
    scale = part.max(axis=1).astype(np.float32).astype(np.float64)
    scale[scale < 2.0 ** -100] = 0.0
    values = ot.moment_values(signed)
    share = np.where(scale[:, None] > 0, part / np.where(scale > 0, scale, 1.0)[:, None], 0.0)
    low = np.searchsorted(values, np.minimum(share * (1 - 2.0 ** -20), 1.0), side="right") - 1
    high = np.searchsorted(values, np.minimum(share * (1 + 2.0 ** -20), 1.0), side="right") - 1
    high = np.minimum(high + 1, len(values) - 1)
    assert np.all(got >= values[low] * scale[:, None] * (1 - 2.0 ** -20))
    assert np.all(got <= values[high] * scale[:, None] * (1 + 2.0 ** -20))
    assert np.all((held == 0) | (np.sign(held) == np.sign(x)))


@pytest.mark.parametrize("grad", [F32, BF16])
def test_adamw_8_bit_whole_rows_a_warp(grad):
    """More than 15 M state elements, where a warp takes a row's blocks in turn: tensors whose last
    blocks and rows are ragged, some that begin off a 16-byte boundary, one of no elements."""
    sizes = [7_000_001, 0, 255, 256, 257, 2047, 2049, 4_194_304, 1_900, 3_000_003, 1, 2_000_000]
    shifts = [0, 0, 1, 0, 2, 3, 0, 0, 1, 1, 0, 2]
    g = torch.Generator(device=DEV).manual_seed(21)

    def one(n, shift, dtype, scale):
        return (torch.randn(n + shift, generator=g, device=DEV) * scale).to(dtype)[shift:]
    params = [one(n, s, F32, 0.1) for n, s in zip(sizes, shifts)]
    grads = [one(n, s, grad, 1e-2) for n, s in zip(sizes, shifts)]
    copies = [one(n, s, BF16, 0.0) if i % 3 else None for i, (n, s) in enumerate(zip(sizes, shifts))]
    opt = train.AdamW(params, grads, copies=copies, **HYPER, weight_decay=0.1, state_bits=8, seed=5)
    assert opt.state_elements > 2048 * 152 * 48
    b1, b2 = HYPER["betas"]
    f = np.float32
    for step in (1, 2):
        m0, v0 = ([h.double().cpu().numpy() for h in opt.views(t)] for t in opt.state_values())
        p0 = [p.double().cpu().numpy() for p in params]
        opt.step()
        m1, v1 = ([h.double().cpu().numpy() for h in opt.views(t)] for t in opt.state_values())
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            gi = grads[i].double().cpu().numpy()
            want, m, v = ot.adamw_step(p0[i], gi, m0[i], v0[i], step, HYPER["lr"], HYPER["betas"],
                                       HYPER["eps"], 0.1)
            mag = np.abs(b1 * m0[i]) + np.abs((1 - b1) * gi)
            change = HYPER["lr"] / (1 - b1 ** step) * mag / (np.sqrt(v / (1 - b2 ** step)) + HYPER["eps"])
            p = params[i].double().cpu().numpy()
            assert np.all(np.abs(p - want) <= 32 * U * change + 4 * U * np.abs(p0[i])), i
            if copies[i] is not None:
                assert torch.equal(copies[i], params[i].to(BF16))
            m32 = (f(b1) * m0[i].astype(f) + f(1 - b1) * gi.astype(f)).astype(np.float64)
            check_codes(m32, m1[i], True)
            check_codes(np.sqrt(v), np.sqrt(v1[i]), False)
        for x in grads:
            x.mul_(-0.7)
