"""Plain fp64 definitions of the training-step operators (test infrastructure).

TEST INFRASTRUCTURE ONLY, as oracle/logprob.py: numpy in float64, sharing nothing
with the CUDA library.  The formulas are those that include/lp_train.h states.
"""

from __future__ import annotations

import numpy as np

__all__ = [
    "residual_norm",
    "residual_norm_backward",
    "policy_loss",
    "adamw_step",
    "moment_values",
    "moment_neighbours",
    "philox_4x32_7",
]


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def residual_norm(residual, branch=None, weight=None, branch_weight=None, gate=None,
                  residual_scale=1.0, branch_scale=1.0, eps=1e-6):
    """(normed, new residual, rstd, branch_rstd); None where a part is absent."""
    new, branch_rstd = _f(residual), None
    if branch is not None:
        n = _f(branch)
        if branch_weight is not None:
            branch_rstd = 1.0 / np.sqrt(np.mean(n * n, axis=1) + eps)
            n = n * branch_rstd[:, None] * _f(branch_weight)
        if gate is not None:
            n = n * _f(gate)
        new = residual_scale * new + branch_scale * n
    if weight is None:
        return None, new, None, branch_rstd
    rstd = 1.0 / np.sqrt(np.mean(new * new, axis=1) + eps)
    return new * rstd[:, None] * _f(weight), new, rstd, branch_rstd


def residual_norm_backward(grad_normed, grad_residual, residual, rstd, branch=None, weight=None,
                           branch_weight=None, branch_rstd=None, gate=None, residual_scale=1.0,
                           branch_scale=1.0):
    """(residual, branch, weight, branch_weight, gate) gradients from the forward's kept values:
    the chain rule through x / rms(x), whose derivative along v is (v - x_hat mean(x_hat v)) / rms."""
    D = 0.0 if grad_residual is None else _f(grad_residual)
    g_weight = g_branch = g_branch_weight = g_gate = None
    if weight is not None:
        x_hat = _f(residual) * _f(rstd)[:, None]
        g_weight = np.sum(_f(grad_normed) * x_hat, axis=0)
        v = _f(grad_normed) * _f(weight)
        D = D + _f(rstd)[:, None] * (v - x_hat * np.mean(x_hat * v, axis=1, keepdims=True))
    if branch is not None:
        y_hat = n = _f(branch)
        if branch_weight is not None:
            y_hat = y_hat * _f(branch_rstd)[:, None]
            n = y_hat * _f(branch_weight)
        g_branch = branch_scale * D
        if gate is not None:
            g_gate = g_branch * n
            if np.ndim(gate) == 1:
                g_gate = g_gate.sum(axis=0)
            g_branch = g_branch * _f(gate)
        if branch_weight is not None:
            g_branch_weight = np.sum(g_branch * y_hat, axis=0)
            v = g_branch * _f(branch_weight)
            g_branch = _f(branch_rstd)[:, None] * (
                v - y_hat * np.mean(y_hat * v, axis=1, keepdims=True))
    return residual_scale * D, g_branch, g_weight, g_branch_weight, g_gate


def policy_loss(logp, old_logp, advantages, mask=None, ref_logp=None, entropy=None,
                cu_seqlens=None, reduction="token", per_sequence=False, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, entropy_coef=0.0):
    """(stats [5], grad_logp, grad_entropy): a loop over the counted rows."""
    T = len(logp)
    sequence = np.full(T, -1)
    if cu_seqlens is not None:
        for i in range(len(cu_seqlens) - 1):
            sequence[cu_seqlens[i]:cu_seqlens[i + 1]] = i
    by_sequence = reduction == "sequence"
    rows = [t for t in range(T) if (mask is None or mask[t])
            and (sequence[t] >= 0 or not (by_sequence or per_sequence))]
    counts = {}
    for t in rows:
        counts[sequence[t]] = counts.get(sequence[t], 0) + 1
    g_logp, g_entropy, stats = np.zeros(T), np.zeros(T), np.zeros(5)
    high, low = np.float32(np.log1p(clip_high)), np.float32(np.log1p(-clip_low))
    for t in rows:
        w = 1.0 / (counts[sequence[t]] * len(counts)) if by_sequence else 1.0 / len(rows)
        A = float(advantages[sequence[t]] if per_sequence else advantages[t])
        # the clip is decided on the float32 difference
        delta32 = np.float32(logp[t]) - np.float32(old_logp[t])
        ratio = np.exp(float(logp[t]) - float(old_logp[t]))
        over, under = A > 0 and delta32 > high, A < 0 and delta32 < low
        value = -A * (1 + clip_high if over else 1 - clip_low if under else ratio)
        grad = 0.0 if over or under else -A * ratio
        kl = 0.0
        if ref_logp is not None:
            r = float(ref_logp[t]) - float(logp[t])
            kl = np.expm1(r) - r
            grad -= kl_coef * np.expm1(r)
        stats += w * np.array([0.0, value, kl, 0.0 if entropy is None else float(entropy[t]),
                               float(over or under)])
        g_logp[t] = w * grad
        g_entropy[t] = -entropy_coef * w
    stats[0] = stats[1] + (kl_coef if ref_logp is not None else 0.0) * stats[2] \
        - (entropy_coef if entropy is not None else 0.0) * stats[3]
    return stats, g_logp, None if entropy is None else g_entropy


def adamw_step(param, grad, m, v, step, lr, betas, eps, weight_decay):
    """(param, m, v) after step number `step` (from 1)."""
    param, grad, m, v = _f(param), _f(grad), _f(m), _f(v)
    b1, b2 = betas
    m = b1 * m + (1 - b1) * grad
    v = b2 * v + (1 - b2) * grad * grad
    root = np.sqrt(v / (1 - b2 ** step)) + eps
    return param * (1 - lr * weight_decay) - lr * (m / (1 - b1 ** step)) / root, m, v


def moment_values(signed):
    """The magnitudes, relative to the block's scale, of all codes of an 8-bit moment: zero,
    then 8 (signed) or 16 equal steps to the octave up to 1 at the last code."""
    steps, top = (8, 127) if signed else (16, 255)
    values = [0.0]
    for c in range(1, top + 1):
        octave, step = divmod(c - top, steps)
        values.append(2.0 ** octave * (1 + step / steps))
    return np.array(values)


def moment_neighbours(x, scale, signed):
    """For each element the two magnitudes (times scale) that enclose |x|, and how far |x| is
    from the lower to the upper one."""
    values = moment_values(signed)
    part = np.minimum(np.abs(_f(x)) / scale, 1.0) if scale > 0 else np.zeros(np.shape(x))
    low = np.searchsorted(values, part, side="right") - 1
    high = np.minimum(low + 1, len(values) - 1)
    gap = np.where(high > low, values[high] - values[low], 1.0)
    return values[low] * scale, values[high] * scale, (part - values[low]) / gap


def philox_4x32_7(counter, key):
    """The four words of Philox 4x32 with 7 rounds (Salmon et al., SC11), in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(7):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c
