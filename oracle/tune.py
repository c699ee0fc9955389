"""The fine-tuning operators in float64 (numpy): the definitions of include/lp_tune.h.  Test
infrastructure only; shares no code with the GPU path."""

from __future__ import annotations

import numpy as np

# a Newton-Schulz step takes a singular value s to A s + B s^3 + C s^5
A, B, C = 3.4445, -4.7750, 2.0315


def layer_norm(residual, *, branch=None, weight=None, bias=None, eps=1e-5):
    """(normed, new residual stream, mean, rstd)."""
    new = residual if branch is None else residual + branch
    mean = new.mean(axis=1)
    off = new - mean[:, None]
    rstd = 1.0 / np.sqrt((off * off).mean(axis=1) + eps)
    normed = off * rstd[:, None]
    if weight is not None:
        normed = normed * weight
    if bias is not None:
        normed = normed + bias
    return normed, new, mean, rstd


def layer_norm_backward(grad_normed, grad_residual, residual, mean, rstd, *, weight=None):
    """(gradient of the residual and of the branch, of the weight, of the bias)."""
    x = (residual - mean[:, None]) * rstd[:, None]
    dx = grad_normed if weight is None else grad_normed * weight
    D = rstd[:, None] * (dx - dx.mean(axis=1, keepdims=True) - x * (dx * x).mean(axis=1, keepdims=True))
    if grad_residual is not None:
        D = D + grad_residual
    return D, (grad_normed * x).sum(axis=0), grad_normed.sum(axis=0)


def _log1pexp(v):
    """log(1 + exp(v)) without overflow."""
    return np.logaddexp(0.0, v)


def _sigmoid(v):
    return np.exp(-np.logaddexp(0.0, -v))


def preference_loss(logp, cu_seqlens, *, ref_logp=None, mask=None, kind="sigmoid", beta=0.1, margin=0.0,
                    label_smoothing=0.0, average=False, nll_coef=0.0, halves=False):
    """(stats [6], rewards [n], grad_logp [T]): plain loops over the sequences and the pairs."""
    T, n = logp.shape[0], cu_seqlens.shape[0] - 1
    keep = np.ones(T, bool) if mask is None else mask.astype(bool)
    rows = [np.arange(max(cu_seqlens[i], 0), min(cu_seqlens[i + 1], T)) for i in range(n)]
    rows = [r[keep[r]] for r in rows]
    score, likely = np.zeros(n), np.zeros(n)
    with np.errstate(invalid="ignore", over="ignore"):
        for i, r in enumerate(rows):
            likely[i] = logp[r].astype(np.float64).sum()
            score[i] = likely[i] - (0.0 if ref_logp is None else ref_logp[r].astype(np.float64).sum())
            if average and len(r):
                score[i] /= len(r)
        pairs = [(i, i + n // 2) if halves else (2 * i, 2 * i + 1) for i in range(n // 2)]
        pairs = [(c, r) for c, r in pairs if len(rows[c]) and len(rows[r])]
        stats, grad = np.zeros(6), np.zeros(T)
        for c, r in pairs:
            w = 1.0 / len(pairs)
            z = beta * (score[c] - score[r]) - margin
            if kind == "sigmoid":
                loss = slope = 0.0  # a term without a weight is none, however large
                if label_smoothing != 1:
                    loss = (1 - label_smoothing) * _log1pexp(-z)
                    slope = -(1 - label_smoothing) * _sigmoid(-z)
                if label_smoothing:
                    loss, slope = loss + label_smoothing * _log1pexp(z), slope + label_smoothing * _sigmoid(z)
                if z != z:
                    loss = slope = z
            elif kind == "hinge":
                loss, slope = max(0.0, 1.0 - z) if z == z else z, -1.0 if z < 1 else (0.0 if z == z else z)
            else:
                loss, slope = ((z - 0.5) / beta) ** 2, 2 * (z - 0.5) / beta ** 2
            nll = -likely[c] / len(rows[c])
            stats += w * np.array([loss + (nll_coef * nll if nll_coef else 0.0), loss, nll,
                                   float(score[c] > score[r]), beta * score[c], beta * score[r]])
            grad[rows[c]] = w * (slope * beta / (len(rows[c]) if average else 1) - nll_coef / len(rows[c]))
            grad[rows[r]] = -w * slope * beta / (len(rows[r]) if average else 1)
    return stats, beta * score, grad


def newton_schulz(u, steps, eps):
    """The update's approximate orthogonal factor, through its singular values: each step takes s to
    A s + B s^3 + C s^5 after all have been divided by the Frobenius norm plus eps."""
    U, s, Vt = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + eps)
    for _ in range(steps):
        s = s * (A + s * s * (B + C * s * s))
    return (U * s) @ Vt


def muon_scale(rows, cols, scaling):
    """The factor of the learning rate that a matrix's shape gives."""
    return max(1.0, rows / cols) ** 0.5 if scaling == "spectral" else 0.2 * max(rows, cols) ** 0.5


def muon_step(param, grad, momentum_buffer, *, lr, momentum=0.95, nesterov=True, weight_decay=0.0,
              lr_scale=1.0, scaling="spectral", steps=5, eps=1e-7):
    """(param, momentum buffer) after a step."""
    m = momentum * momentum_buffer + grad
    u = grad + momentum * m if nesterov else m
    rate = lr * lr_scale
    x = newton_schulz(u, steps, eps)
    return param * (1 - rate * weight_decay) - rate * muon_scale(*param.shape, scaling) * x, m
