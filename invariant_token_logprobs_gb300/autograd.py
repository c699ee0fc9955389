"""torch.autograd bindings of the fused path, of the logits path and of the
training-step operators.

    logp, entropy = linear_logprob(H, W, y, temperature=1.0)
    logp, entropy = logprob_from_logits(z, y, temperature=1.0)
    logp, entropy = vocab_parallel_linear_logprob(H, W_shard, y, V, group)
    logp, entropy = vocab_parallel_logprob_from_logits(z_shard, y, V, group)
    h, residual   = residual_norm(residual, branch, weight=..., branch_weight=..., gate=...)
    loss, stats   = policy_loss(logp, old_logp, advantages, entropy=entropy, ...)
    h, residual   = layer_norm(residual, branch, weight=..., bias=...)
    loss, stats, rewards = preference_loss(logp, cu_seqlens, ref_logp=..., ...)

The first four return the selected-token log-probabilities and entropies of
z = H W^T / tau (lp_linear_logprob_lse) and back-propagate into H and W through
lp_linear_logprob_backward with the forward's log Z and entropy kept, so the
backward does not recompute them.  The next two are train.residual_norm and
train.policy_loss, on either side of them in a training step, and the last two
tune.layer_norm and tune.preference_loss.  This is argument marshalling only: the
computation runs in liblp's kernels, on the current stream; torch casts
gradients, and scales those that a loss has written by its own.

The vocabulary-parallel forms run on every rank of a torch.distributed group
(1, 2 or 4 ranks, rank r holding shard r of W's rows or of the logits'
columns, see vocab_parallel.shard_of_rank): the forward all-gathers the
shards' quarter states and every rank gets the single-GPU logp and entropy;
the backward gives every rank the single-GPU grad_H (the shards' partial
grad_H all-gathered and merged in a fixed order) and its own rows of grad_W,
or its own columns of dL/dz, with the single-GPU bits.

Gradients come back in the inputs' dtypes: grad_H is the float32 result
rounded to H's dtype; grad_W is asked of the library in bfloat16 when W is
bfloat16 (the float32 result rounded to nearest even, the same bits as
rounding it afterwards) and in float32 otherwise.  An output the loss does not
use contributes nothing (its upstream gradient is passed as absent).  A
gradient of a gradient is refused: the backward kernels have no derivative.
A forward and backward pass can be captured in a CUDA graph as torch's own can:
after a warm-up on a side stream, with no earlier eager graph of the same leaves
still alive (torch ends the process where one is).
"""

from __future__ import annotations

import functools
from typing import Optional

import torch

from . import lp, train, tune
from . import vocab_parallel as vp


class _Refusal(torch.autograd.Function):
    """Gradients as they are, whose own gradient is refused."""

    @staticmethod
    def forward(ctx, *grads):
        # copies: a view could not be scaled in place, as a clip by the norm does
        return tuple(None if g is None else g.clone() for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("a gradient of a gradient was asked for: the library's backward calls "
                           "have no derivative")


def _first_order(backward):
    """A backward whose gradients are no constants of a graph made with create_graph=True: going
    back through them raises.  (torch's once_differentiable refuses only where an upstream gradient
    has a graph, so that the plain sum of an output would still lose its second-order terms.)"""
    @functools.wraps(backward)
    def wrapped(ctx, *upstream):
        with torch.no_grad():
            grads = backward(ctx, *upstream)
        if not torch.is_grad_enabled():
            return grads
        return _Refusal.apply(*[None if g is None else g.detach().requires_grad_() for g in grads])
    return wrapped


class _LinearLogprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, temperature):
        logp, entropy, lse = lp.linear_logprob_lse(H, W, y, temperature)
        ctx.save_for_backward(H, W, y, lse, entropy)
        ctx.temperature = float(temperature)
        ctx.set_materialize_grads(False)
        return logp, entropy

    @staticmethod
    @_first_order
    def backward(ctx, g_logp, g_entropy):
        H, W, y, lse, entropy = ctx.saved_tensors
        need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if (not need_h and not need_w) or (g_logp is None and g_entropy is None):
            return None, None, None, None
        gl = None if g_logp is None else g_logp.float().contiguous()
        ge = None if g_entropy is None else g_entropy.float().contiguous()
        w_dtype = torch.bfloat16 if W.dtype == torch.bfloat16 else torch.float32
        grad_h, grad_w = lp.linear_logprob_backward(
            H, W, y, gl, ge, temperature=ctx.temperature, with_grad_W=need_w,
            saved_lse=lse, saved_entropy=entropy, grad_W_dtype=w_dtype)
        grad_h = grad_h.to(H.dtype) if need_h else None
        grad_w = grad_w.to(W.dtype) if need_w else None
        return grad_h, grad_w, None, None


def linear_logprob(H: torch.Tensor, W: torch.Tensor, y: torch.Tensor,
                   temperature: float = 1.0):
    """(logp [T], entropy [T]) float32 of the fused path, differentiable in H and W
    (bf16 H [T, d] and W [V, d], int64 targets y [T])."""
    return _LinearLogprob.apply(H, W, y, temperature)


class _LogprobFromLogits(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, y, temperature):
        logp, entropy, lse = lp.logprob_from_logits_lse(z, y, temperature)
        ctx.save_for_backward(z, y, lse, entropy)
        ctx.temperature = float(temperature)
        ctx.set_materialize_grads(False)
        return logp, entropy

    @staticmethod
    @_first_order
    def backward(ctx, g_logp, g_entropy):
        z, y, lse, entropy = ctx.saved_tensors
        if not ctx.needs_input_grad[0] or (g_logp is None and g_entropy is None):
            return None, None, None
        gl = None if g_logp is None else g_logp.float().contiguous()
        ge = None if g_entropy is None else g_entropy.float().contiguous()
        grad = lp.logprob_from_logits_backward(z, y, gl, ge, ctx.temperature, saved_lse=lse,
                                               saved_entropy=entropy)
        return grad, None, None


def logprob_from_logits(z: torch.Tensor, y: torch.Tensor, temperature: float = 1.0):
    """(logp [T], entropy [T]) float32 of the logits path, differentiable in the
    float32 logits z [T, V] (rows contiguous; int64 targets y [T]); the backward
    is lp_logprob_from_logits_backward with the forward's log Z and entropy."""
    return _LogprobFromLogits.apply(z, y, temperature)


class _VocabParallelLinearLogprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W_shard, y, vocab_total, group, temperature):
        logp, entropy, lse = vp.vocab_parallel_linear_logprob_lse(H, W_shard, y, vocab_total,
                                                                  group, temperature)
        ctx.save_for_backward(H, W_shard, y, lse, entropy)
        ctx.vocab_total = int(vocab_total)
        ctx.group = group
        ctx.temperature = float(temperature)
        ctx.set_materialize_grads(False)
        return logp, entropy

    @staticmethod
    @_first_order
    def backward(ctx, g_logp, g_entropy):
        H, W_shard, y, lse, entropy = ctx.saved_tensors
        need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        # every rank runs the exchange of the partial grad_H, so the ranks' calls
        # stay matched whatever their own inputs need
        gl = None if g_logp is None else g_logp.float().contiguous()
        ge = None if g_entropy is None else g_entropy.float().contiguous()
        if gl is None and ge is None:
            gl = torch.zeros(H.shape[0], dtype=torch.float32, device=H.device)
        w_dtype = torch.bfloat16 if W_shard.dtype == torch.bfloat16 else torch.float32
        grad_h, grad_w = vp.vocab_parallel_linear_logprob_backward(
            H, W_shard, y, ctx.vocab_total, lse, entropy, gl, ge, ctx.group, ctx.temperature,
            with_grad_W=need_w, grad_W_dtype=w_dtype)
        grad_h = grad_h.to(H.dtype) if need_h else None
        grad_w = grad_w.to(W_shard.dtype) if need_w else None
        return grad_h, grad_w, None, None, None, None


def vocab_parallel_linear_logprob(H: torch.Tensor, W_shard: torch.Tensor, y: torch.Tensor,
                                  vocab_total: int, group=None, temperature: float = 1.0):
    """(logp [T], entropy [T]) of the fused path with W split by rows across the
    ranks of `group`, differentiable in H (every rank gets the whole,
    single-GPU grad_H) and in W_shard (its rows of grad_W); V % 64 == 0 for
    more than one rank."""
    return _VocabParallelLinearLogprob.apply(H, W_shard, y, vocab_total, group, temperature)


class _VocabParallelLogprobFromLogits(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z_shard, y, vocab_total, group, temperature):
        logp, entropy, lse = vp.vocab_parallel_logprob_from_logits_lse(z_shard, y, vocab_total,
                                                                       group, temperature)
        ctx.save_for_backward(z_shard, y, lse, entropy)
        ctx.vocab_total = int(vocab_total)
        ctx.group = group
        ctx.temperature = float(temperature)
        ctx.set_materialize_grads(False)
        return logp, entropy

    @staticmethod
    @_first_order
    def backward(ctx, g_logp, g_entropy):
        z_shard, y, lse, entropy = ctx.saved_tensors
        if not ctx.needs_input_grad[0] or (g_logp is None and g_entropy is None):
            return None, None, None, None, None
        gl = None if g_logp is None else g_logp.float().contiguous()
        ge = None if g_entropy is None else g_entropy.float().contiguous()
        grad = vp.vocab_parallel_logprob_from_logits_backward(
            z_shard, y, ctx.vocab_total, lse, entropy, gl, ge, ctx.group, ctx.temperature)
        return grad, None, None, None, None


def vocab_parallel_logprob_from_logits(z_shard: torch.Tensor, y: torch.Tensor, vocab_total: int,
                                       group=None, temperature: float = 1.0):
    """(logp [T], entropy [T]) from fp32 logits split by columns across the ranks
    of `group`, differentiable in z_shard (its columns of dL/dz; no exchange in
    the backward)."""
    return _VocabParallelLogprobFromLogits.apply(z_shard, y, vocab_total, group, temperature)


def _rows(g):
    """A gradient as rows that the library can read."""
    return g if g is None or (g.stride(1) == 1 and g.stride(0) >= g.shape[1]) else g.contiguous()


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, branch, weight, branch_weight, gate, residual_scale, branch_scale,
                eps):
        out = train.residual_norm(residual, branch, weight=weight, branch_weight=branch_weight,
                                  gate=gate, residual_scale=residual_scale,
                                  branch_scale=branch_scale, eps=eps)
        ctx.save_for_backward(branch, weight, branch_weight, gate, out.residual, out.rstd,
                              out.branch_rstd)
        ctx.scales = float(residual_scale), float(branch_scale)
        ctx.set_materialize_grads(False)
        # without a branch the stream is the input, which is no output of this function
        return out.normed, None if branch is None else out.residual

    @staticmethod
    @_first_order
    def backward(ctx, g_normed, g_residual):
        branch, weight, branch_weight, gate, residual, rstd, branch_rstd = ctx.saved_tensors
        if g_normed is None and g_residual is None:
            return (None,) * 8
        if weight is not None and g_normed is None:
            g_normed = torch.zeros_like(residual if branch is None else branch)
        _, _, need_w, need_bw, need_gate = ctx.needs_input_grad[:5]
        row_gate = gate is not None and gate.dim() == 1
        g = train.residual_norm_backward(
            _rows(g_normed), _rows(g_residual), residual, rstd, branch=branch, weight=weight,
            branch_weight=branch_weight, branch_rstd=branch_rstd, gate=gate,
            residual_scale=ctx.scales[0], branch_scale=ctx.scales[1],
            weight_grads=need_w or need_bw or (need_gate and row_gate))
        cast = lambda t, like: None if t is None else t.to(like.dtype)  # noqa: E731
        return (g.residual, g.branch, cast(g.weight, weight), cast(g.branch_weight, branch_weight),
                cast(g.gate, gate), None, None, None)


def residual_norm(residual: torch.Tensor, branch: Optional[torch.Tensor] = None, *,
                  weight: Optional[torch.Tensor] = None,
                  branch_weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                  branch_scale: float = 1.0, eps: float = 1e-6):
    """(normed, new residual stream) of train.residual_norm, differentiable in the residual, the
    branch, both weights and the gate; the backward is lp_residual_norm_backward with the
    forward's reciprocal roots kept.  Gradients come in the inputs' dtypes (those of the weights
    and of a one-row gate are float32 sums rounded once)."""
    normed, new = _ResidualNorm.apply(residual, branch, weight, branch_weight, gate,
                                      residual_scale, branch_scale, eps)
    return normed, residual if branch is None else new


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, branch, weight, bias, eps):
        out = tune.layer_norm(residual, branch, weight=weight, bias=bias, eps=eps)
        ctx.save_for_backward(weight, bias, out.residual, out.mean, out.rstd)
        ctx.act = None if branch is None else branch.dtype
        ctx.set_materialize_grads(False)
        # without a branch the stream is the input, which is no output of this function
        return out.normed, None if branch is None else out.residual

    @staticmethod
    @_first_order
    def backward(ctx, g_normed, g_residual):
        weight, bias, residual, mean, rstd = ctx.saved_tensors
        if g_normed is None and g_residual is None:
            return (None,) * 5
        if g_normed is None:
            g_normed = torch.zeros_like(residual, dtype=ctx.act or residual.dtype)
        need_w, need_b = ctx.needs_input_grad[2:4]
        g = tune.layer_norm_backward(_rows(g_normed), _rows(g_residual), residual, mean, rstd,
                                     weight=weight, bias=bias, branch=ctx.act is not None,
                                     weight_grads=need_w or need_b)
        cast = lambda t, like: None if t is None else t.to(like.dtype)  # noqa: E731
        return g.residual, g.branch, cast(g.weight, weight), cast(g.bias, bias), None


def layer_norm(residual: torch.Tensor, branch: Optional[torch.Tensor] = None, *,
               weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5):
    """(normed, new residual stream) of tune.layer_norm, differentiable in the residual, the branch,
    the weight and the bias; the backward is lp_layer_norm_backward with the forward's means and
    reciprocal roots kept.  Gradients come in the inputs' dtypes (those of weight and bias are float32
    sums rounded once)."""
    normed, new = _LayerNorm.apply(residual, branch, weight, bias, eps)
    return normed, residual if branch is None else new


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, entropy, old_logp, advantages, kw):
        out = train.policy_loss(logp, old_logp, advantages, entropy=entropy, **kw)
        ctx.save_for_backward(out.grad_logp, out.grad_entropy)
        ctx.mark_non_differentiable(out.stats)
        return out.stats[0].clone(), out.stats

    @staticmethod
    @_first_order
    def backward(ctx, g_loss, _):
        g_logp, g_entropy = ctx.saved_tensors
        need_logp, need_entropy = ctx.needs_input_grad[:2]
        return (g_logp * g_loss if need_logp else None,
                g_entropy * g_loss if need_entropy and g_entropy is not None else None,
                None, None, None)


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                entropy: Optional[torch.Tensor] = None, stream=None, **kw):
    """(loss, stats [5]) of train.policy_loss, the loss a float32 scalar that is differentiable in
    logp and entropy: the gradients are written by the forward call and scaled in the backward.
    Keyword arguments are train.policy_loss's.  With a stream all of the forward runs there, and so
    does its part of the backward, which autograd orders; using the results after the work on that
    stream is the caller's to order, as in train.py."""
    if stream is not None:
        return train._on_stream(stream, logp, policy_loss, logp, old_logp, advantages,
                                entropy=entropy, **kw)
    return _PolicyLoss.apply(logp, entropy, old_logp, advantages, kw)


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, cu_seqlens, kw):
        out = tune.preference_loss(logp, cu_seqlens, **kw)
        ctx.save_for_backward(out.grad_logp)
        ctx.mark_non_differentiable(out.stats, out.rewards)
        return out.stats[0].clone(), out.stats, out.rewards

    @staticmethod
    @_first_order
    def backward(ctx, g_loss, *_):
        return ctx.saved_tensors[0] * g_loss, None, None


def preference_loss(logp: torch.Tensor, cu_seqlens: torch.Tensor, *, stream=None, **kw):
    """(loss, stats [6], rewards [n]) of tune.preference_loss, the loss a float32 scalar that is
    differentiable in logp: the gradient is written by the forward call and scaled in the backward.
    Keyword arguments are tune.preference_loss's; a stream is treated as policy_loss does."""
    if stream is not None:
        return train._on_stream(stream, logp, preference_loss, logp, cu_seqlens, **kw)
    return _PreferenceLoss.apply(logp, cu_seqlens, kw)
