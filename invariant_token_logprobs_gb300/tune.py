"""The operators of fine-tuning beside those of train.py: ctypes binding of the entry points
declared in include/lp_tune.h.

    out  = layer_norm(residual, branch, weight=..., bias=...)
    grad = layer_norm_backward(grad_normed, grad_residual, out.residual, out.mean, out.rstd, ...)
    loss = preference_loss(logp, cu_seqlens, ref_logp=..., mask=...)

As in train.py this is argument marshalling only: every step of the computation runs in liblp's
kernels on the current stream, there is no fallback, the calls' checks and allocations are compiled
(csrc/tune_calls.cpp, built next to liblp), a call given another stream runs there with its outputs
and workspace allocated for that stream, ordering it after the work that made its inputs is the
caller's, and small outputs of one dtype are parts of one allocation.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import re
from typing import NamedTuple, Optional

import torch

from . import _build_lib, lp
from .lp import LpError
from .train import _on_stream

__all__ = [
    "LayerNorm",
    "LayerNormGrad",
    "PreferenceLoss",
    "declared_symbols",
    "layer_norm",
    "layer_norm_backward",
    "layer_norm_backward_workspace_size",
    "load",
    "load_calls",
    "preference_loss",
    "preference_loss_workspace_size",
]

HEADER = os.path.join(os.path.dirname(lp.HEADER), "lp_tune.h")

_i64 = ctypes.c_int64
_int = ctypes.c_int
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_f64 = ctypes.c_double

_SIGNATURES = {
    "lp_layer_norm": (
        _int, [_vp, _i64, _int, _vp, _i64, _int, _vp, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp,
               _i64, _vp, _vp, _vp]),
    "lp_layer_norm_backward_workspace_size": (_sz, [_i64, _i64]),
    "lp_layer_norm_backward": (
        _int, [_vp, _i64, _int, _int, _vp, _int, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp,
               _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
    "lp_preference_loss_workspace_size": (_sz, [_i64, _i64]),
    "lp_preference_loss": (
        _int, [_vp, _vp, _vp, _vp, _i64, _i64, _int, _int, _int, _f64, _f64, _f64, _f64, _vp, _vp,
               _vp, _vp, _sz, _vp]),
}

_lib: Optional[ctypes.CDLL] = None
_calls = None

# what tune_calls.cpp calls, in the order of its table
_BOUND = ("lp_layer_norm", "lp_layer_norm_backward_workspace_size", "lp_layer_norm_backward",
          "lp_preference_loss_workspace_size", "lp_preference_loss")


def declared_symbols() -> list[str]:
    """Names of the entry points include/lp_tune.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^LP_API\s+[\w\s\*]+?\b(lp_\w+)\s*\(", text, flags=re.M)


def load() -> ctypes.CDLL:
    """lp.load() with the signatures of this module's entry points."""
    global _lib
    if _lib is None:
        lib = lp.load()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def load_calls():
    """The compiled calls, bound to the loaded library's entry points."""
    global _calls
    if _calls is None:
        lib, path = load(), _build_lib.build_calls(quiet=True, module="tune")
        loader = importlib.machinery.ExtensionFileLoader("_tune_calls", path)
        spec = importlib.util.spec_from_file_location("_tune_calls", path, loader=loader)
        calls = importlib.util.module_from_spec(spec)
        loader.exec_module(calls)
        calls.bind(LpError, tuple(ctypes.cast(getattr(lib, f), _vp).value for f in _BOUND))
        _calls = calls
    return _calls


# ------------------------------------------------------------------- layer norm

class LayerNorm(NamedTuple):
    normed: torch.Tensor    # [T, d], the branch's dtype
    residual: torch.Tensor  # [T, d], the new residual stream
    mean: torch.Tensor      # [T] float32
    rstd: torch.Tensor      # [T] float32


class LayerNormGrad(NamedTuple):
    residual: torch.Tensor
    branch: Optional[torch.Tensor]  # None without branch; the residual's own where the dtypes are equal
    weight: Optional[torch.Tensor]  # [d] float32
    bias: Optional[torch.Tensor]    # [d] float32


def layer_norm(residual: torch.Tensor, branch: Optional[torch.Tensor] = None, *,
               weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, in_place: bool = False, stream=None) -> LayerNorm:
    """The residual stream r' = residual + branch and its layer norm
    h = (r' - mean) * rsqrt(variance + eps) * weight + bias.

    residual [T, d] and branch [T, d] are float32 or bfloat16 each; weight and bias [d] share a dtype,
    each may be left out; h comes in the branch's dtype (the residual's without branch).  Without
    branch the residual is normed as it stands.  in_place=True writes r' over the residual."""
    if stream is not None:
        return _on_stream(stream, residual, layer_norm, residual, branch, weight=weight, bias=bias,
                          eps=eps, in_place=in_place)
    return LayerNorm._make((_calls or load_calls()).layer_norm(residual, branch, weight, bias, eps,
                                                               in_place))


def layer_norm_backward_workspace_size(T: int, d: int) -> int:
    return int(load().lp_layer_norm_backward_workspace_size(T, d))


def layer_norm_backward(grad_normed: torch.Tensor, grad_residual: Optional[torch.Tensor],
                        residual: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, *,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        branch: bool = False, weight_grads: bool = True,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> LayerNormGrad:
    """The gradients of layer_norm: grad_normed and grad_residual are those of its normed and residual
    outputs (grad_residual may be None), residual, mean and rstd its outputs, weight and bias its inputs
    (of the bias only that it was there is used).  branch says whether there was one: its gradient is
    the residual's, in grad_normed's dtype, and the very same tensor where the dtypes are equal.
    weight_grads=False leaves out the gradients that are sums over the rows."""
    if stream is not None:
        return _on_stream(stream, residual, layer_norm_backward, grad_normed, grad_residual, residual,
                          mean, rstd, weight=weight, bias=bias, branch=branch,
                          weight_grads=weight_grads, workspace=workspace)
    return LayerNormGrad._make((_calls or load_calls()).layer_norm_backward(
        grad_normed, grad_residual, residual, mean, rstd, weight, bias, branch, weight_grads, workspace))


# -------------------------------------------------------------- preference loss

class PreferenceLoss(NamedTuple):
    stats: torch.Tensor      # [6]: loss, without the nll term, nll, accuracy, chosen's and rejected's reward
    rewards: torch.Tensor    # [n]: beta times each sequence's score
    grad_logp: torch.Tensor  # [T]


_KINDS = {"sigmoid": 0, "hinge": 1, "square": 2}


def preference_loss_workspace_size(T: int, n_sequences: int) -> int:
    return int(load().lp_preference_loss_workspace_size(T, n_sequences))


def preference_loss(logp: torch.Tensor, cu_seqlens: torch.Tensor, *,
                    ref_logp: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                    kind: str = "sigmoid", beta: float = 0.1, margin: float = 0.0,
                    label_smoothing: float = 0.0, average: bool = False, nll_coef: float = 0.0,
                    halves: bool = False, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> PreferenceLoss:
    """The loss of pairs of a chosen and a rejected sequence, from the log-probabilities of their
    tokens, and its gradient with respect to logp.

    cu_seqlens [n + 1] int64 are the row offsets of n sequences; pair i is of the sequences 2 i (chosen)
    and 2 i + 1 (rejected), or with halves=True of i and i + n / 2.  A sequence's score is the sum over
    its counted rows (mask [T], bool or uint8) of logp - ref_logp, or their mean with average=True; a
    pair's z = beta * (the chosen's score - the rejected's) - margin, and its loss by `kind`
    "sigmoid" log(1 + exp(-z)), with label_smoothing e (1 - e) of it and e of log(1 + exp(z));
    "hinge" max(0, 1 - z); "square" ((z - 1/2) / beta)^2.  nll_coef times the chosen's mean of -logp is
    added.  The loss is the mean over the pairs both of whose sequences have a counted row."""
    if stream is not None:
        return _on_stream(stream, logp, preference_loss, logp, cu_seqlens, ref_logp=ref_logp, mask=mask,
                          kind=kind, beta=beta, margin=margin, label_smoothing=label_smoothing,
                          average=average, nll_coef=nll_coef, halves=halves, workspace=workspace)
    if kind not in _KINDS:
        raise ValueError("kind must be 'sigmoid', 'hinge' or 'square'")
    return PreferenceLoss._make((_calls or load_calls()).preference_loss(
        logp, cu_seqlens, ref_logp, mask, _KINDS[kind], average, halves, beta, margin, label_smoothing,
        nll_coef, workspace))
