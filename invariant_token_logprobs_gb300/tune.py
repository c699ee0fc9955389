"""The operators of fine-tuning beside those of train.py: ctypes binding of the entry points
declared in include/lp_tune.h.

    out  = layer_norm(residual, branch, weight=..., bias=...)
    grad = layer_norm_backward(grad_normed, grad_residual, out.residual, out.mean, out.rstd, ...)

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
    "declared_symbols",
    "layer_norm",
    "layer_norm_backward",
    "layer_norm_backward_workspace_size",
    "load",
    "load_calls",
]

HEADER = os.path.join(os.path.dirname(lp.HEADER), "lp_tune.h")

_i64 = ctypes.c_int64
_int = ctypes.c_int
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_f32 = ctypes.c_float

_SIGNATURES = {
    "lp_layer_norm": (
        _int, [_vp, _i64, _int, _vp, _i64, _int, _vp, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp,
               _i64, _vp, _vp, _vp]),
    "lp_layer_norm_backward_workspace_size": (_sz, [_i64, _i64]),
    "lp_layer_norm_backward": (
        _int, [_vp, _i64, _int, _int, _vp, _int, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp,
               _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
}

_lib: Optional[ctypes.CDLL] = None
_calls = None

# what tune_calls.cpp calls, in the order of its table
_BOUND = ("lp_layer_norm", "lp_layer_norm_backward_workspace_size", "lp_layer_norm_backward")


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
