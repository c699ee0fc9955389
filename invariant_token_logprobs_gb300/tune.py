"""The operators of fine-tuning beside those of train.py: ctypes binding of the entry points
declared in include/lp_tune.h.

    out  = layer_norm(residual, branch, weight=..., bias=...)
    grad = layer_norm_backward(grad_normed, grad_residual, out.residual, out.mean, out.rstd, ...)
    loss = preference_loss(logp, cu_seqlens, ref_logp=..., mask=...)
    optimizer = Muon(params, grads, copies=...); optimizer.step()

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
import math
import os
import re
from typing import NamedTuple, Optional, Sequence, Union

import torch

from . import _build_lib, lp
from .lp import LpError
from .train import _disjoint, _dtype_code, _on_one_device, _on_stream, _per_tensor

__all__ = [
    "LayerNorm",
    "LayerNormGrad",
    "MUON_ALIGN",
    "Muon",
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

MUON_ALIGN = 64  # elements that the flat momentum of each matrix is a multiple of

_i64 = ctypes.c_int64
_int = ctypes.c_int
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_f64 = ctypes.c_double


class _MuonTensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("copy", _vp), ("grad", _vp), ("momentum", _vp), ("rows", _i64),
                ("cols", _i64), ("lr_scale", _f32), ("weight_decay", _f32), ("update_scale", _f32),
                ("grad_dtype", _int)]


_tensors = ctypes.POINTER(_MuonTensor)

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
    "lp_muon_plan_size": (_sz, [_tensors, _i64]),
    "lp_muon_plan": (_int, [_tensors, _i64, _vp, _sz]),
    "lp_muon_workspace_size": (_sz, [_vp]),
    "lp_muon_step": (_int, [_vp, _vp, _f64, _f64, _int, _int, _f64, _vp, _sz, _vp]),
}

_lib: Optional[ctypes.CDLL] = None
_calls = None

# what tune_calls.cpp calls, in the order of its table
_BOUND = ("lp_layer_norm", "lp_layer_norm_backward_workspace_size", "lp_layer_norm_backward",
          "lp_preference_loss_workspace_size", "lp_preference_loss", "lp_muon_workspace_size",
          "lp_muon_step")


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


# ------------------------------------------------------------------------- Muon

def _update_scale(scaling: Union[str, float], rows: int, cols: int) -> float:
    """The factor of the learning rate that a matrix's shape gives."""
    if scaling == "spectral":
        return math.sqrt(max(1.0, rows / max(cols, 1)))
    if scaling == "rms":
        return 0.2 * math.sqrt(max(rows, cols))
    if isinstance(scaling, str):
        raise ValueError("scaling must be 'spectral', 'rms' or a number")
    return float(scaling)


class Muon:
    """Muon over a list of matrices: the momentum of each is orthogonalised by Newton-Schulz products
    before it is taken off the parameters, for the matrices of a model's blocks (embeddings, heads and
    vectors go to train.AdamW).

        M = momentum M + g;  u = g + momentum M (nesterov) or M;  X = u / (|u| + eps)
        steps times X = a X + b (X X^T) X + c (X X^T)^2 X;  p = p (1 - lr weight_decay) - lr s X

    params are contiguous float32 matrices, updated in place; grads their gradients (float32 or
    bfloat16), read at every step from the same memory; copies, where given, bfloat16 matrices (or None)
    that receive the updated params.  s is by `scaling` "spectral" sqrt(max(1, rows / cols)), "rms" 0.2
    sqrt(max(rows, cols)), which moves elements as far as AdamW does, or a number.  weight_decay and
    lr_scale, which multiplies lr, are numbers or one for each matrix.  eps is 1e-16 at least.

    The products are of operands of 22 bits, and sums that the tensor core cuts off where float32 rounds:
    X is within 1e-6 of its norm where an update's signs are mixed, as float32 products leave it, and
    within 1e-5 where rows are of one sign (float32 products 2e-6).  An element below 2^-16 of the norm keeps
    an absolute 2^-39 of it.

    `state`, as state_dict() gives it, continues from it with its buffer.  set_grads() names other
    gradient tensors.  A step on any stream keeps its tensors' memory until it is done.  A matrix whose
    update's norm is not finite is left as it was, its momentum too."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], *,
                 copies: Optional[Sequence[Optional[torch.Tensor]]] = None, lr: float = 0.02,
                 momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: Union[float, Sequence[float]] = 0.0,
                 lr_scale: Union[float, Sequence[float]] = 1.0, scaling: Union[str, float] = "spectral",
                 steps: int = 5, eps: float = 1e-7, state: Optional[dict] = None):
        self.params = list(params)
        n = len(self.params)
        if n == 0:
            raise ValueError("no tensors")
        self.copies = [None] * n if copies is None else list(copies)
        if len(self.copies) != n:
            raise ValueError("copies must have one tensor or None for each param")
        for p, c in zip(self.params, self.copies):
            if p.dtype != torch.float32 or not p.is_contiguous() or p.dim() != 2:
                raise TypeError("params must be contiguous float32 matrices")
            if c is not None and (c.dtype != torch.bfloat16 or c.shape != p.shape or
                                  not c.is_contiguous()):
                raise TypeError("copies must be contiguous bfloat16 tensors of the params' shapes")
        self.lr, self.momentum, self.nesterov = float(lr), float(momentum), bool(nesterov)
        self.steps, self.eps = int(steps), float(eps)
        if not 1 <= self.steps <= 32:
            raise ValueError("steps must be 1 to 32")
        self._scales = tuple(_update_scale(scaling, *p.shape) for p in self.params)
        weight_decay = _per_tensor(weight_decay, n, "weight_decay")
        lr_scale = _per_tensor(lr_scale, n, "lr_scale")
        _on_one_device(self.params + [c for c in self.copies if c is not None])
        size = sum(-(-p.numel() // MUON_ALIGN) * MUON_ALIGN for p in self.params)
        if state is None:
            self.momentum_buffer = torch.zeros(size, dtype=torch.float32, device=self.params[0].device)
        else:
            flat = state["momentum"]
            if flat.dtype != torch.float32 or flat.shape != (size,) or not flat.is_contiguous():
                raise ValueError(f"momentum must be a contiguous float32 vector of {size}")
            if flat.data_ptr() % 16 != 0:
                raise ValueError("momentum must be 16-byte aligned")
            _on_one_device([self.params[0], flat])
            self.momentum_buffer = flat
        self._captured: list = []  # plans and gradients of steps that are parts of graphs
        self._lay_out(list(grads), weight_decay, lr_scale)

    def set_grads(self, grads: Sequence[torch.Tensor]) -> None:
        """Lays the plan of the step out for these gradient tensors.  When they are refused the
        optimizer stays as it was.  A step that was captured before goes on reading the gradients
        that it was captured with, which the optimizer keeps."""
        self._lay_out(list(grads), self._weight_decay, self._lr_scale)

    @property
    def weight_decay(self) -> tuple[float, ...]:
        """Each matrix's weight decay; assigned as a number or one for each matrix, it holds from the
        next step on."""
        return self._weight_decay

    @weight_decay.setter
    def weight_decay(self, value: Union[float, Sequence[float]]) -> None:
        self._lay_out(self.grads, _per_tensor(value, len(self.params), "weight_decay"), self._lr_scale)

    @property
    def lr_scale(self) -> tuple[float, ...]:
        """Each matrix's factor of the learning rate, assigned like weight_decay."""
        return self._lr_scale

    @lr_scale.setter
    def lr_scale(self, value: Union[float, Sequence[float]]) -> None:
        self._lay_out(self.grads, self._weight_decay, _per_tensor(value, len(self.params), "lr_scale"))

    def momenta(self) -> list[torch.Tensor]:
        """The momentum of each matrix, in its shape: parts of momentum_buffer."""
        out, at = [], 0
        for p in self.params:
            out.append(self.momentum_buffer[at:at + p.numel()].view(p.shape))
            at += -(-p.numel() // MUON_ALIGN) * MUON_ALIGN
        return out

    def _lay_out(self, grads: list[torch.Tensor], weight_decay: tuple[float, ...],
                 lr_scale: tuple[float, ...]) -> None:
        """Checks these and lays the plan out; nothing is kept of what is refused."""
        if len(grads) != len(self.params):
            raise ValueError("grads must have one tensor for each param")
        copies = [c for c in self.copies if c is not None]
        written = self.params + copies + [self.momentum_buffer]
        _on_one_device(written + grads)
        for p, g in zip(self.params, grads):
            _dtype_code(g, "gradients")
            if g.shape != p.shape or not g.is_contiguous():
                raise ValueError("gradients must be contiguous and of the params' shapes")
        if not _disjoint(written):
            raise ValueError("params, copies and momenta must not share memory")
        if not _disjoint(written, grads):
            raise ValueError("gradients must not share memory with params, copies or momenta")
        lib = load()
        n = len(self.params)
        records = (_MuonTensor * n)(*[
            _MuonTensor(p.data_ptr(), None if c is None else c.data_ptr(), g.data_ptr(), m.data_ptr(),
                        p.shape[0], p.shape[1], s, w, u, _dtype_code(g, "gradients"))
            for p, c, g, m, s, w, u in zip(self.params, self.copies, grads, self.momenta(), lr_scale,
                                           weight_decay, self._scales)])
        size = int(lib.lp_muon_plan_size(records, n))
        host = torch.empty(max(size, 8), dtype=torch.uint8, device="cpu")
        lp._check("lp_muon_plan", lib.lp_muon_plan(records, n, host.data_ptr(), size))
        plan = host.to(self.params[0].device)
        home = torch.cuda.current_stream(plan.device).cuda_stream if plan.is_cuda else 0
        self.grads, self._plan_host, self._plan, self._streams = grads, host, plan, [home]
        self._weight_decay, self._lr_scale = weight_decay, lr_scale
        self._given = (tuple(self.params + copies), tuple(grads))

    def state_dict(self) -> dict:
        """The momenta's buffer (not copied)."""
        return {"momentum": self.momentum_buffer}

    def step(self, lr: Optional[float] = None, stream=None) -> None:
        """One step.  Captured in a graph it is a step at every replay, with the learning rate that it
        was captured with; the optimizer has to outlive the graph."""
        if stream is not None:
            return _on_stream(stream, self.params[0], self.step, lr)
        (_calls or load_calls()).muon_step(
            self._plan_host, self._plan, self.momentum_buffer, self.lr if lr is None else lr, self.momentum,
            self.nesterov, self.steps, self.eps, *self._given, self._streams, self._captured)
