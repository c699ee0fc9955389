"""The operators of a training step on either side of the log-probabilities:
ctypes binding of the entry points declared in include/lp_train.h.

    out  = residual_norm(residual, branch, weight=..., branch_weight=..., gate=...)
    grad = residual_norm_backward(grad_normed, grad_residual, out.residual, out.rstd, ...)
    loss = policy_loss(logp, old_logp, advantages, mask=..., cu_seqlens=..., ...)
    optimizer = AdamW(params, grads, copies=..., state_bits=8); optimizer.step(max_norm=1.0)

Argument marshalling only, as in lp.py: every step of the computation runs in
liblp's kernels on the current stream, and there is no fallback.  The calls'
checks and allocations are compiled (csrc/train_calls.cpp, built next to liblp),
since the smallest ones take 3 us on the GPU.  A call given
another stream runs there, its outputs and workspace are allocated for that
stream, and ordering it after the work that made its inputs is the caller's.

Small outputs of one dtype (up to 64 KB each, or 256 KB a call) are parts of one allocation:
any of them keeps its memory, and torch.save writes all of it.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import re
from typing import NamedTuple, Optional, Sequence, Union

import torch

from . import _build_lib, lp
from .lp import LpError

__all__ = [
    "ResidualNorm",
    "ResidualNormGrad",
    "PolicyLoss",
    "AdamW",
    "ADAMW_ALIGN",
    "ADAMW_BLOCK",
    "declared_symbols",
    "load",
    "load_calls",
    "residual_norm",
    "residual_norm_backward",
    "residual_norm_backward_workspace_size",
    "policy_loss",
    "policy_loss_workspace_size",
]

HEADER = os.path.join(os.path.dirname(lp.HEADER), "lp_train.h")

FLOAT32, BFLOAT16 = 0, 1
REDUCE_TOKEN, REDUCE_SEQUENCE = 0, 1
ADAMW_ALIGN = 2048  # LP_ADAMW_ALIGN
ADAMW_BLOCK = 256   # LP_ADAMW_BLOCK

_i64 = ctypes.c_int64
_int = ctypes.c_int
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_f64 = ctypes.c_double


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("copy", _vp), ("grad", _vp), ("n", _i64), ("lr_scale", _f32),
                ("weight_decay", _f32), ("grad_dtype", _int), ("reserved", _int)]


_tensors = ctypes.POINTER(_AdamwTensor)

_SIGNATURES = {
    "lp_residual_norm": (
        _int, [_vp, _i64, _int, _vp, _i64, _vp, _i64, _int, _vp, _vp, _int, _i64, _i64, _f32, _f32,
               _f32, _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    "lp_residual_norm_backward_workspace_size": (_sz, [_i64, _i64]),
    "lp_residual_norm_backward": (
        _int, [_vp, _i64, _int, _vp, _i64, _vp, _i64, _int, _vp, _vp, _int, _i64, _i64, _f32, _f32,
               _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _sz,
               _vp]),
    "lp_policy_loss_workspace_size": (_sz, [_i64, _i64]),
    "lp_policy_loss": (
        _int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _i64, _i64, _int, _f64, _f64, _f64, _f64,
               _vp, _vp, _vp, _vp, _sz, _vp]),
    "lp_adamw_state_elements": (_i64, [_tensors, _i64]),
    "lp_adamw_plan_size": (_sz, [_tensors, _i64]),
    "lp_adamw_plan": (_int, [_tensors, _i64, _vp, _sz]),
    "lp_adamw_grad_norm_workspace_size": (_sz, [_i64]),
    "lp_adamw_grad_norm": (_int, [_vp, _i64, _i64, _f32, _vp, _vp, _sz, _vp]),
    "lp_adamw_step": (
        _int, [_vp, _i64, _i64, _int, _vp, _vp, _vp, _vp, _f64, _f64, _f64, _f64, _i64,
               ctypes.c_uint64, _vp, _vp]),
    "lp_adamw_state_values": (_int, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp]),
}

_lib: Optional[ctypes.CDLL] = None
_calls = None

# what train_calls.cpp calls, in the order of its table
_BOUND = ("lp_residual_norm", "lp_residual_norm_backward_workspace_size",
          "lp_residual_norm_backward", "lp_policy_loss_workspace_size", "lp_policy_loss",
          "lp_adamw_grad_norm_workspace_size", "lp_adamw_grad_norm", "lp_adamw_step",
          "lp_adamw_state_values")


def declared_symbols() -> list[str]:
    """Names of the entry points include/lp_train.h declares."""
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
        lib, path = load(), _build_lib.build_calls(quiet=True)
        loader = importlib.machinery.ExtensionFileLoader("_train_calls", path)
        spec = importlib.util.spec_from_file_location("_train_calls", path, loader=loader)
        calls = importlib.util.module_from_spec(spec)
        loader.exec_module(calls)
        calls.bind(LpError, tuple(ctypes.cast(getattr(lib, f), _vp).value for f in _BOUND))
        _calls = calls
    return _calls


def _dtype_code(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.bfloat16:
        return BFLOAT16
    if t.dtype == torch.float32:
        return FLOAT32
    raise TypeError(f"{what} must be float32 or bfloat16")


def _on_one_device(tensors: Sequence[torch.Tensor]) -> None:
    if not all(t.is_cuda and t.device == tensors[0].device for t in tensors):
        raise ValueError("expected CUDA tensors of one device")


def _on_stream(stream, near, call, *args, **kw):
    """call(*args, **kw) with `stream` (a torch stream, or a handle of the device that the tensor
    `near` is on) as the current one."""
    device = getattr(near, "device", None)
    if device is None or device.type != "cuda":
        raise ValueError("expected CUDA tensors")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError("the stream is one of another device")
    with torch.cuda.stream(stream):
        return call(*args, **kw)


# ---------------------------------------------------------------- residual norm

class ResidualNorm(NamedTuple):
    normed: Optional[torch.Tensor]       # [T, d], the branch's dtype; None without weight
    residual: torch.Tensor               # [T, d], the new residual stream
    rstd: Optional[torch.Tensor]         # [T] float32; None without weight
    branch_rstd: Optional[torch.Tensor]  # [T] float32; None without branch_weight


class ResidualNormGrad(NamedTuple):
    residual: torch.Tensor
    branch: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]         # [d] float32
    branch_weight: Optional[torch.Tensor]  # [d] float32
    gate: Optional[torch.Tensor]           # [T, d] in the gate's dtype, or [d] float32


def residual_norm(residual: torch.Tensor, branch: Optional[torch.Tensor] = None, *,
                  weight: Optional[torch.Tensor] = None,
                  branch_weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                  branch_scale: float = 1.0, eps: float = 1e-6, in_place: bool = False,
                  stream=None) -> ResidualNorm:
    """The residual stream r' = residual_scale * residual + branch_scale * gate * n and its
    norm h = rms_norm(r') * weight, where n = rms_norm(branch) * branch_weight (branch itself
    without branch_weight).

    residual [T, d] and branch [T, d] are float32 or bfloat16 each; gate has the branch's dtype
    and is [T, d] or one row [d]; the weights [d] share a dtype; h comes in the branch's dtype
    (the residual's without branch).  Without branch the residual is normed as it stands.
    in_place=True writes r' over the residual."""
    if stream is not None:
        return _on_stream(stream, residual, residual_norm, residual, branch, weight=weight,
                          branch_weight=branch_weight, gate=gate, residual_scale=residual_scale,
                          branch_scale=branch_scale, eps=eps, in_place=in_place)
    return ResidualNorm._make((_calls or load_calls()).residual_norm(
        residual, branch, weight, branch_weight, gate, residual_scale, branch_scale, eps, in_place))


def residual_norm_backward_workspace_size(T: int, d: int) -> int:
    return int(load().lp_residual_norm_backward_workspace_size(T, d))


def residual_norm_backward(grad_normed: Optional[torch.Tensor],
                           grad_residual: Optional[torch.Tensor], residual: torch.Tensor,
                           rstd: Optional[torch.Tensor], *,
                           branch: Optional[torch.Tensor] = None,
                           weight: Optional[torch.Tensor] = None,
                           branch_weight: Optional[torch.Tensor] = None,
                           branch_rstd: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                           branch_scale: float = 1.0, weight_grads: bool = True,
                           workspace: Optional[torch.Tensor] = None,
                           stream=None) -> ResidualNormGrad:
    """The gradients of residual_norm: grad_normed and grad_residual are those of its normed and
    residual outputs (grad_residual may be None when there is a weight; grad_normed is None
    without weight), residual, rstd and branch_rstd its outputs, the rest its inputs.
    weight_grads=False leaves out the gradients that are sums over the rows (weight,
    branch_weight and a one-row gate)."""
    if stream is not None:
        return _on_stream(stream, residual, residual_norm_backward, grad_normed, grad_residual,
                          residual, rstd, branch=branch, weight=weight, branch_weight=branch_weight,
                          branch_rstd=branch_rstd, gate=gate, residual_scale=residual_scale,
                          branch_scale=branch_scale, weight_grads=weight_grads,
                          workspace=workspace)
    return ResidualNormGrad._make((_calls or load_calls()).residual_norm_backward(
        grad_normed, grad_residual, residual, rstd, branch, weight, branch_weight, branch_rstd, gate,
        residual_scale, branch_scale, weight_grads, workspace))


# ------------------------------------------------------------------ policy loss

class PolicyLoss(NamedTuple):
    stats: torch.Tensor                   # [5]: loss, policy, kl, entropy, clipped share
    grad_logp: torch.Tensor               # [T]
    grad_entropy: Optional[torch.Tensor]  # [T]; None without entropy


def policy_loss_workspace_size(T: int, n_sequences: int) -> int:
    return int(load().lp_policy_loss_workspace_size(T, n_sequences))


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                mask: Optional[torch.Tensor] = None, ref_logp: Optional[torch.Tensor] = None,
                entropy: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                reduction: str = "token", per_sequence: bool = False, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, entropy_coef: float = 0.0,
                workspace: Optional[torch.Tensor] = None, stream=None) -> PolicyLoss:
    """The clipped policy-gradient loss of T rows and its gradients with respect to logp and
    entropy.

    advantages are [T], or one for each sequence with per_sequence=True; mask [T] (bool or
    uint8) says which rows count; cu_seqlens [n + 1] int64 are the sequences' row offsets, needed
    for reduction="sequence" (the mean over sequences of their rows' means; "token" is the mean
    over all counted rows) and for per_sequence.  ref_logp adds kl_coef times the estimate
    exp(r) - r - 1 of the divergence from the reference, entropy subtracts entropy_coef times the
    entropy."""
    if stream is not None:
        return _on_stream(stream, logp, policy_loss, logp, old_logp, advantages, mask=mask,
                          ref_logp=ref_logp, entropy=entropy, cu_seqlens=cu_seqlens,
                          reduction=reduction, per_sequence=per_sequence, clip_low=clip_low,
                          clip_high=clip_high, kl_coef=kl_coef, entropy_coef=entropy_coef,
                          workspace=workspace)
    if reduction not in ("token", "sequence"):
        raise ValueError("reduction must be 'token' or 'sequence'")
    return PolicyLoss._make((_calls or load_calls()).policy_loss(
        logp, old_logp, advantages, mask, ref_logp, entropy, cu_seqlens, reduction == "sequence",
        per_sequence, clip_low, clip_high, kl_coef, entropy_coef, workspace))


# ------------------------------------------------------------------------ AdamW

def _per_tensor(value: Union[float, Sequence[float]], n: int, what: str) -> tuple[float, ...]:
    values = (float(value),) * n if isinstance(value, (int, float)) else tuple(float(v) for v in value)
    if len(values) != n:
        raise ValueError(f"{what} must be a number or one for each tensor")
    return values


def _disjoint(written: Sequence[torch.Tensor], read: Sequence[torch.Tensor] = ()) -> bool:
    """Whether no tensor that is written shares memory with another, written or read."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), kind)
                   for kind, tensors in ((0, written), (1, read)) for t in tensors if t.numel() > 0)
    end = [0, 0]  # of the spans before, by kind
    for start, stop, kind in spans:
        if start < end[0] or (kind == 0 and start < end[1]):
            return False
        end[kind] = max(end[kind], stop)
    return True


_MOMENTS = ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")


class AdamW:
    """AdamW with decoupled weight decay over a list of tensors, one launch a step.

    params are contiguous float32 tensors of any shapes, updated in place; grads their
    gradients (float32 or bfloat16), read at every step from the same memory, such as the main
    gradients that lp.linear_logprob_backward(accumulate_into=...) adds to; copies, where given,
    bfloat16 tensors (or None) that receive the updated params.  weight_decay and lr_scale are
    numbers or one for each tensor.

    state_bits=8 holds the first moment and the root of the second in a byte an element and one
    scale for 256 elements, rounded without bias under `seed`, which leaves the second moment 2 to
    3% high on average; 32 holds both moments in float32.  With 8 bits an element far below its
    block's largest (by 2^16 and more) may lose its root before its first moment and then take one
    step of up to lr * |first moment| / eps: use 32 for tensors that mix such sizes.

    `state`, as state_dict() gives it, continues from it with its buffers, and with its seed where
    none is given.  set_grads() names other gradient tensors.  A step on any stream keeps its
    tensors' memory until it is done, so that they, and the optimizer, may be dropped right after
    it.  eps is 2^-126 at least."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], *,
                 copies: Optional[Sequence[Optional[torch.Tensor]]] = None, lr: float = 1e-3,
                 betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: Union[float, Sequence[float]] = 0.01,
                 lr_scale: Union[float, Sequence[float]] = 1.0, state_bits: int = 32,
                 seed: Optional[int] = None, state: Optional[dict] = None):
        self.params = list(params)
        n = len(self.params)
        if n == 0:
            raise ValueError("no tensors")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.copies = [None] * n if copies is None else list(copies)
        if len(self.copies) != n:
            raise ValueError("copies must have one tensor or None for each param")
        self.lr, self.betas, self.eps = float(lr), (float(betas[0]), float(betas[1])), float(eps)
        self._weight_decay = _per_tensor(weight_decay, n, "weight_decay")
        self._lr_scale = _per_tensor(lr_scale, n, "lr_scale")
        if seed is None:
            seed = 0 if state is None else state.get("seed", 0)
        self.state_bits, self.seed = state_bits, int(seed) & (2**64 - 1)
        for p, c in zip(self.params, self.copies):
            if p.dtype != torch.float32 or not p.is_contiguous():
                raise TypeError("params must be contiguous float32 tensors")
            if c is not None and (c.dtype != torch.bfloat16 or c.shape != p.shape or
                                  not c.is_contiguous()):
                raise TypeError("copies must be contiguous bfloat16 tensors of the params' shapes")
        self._captured: list = []  # plans and gradients of steps that are parts of graphs
        self.set_grads(grads)
        self._allocate(state)

    def set_grads(self, grads: Sequence[torch.Tensor]) -> None:
        """Lays the plan of the step out for these gradient tensors.  When they are refused the
        optimizer stays as it was.  A step that was captured before goes on reading the gradients
        that it was captured with, which the optimizer keeps."""
        self._lay_out(list(grads), self._weight_decay, self._lr_scale)

    @property
    def weight_decay(self) -> tuple[float, ...]:
        """Each tensor's weight decay; assigned as a number or one for each tensor, it holds from
        the next step on."""
        return self._weight_decay

    @weight_decay.setter
    def weight_decay(self, value: Union[float, Sequence[float]]) -> None:
        self._lay_out(self.grads, _per_tensor(value, len(self.params), "weight_decay"), self._lr_scale)

    @property
    def lr_scale(self) -> tuple[float, ...]:
        """Each tensor's factor of the learning rate, assigned like weight_decay."""
        return self._lr_scale

    @lr_scale.setter
    def lr_scale(self, value: Union[float, Sequence[float]]) -> None:
        self._lay_out(self.grads, self._weight_decay, _per_tensor(value, len(self.params), "lr_scale"))

    def _lay_out(self, grads: list[torch.Tensor], weight_decay: tuple[float, ...],
                 lr_scale: tuple[float, ...]) -> None:
        """Checks these and lays the plan out; nothing is kept of what is refused."""
        if len(grads) != len(self.params):
            raise ValueError("grads must have one tensor for each param")
        written = self._written()
        _on_one_device(written + grads)
        for p, g in zip(self.params, grads):
            _dtype_code(g, "gradients")
            if g.shape != p.shape or not g.is_contiguous():
                raise ValueError("gradients must be contiguous and of the params' shapes")
        if not _disjoint(written):
            raise ValueError("params, copies and moments must not share memory")
        lib = load()
        n = len(self.params)
        records = (_AdamwTensor * n)(*[
            _AdamwTensor(p.data_ptr(), None if c is None else c.data_ptr(), g.data_ptr(), p.numel(), s, w,
                         _dtype_code(g, "gradients"), 0)
            for p, c, g, s, w in zip(self.params, self.copies, grads, lr_scale, weight_decay)])
        elements = int(lib.lp_adamw_state_elements(records, n))
        size = int(lib.lp_adamw_plan_size(records, n))
        host = torch.empty(max(size, 1), dtype=torch.uint8)
        lp._check("lp_adamw_plan", lib.lp_adamw_plan(records, n, host.data_ptr(), size))
        if not _disjoint(written, grads):
            raise ValueError("gradients must not share memory with params, copies or moments")
        plan = host.to(self.params[0].device)
        home = torch.cuda.current_stream(plan.device).cuda_stream if plan.is_cuda else 0
        self.grads, self.state_elements, self._plan, self._streams = grads, elements, plan, [home]
        self._weight_decay, self._lr_scale = weight_decay, lr_scale
        self._given = (tuple(self.params + [c for c in self.copies if c is not None]), tuple(grads))

    def _allocate(self, state: Optional[dict]) -> None:
        n, device = self.state_elements, self.params[0].device
        small = self.state_bits == 8
        kind = torch.uint8 if small else torch.float32
        self.step_count = 0 if state is None else int(state["step"])
        wanted = {"exp_avg": (n, kind), "exp_avg_sq": (n, kind)}
        if small:
            wanted["exp_avg_scale"] = wanted["exp_avg_sq_scale"] = (n // ADAMW_BLOCK, torch.float32)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        for name, (count, dtype) in wanted.items():
            if state is None:
                t = torch.zeros(count, dtype=dtype, device=device)
            else:
                t = state[name]
                if t.dtype != dtype or t.shape != (count,) or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} vector of {count}")
                _on_one_device([self.params[0], t])
            setattr(self, name, t)
        if not _disjoint(self._written(), self.grads):
            raise ValueError("moments must not share memory with params, copies or gradients")

    def _written(self) -> list[torch.Tensor]:
        """What a step writes: params, copies and, once they are there, the moments."""
        moments = [getattr(self, name, None) for name in _MOMENTS]
        return self.params + [t for t in self.copies + moments if t is not None]

    def state_dict(self) -> dict:
        """The step count, the seed and the moments' buffers (not copied)."""
        return {"step": self.step_count, "seed": self.seed, "exp_avg": self.exp_avg,
                "exp_avg_sq": self.exp_avg_sq, "exp_avg_scale": self.exp_avg_scale,
                "exp_avg_sq_scale": self.exp_avg_sq_scale}

    def step(self, lr: Optional[float] = None, max_norm: Optional[float] = None,
             stream=None) -> Optional[torch.Tensor]:
        """One step.  With max_norm the gradients are scaled by min(1, max_norm / (norm + 1e-6))
        of their global 2-norm, which is returned as a float32 scalar on the device; a norm that
        is not finite leaves every param and moment as it was (the step is counted).

        A step that is captured in a graph repeats itself at every replay: its number, learning
        rate and random bits are part of it, and nothing is counted.  The optimizer has to outlive
        the graph."""
        if stream is not None:
            return _on_stream(stream, self.params[0], self.step, lr, max_norm)
        norm = (_calls or load_calls()).adamw_step(
            self._plan, len(self.params), self.state_elements, self.state_bits, self.exp_avg,
            self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale, self.lr if lr is None else lr,
            self.betas[0], self.betas[1], self.eps, self.step_count + 1, self.seed, max_norm,
            *self._given, self._streams, self._captured)
        self.step_count += 1
        return norm

    def state_values(self, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """(first moment, second moment) as flat float32: the buffers themselves for 32-bit
        moments, what the bytes stand for for 8-bit ones.  views() cuts them by tensor."""
        if self.state_bits == 32:
            return self.exp_avg, self.exp_avg_sq
        if stream is not None:
            return _on_stream(stream, self.exp_avg, self.state_values)
        return (_calls or load_calls()).adamw_state_values(
            self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale)

    def views(self, flat: torch.Tensor) -> list[torch.Tensor]:
        """The part of a flat moment buffer that belongs to each param, in its shape."""
        out, at = [], 0
        for p in self.params:
            out.append(flat[at:at + p.numel()].view(p.shape))
            at += -(-p.numel() // ADAMW_ALIGN) * ADAMW_ALIGN
        return out
