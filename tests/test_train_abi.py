"""The training-step operators' C ABI without a GPU: exports, argument checks on the host in
their order, the optimizer plan, and a C program against include/lp_train.h.  Valid calls on a
machine without a GB300 fail with LP_ERR_UNSUPPORTED_DEVICE."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import _build_lib, lp, train

OK, INVALID, MISALIGNED, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3, 4
A = 1 << 20    # fake, well-aligned device addresses, far apart; never dereferenced
STEP = 1 << 24
NAN, INF = float("nan"), float("inf")
# what a valid call answers here: these tests run none on a GPU
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses stay off the GPU")


@pytest.fixture(scope="module")
def lib():
    return train.load()


def addresses(n):
    return [A + i * STEP for i in range(n)]


def test_exports_every_declared_symbol(lib):
    names = train.declared_symbols()
    assert len(names) == 12 and set(names) == set(train._SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


class Call:
    """A call by argument names, with some of them replaced."""

    def __init__(self, fn, **args):
        self.fn, self.args = fn, args

    def __call__(self, **kw):
        assert set(kw) <= set(self.args), set(kw) - set(self.args)
        return self.fn(*{**self.args, **kw}.values())


def norm_call(lib):
    a = addresses(9)
    return Call(lib.lp_residual_norm, residual=a[0], ld_residual=64, residual_dtype=1, branch=a[1],
                ld_branch=64, gate=a[2], ld_gate=0, act_dtype=1, branch_weight=a[3], weight=a[4],
                weight_dtype=0, T=8, d=64, residual_scale=1.0, branch_scale=1.0, eps=1e-6,
                residual_out=a[5], ld_residual_out=64, normed=a[6], ld_normed=64, branch_rstd=a[7],
                rstd=a[8], stream=None)


@no_gpu
def test_residual_norm_arguments(lib):
    call = norm_call(lib)
    assert call() == UNSUPPORTED
    assert call(T=0) == OK
    for bad in (dict(T=-1), dict(d=0), dict(d=16385), dict(residual_dtype=2), dict(act_dtype=-1),
                dict(weight_dtype=7), dict(ld_residual=63), dict(ld_branch=63), dict(ld_gate=63),
                dict(ld_gate=-64), dict(ld_normed=63), dict(ld_residual_out=63), dict(residual=None),
                dict(residual_out=None), dict(normed=None), dict(eps=-1e-6), dict(eps=NAN),
                dict(eps=INF), dict(residual_scale=NAN), dict(branch_scale=INF),
                dict(weight=None),                       # normed and rstd without weight
                dict(branch_weight=None),                # branch_rstd without branch_weight
                dict(branch=None),                       # gate, branch_weight without branch
                dict(ld_residual=1 << 60)):
        assert call(**bad) == INVALID, bad
    # the optional parts
    assert call(weight=None, normed=None, rstd=None) == UNSUPPORTED
    assert call(branch_weight=None, branch_rstd=None) == UNSUPPORTED
    assert call(gate=None) == UNSUPPORTED
    assert call(ld_gate=64) == UNSUPPORTED
    assert call(rstd=None, branch_rstd=None) == UNSUPPORTED
    bare = dict(branch=None, gate=None, branch_weight=None, branch_rstd=None, residual_out=None)
    assert call(**bare) == UNSUPPORTED
    assert call(**bare, residual_scale=0.5) == INVALID
    assert call(**bare, weight=None, normed=None, rstd=None) == INVALID
    # alignment: to the element only
    assert call(residual=A + 2) == UNSUPPORTED
    assert call(residual=A + 1) == MISALIGNED
    assert call(weight=call.args["weight"] + 2) == MISALIGNED
    assert call(rstd=call.args["rstd"] + 2) == MISALIGNED
    # overlaps: in place is fine, anything else is not
    assert call(residual_out=A) == UNSUPPORTED
    assert call(residual_out=A, ld_residual_out=128) == INVALID
    assert call(residual_out=A + 128) == INVALID
    assert call(normed=call.args["branch"]) == INVALID
    assert call(normed=call.args["residual_out"] + 2 * 63) == INVALID
    # columns of one wide buffer do not overlap
    wide = dict(residual_out=A + 2 * 64, ld_residual_out=128, ld_residual=128)
    assert call(**wide) == UNSUPPORTED
    assert call(**{**wide, "residual_out": A + 2 * 63}) == INVALID


def norm_grad_call(lib):
    a = addresses(15)
    return Call(lib.lp_residual_norm_backward, residual_out=a[0], ld_residual_out=64,
                residual_dtype=0, branch=a[1], ld_branch=64, gate=a[2], ld_gate=0, act_dtype=1,
                branch_weight=a[3], weight=a[4], weight_dtype=1, T=8, d=64, residual_scale=1.0,
                branch_scale=0.5, branch_rstd=a[5], rstd=a[6], grad_normed=a[7], ld_grad_normed=64,
                grad_residual_out=a[8], ld_grad_residual_out=64, grad_residual=a[9],
                ld_grad_residual=64, grad_branch=a[10], ld_grad_branch=64, grad_gate=a[11],
                ld_grad_gate=64, grad_branch_weight=a[12], grad_weight=a[13], workspace=a[14],
                workspace_bytes=train.residual_norm_backward_workspace_size(8, 64), stream=None)


@no_gpu
def test_residual_norm_backward_arguments(lib):
    call = norm_grad_call(lib)
    assert call() == UNSUPPORTED
    for bad in (dict(T=-1), dict(d=0), dict(d=16385), dict(residual_out=None), dict(rstd=None),
                dict(branch_rstd=None), dict(grad_normed=None), dict(grad_residual=None),
                dict(grad_branch=None), dict(workspace=None), dict(branch=None), dict(weight=None),
                dict(gate=None), dict(branch_weight=None), dict(ld_grad_normed=63),
                dict(ld_grad_residual=1), dict(branch_scale=NAN), dict(ld_grad_branch=63),
                dict(grad_branch=call.args["grad_normed"]),
                dict(grad_residual=call.args["residual_out"]),
                dict(workspace=call.args["grad_residual"]),
                dict(grad_weight=call.args["grad_branch_weight"])):
        assert call(**bad) == INVALID, bad
    assert call(grad_residual=call.args["grad_residual_out"]) == UNSUPPORTED  # in place
    assert call(grad_residual_out=None) == UNSUPPORTED
    none = dict(weight=None, rstd=None, residual_out=None, grad_normed=None, grad_weight=None)
    assert call(**none) == UNSUPPORTED
    assert call(**none, grad_residual_out=None) == INVALID
    # without sums no workspace is needed
    sums = dict(grad_weight=None, grad_branch_weight=None, grad_gate=None)
    assert call(**sums, workspace=None, workspace_bytes=0) == UNSUPPORTED
    assert call(workspace=call.args["workspace"] + 128) == MISALIGNED
    assert call(grad_weight=call.args["grad_weight"] + 2) == MISALIGNED
    assert call(workspace_bytes=call.args["workspace_bytes"] - 1) == WS_SMALL
    assert train.residual_norm_backward_workspace_size(-1, 64) == 0
    assert train.residual_norm_backward_workspace_size(8, 16385) == 0


@no_gpu
def test_policy_loss_arguments(lib):
    a = addresses(11)
    call = Call(lib.lp_policy_loss, logp=a[0], old_logp=a[1], ref_logp=a[2], entropy=a[3],
                advantages=a[4], advantages_per_sequence=1, mask=a[5], cu_seqlens=a[6], T=100,
                n_sequences=4, reduction=1, clip_low=0.2, clip_high=0.2, kl_coef=0.1,
                entropy_coef=0.1, stats=a[7], grad_logp=a[8], grad_entropy=a[9], workspace=a[10],
                workspace_bytes=train.policy_loss_workspace_size(100, 4), stream=None)
    assert call() == UNSUPPORTED
    assert call(T=0) == UNSUPPORTED  # the stats are still written
    for bad in (dict(T=-1), dict(n_sequences=-1), dict(reduction=2), dict(clip_low=1.0),
                dict(clip_low=-0.1), dict(clip_low=NAN), dict(clip_high=-0.1), dict(clip_high=INF),
                dict(kl_coef=NAN), dict(entropy_coef=INF), dict(logp=None), dict(old_logp=None),
                dict(advantages=None), dict(cu_seqlens=None), dict(stats=None),
                dict(grad_logp=None), dict(grad_entropy=None), dict(entropy=None),
                dict(workspace=None), dict(grad_logp=a[0]), dict(stats=a[9] + 4)):
        assert call(**bad) == INVALID, bad
    assert call(entropy=None, grad_entropy=None, ref_logp=None, mask=None) == UNSUPPORTED
    assert call(reduction=0, advantages_per_sequence=0, cu_seqlens=None) == UNSUPPORTED
    assert call(mask=a[5] + 1) == UNSUPPORTED
    for p in ("logp", "stats", "grad_logp", "advantages"):
        assert call(**{p: call.args[p] + 2}) == MISALIGNED, p
    assert call(cu_seqlens=a[6] + 4) == MISALIGNED
    assert call(workspace=a[10] + 64) == MISALIGNED
    assert call(workspace_bytes=call.args["workspace_bytes"] - 1) == WS_SMALL


def tensors(*specs):
    """records of (n, copy?, grad dtype)"""
    out = (train._AdamwTensor * max(1, len(specs)))()
    for i, (n, copy, grad) in enumerate(specs):
        a = A + 4 * i * STEP
        out[i] = train._AdamwTensor(a, a + STEP if copy else None, a + 2 * STEP, n, 1.0, 0.1, grad, 0)
    return out


def test_adamw_plan(lib):
    t = tensors((1, True, 0), (0, False, 0), (2048, False, 1), (2049, True, 1))
    assert lib.lp_adamw_state_elements(t, 4) == 2048 * 4
    size = lib.lp_adamw_plan_size(t, 4)
    assert size == 256 + 4 * 4
    plan = np.zeros(size, dtype=np.uint8)
    p = plan.ctypes.data
    assert lib.lp_adamw_plan(t, 4, p, size) == OK
    assert plan[256:].view(np.int32).tolist() == [0, 2, 3, 3]
    assert lib.lp_adamw_plan(t, 4, p, size - 1) == WS_SMALL
    assert lib.lp_adamw_plan(t, 4, None, size) == INVALID
    assert lib.lp_adamw_plan(None, 4, p, size) == INVALID
    assert lib.lp_adamw_state_elements(None, 0) == 0 and lib.lp_adamw_state_elements(t, -1) == -1
    assert lib.lp_adamw_plan_size(t, -1) == 0

    def changed(**kw):
        t = tensors((300, True, 0))
        for k, v in kw.items():
            setattr(t[0], k, v)
        return lib.lp_adamw_plan(t, 1, p, size)

    assert changed() == OK
    for bad in (dict(n=-1), dict(param=None), dict(grad=None), dict(grad_dtype=2), dict(lr_scale=NAN),
                dict(lr_scale=-1.0), dict(weight_decay=INF), dict(weight_decay=-0.1),
                dict(reserved=1), dict(grad=A + 4), dict(copy=A + 1196)):
        assert changed(**bad) == INVALID, bad
    assert changed(param=A + 2) == MISALIGNED and changed(copy=A + STEP + 1) == MISALIGNED
    assert changed(param=A + 4) == OK and changed(copy=None) == OK


@no_gpu
def test_adamw_arguments(lib):
    a = addresses(8)
    call = Call(lib.lp_adamw_step, plan=a[0], n_tensors=3, state_elements=8192, state_bits=8,
                exp_avg=a[1], exp_avg_sq=a[2], exp_avg_scale=a[3], exp_avg_sq_scale=a[4], lr=1e-3,
                beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=0, grad_scale=a[5], stream=None)
    assert call() == UNSUPPORTED
    assert call(state_elements=0) == OK
    for bad in (dict(plan=None), dict(n_tensors=-1), dict(n_tensors=0), dict(state_elements=8191),
                dict(state_elements=-2048), dict(state_bits=16), dict(exp_avg=None),
                dict(exp_avg_sq=None), dict(exp_avg_scale=None), dict(exp_avg_sq_scale=None),
                dict(state_bits=32), dict(lr=-1.0), dict(lr=NAN), dict(beta1=1.0), dict(beta2=-0.1),
                dict(beta2=NAN), dict(eps=0.0), dict(eps=INF), dict(step=0),
                dict(exp_avg_sq=a[1] + 16)):
        assert call(**bad) == INVALID, bad
    assert call(grad_scale=None) == UNSUPPORTED
    assert call(state_bits=32, exp_avg_scale=None, exp_avg_sq_scale=None) == UNSUPPORTED
    assert call(plan=a[0] + 16) == MISALIGNED and call(exp_avg=a[1] + 8) == MISALIGNED
    norm = Call(lib.lp_adamw_grad_norm, plan=a[0], n_tensors=3, state_elements=8192, max_norm=1.0,
                norm_out=a[1], workspace=a[2],
                workspace_bytes=lib.lp_adamw_grad_norm_workspace_size(8192), stream=None)
    assert norm() == UNSUPPORTED
    for bad in (dict(plan=None), dict(max_norm=0.0), dict(max_norm=NAN), dict(norm_out=None),
                dict(workspace=None), dict(state_elements=100)):
        assert norm(**bad) == INVALID, bad
    assert norm(workspace=a[2] + 16) == MISALIGNED
    assert norm(workspace_bytes=norm.args["workspace_bytes"] - 1) == WS_SMALL
    assert lib.lp_adamw_grad_norm_workspace_size(100) == 0
    values = Call(lib.lp_adamw_state_values, m=a[0], u=a[1], ms=a[2], us=a[3], n=2048, mo=a[4],
                  vo=a[5], stream=None)
    assert values() == UNSUPPORTED and values(n=0) == OK
    for bad in (dict(m=None), dict(us=None), dict(mo=None), dict(n=2047), dict(n=-2048),
                dict(vo=a[4]), dict(mo=a[0])):
        assert values(**bad) == INVALID, bad
    assert values(mo=a[4] + 8) == MISALIGNED


def test_python_refusals():
    """What the Python layer refuses before the library is called."""
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        train.residual_norm(cpu, cpu, weight=torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        train.policy_loss(torch.zeros(4), torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA"):
        train.AdamW([torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError, match="no tensors"):
        train.AdamW([], [])
    with pytest.raises(ValueError, match="state_bits"):
        train.AdamW([torch.zeros(4)], [torch.zeros(4)], state_bits=16)
    with pytest.raises(ValueError, match="reduction"):
        train.policy_loss(torch.zeros(4), torch.zeros(4), torch.zeros(4), reduction="mean")


PROGRAM = r"""
#include <stdio.h>
#include "lp_train.h"

int main(void) {
  lp_adamw_tensor t = {(float*)(uintptr_t)(1u << 20), NULL, (const void*)(uintptr_t)(1u << 24), 4097,
                       1.0f, 0.0f, LP_FLOAT32, 0};
  char plan[512];
  if (lp_adamw_state_elements(&t, 1) != 3 * LP_ADAMW_ALIGN) return 1;
  if (lp_adamw_plan_size(&t, 1) > sizeof(plan)) return 2;
  if (lp_adamw_plan(&t, 1, plan, sizeof(plan)) != LP_OK) return 3;
  if (lp_residual_norm_backward_workspace_size(512, 4096) == 0) return 4;
  if (lp_policy_loss_workspace_size(512, 0) == 0) return 5;
  if (lp_adamw_step(plan, 1, 100, 32, plan, plan, NULL, NULL, 0.1, 0.9, 0.9, 1e-8, 1, 0, NULL,
                    NULL) != LP_ERR_INVALID_ARGUMENT) return 6;
  printf("ok\n");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_c_program_against_the_header(tmp_path):
    path = lp.load()._name
    src = tmp_path / "abi.c"
    src.write_text(PROGRAM)
    exe = tmp_path / "abi"
    include = os.path.join(_build_lib.ROOT, "include")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-I", include, str(src),
                    "-o", str(exe), "-L", os.path.dirname(path), "-l:" + os.path.basename(path),
                    "-Wl,-rpath," + os.path.dirname(path)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.returncode
