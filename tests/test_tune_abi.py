"""The fine-tuning operators' C ABI without a GPU: exports, argument checks on the host in their order, Muon's
plan, and a C program against include/lp_tune.h.  Valid calls on a machine without a GB300 fail with
LP_ERR_UNSUPPORTED_DEVICE."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from invariant_token_logprobs_gb300 import _build_lib, lp, tune
from test_train_abi import A, INF, INVALID, MISALIGNED, NAN, OK, STEP, UNSUPPORTED, WS_SMALL, Call, addresses

# what a valid call answers here: these tests run none on a GPU
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses stay off the GPU")


@pytest.fixture(scope="module")
def lib():
    return tune.load()


def test_exports_every_declared_symbol(lib):
    names = tune.declared_symbols()
    assert len(names) == 9 and set(names) == set(tune._SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


@no_gpu
def test_layer_norm_arguments(lib):
    a = addresses(8)
    call = Call(lib.lp_layer_norm, residual=a[0], ld_residual=64, residual_dtype=1, branch=a[1], ld_branch=64,
                act_dtype=1, weight=a[2], bias=a[3], weight_dtype=0, T=8, d=64, eps=1e-5, residual_out=a[4],
                ld_residual_out=64, normed=a[5], ld_normed=64, mean=a[6], rstd=a[7], stream=None)
    assert call() == UNSUPPORTED
    assert call(T=0) == OK
    for bad in (dict(T=-1), dict(d=0), dict(d=16385), dict(residual_dtype=2), dict(act_dtype=-1), dict(weight_dtype=7),
                dict(ld_residual=63), dict(ld_branch=63), dict(ld_normed=63), dict(ld_residual_out=63),
                dict(residual=None), dict(residual_out=None), dict(normed=None), dict(eps=-1e-6), dict(eps=NAN),
                dict(eps=INF), dict(branch=None), dict(ld_residual=1 << 60), dict(T=1 << 31)):
        assert call(**bad) == INVALID, bad
    assert call(branch=None, residual_out=None) == UNSUPPORTED
    assert call(weight=None) == call(bias=None) == call(mean=None) == call(rstd=None) == UNSUPPORTED
    # alignment: to the element only
    assert call(residual=A + 2) == UNSUPPORTED
    assert call(residual=A + 1) == MISALIGNED
    assert call(bias=call.args["bias"] + 2) == MISALIGNED
    assert call(mean=call.args["mean"] + 2) == MISALIGNED
    # overlaps: in place is fine, anything else is not
    assert call(residual_out=A) == UNSUPPORTED
    assert call(residual_out=A, ld_residual_out=128) == INVALID
    assert call(normed=call.args["branch"]) == INVALID
    assert call(mean=call.args["rstd"]) == INVALID
    assert call(normed=call.args["residual_out"] + 2 * 63) == INVALID


@no_gpu
def test_layer_norm_backward_arguments(lib):
    a = addresses(11)
    call = Call(lib.lp_layer_norm_backward, residual_out=a[0], ld_residual_out=64, residual_dtype=0, act_dtype=1,
                weight=a[1], weight_dtype=1, T=8, d=64, mean=a[2], rstd=a[3], grad_normed=a[4], ld_grad_normed=64,
                grad_residual_out=a[5], ld_grad_residual_out=64, grad_residual=a[6], ld_grad_residual=64,
                grad_branch=a[7], ld_grad_branch=64, grad_weight=a[8], grad_bias=a[9], workspace=a[10],
                workspace_bytes=tune.layer_norm_backward_workspace_size(8, 64), stream=None)
    assert call() == UNSUPPORTED
    for bad in (dict(T=-1), dict(d=0), dict(d=16385), dict(residual_out=None), dict(mean=None), dict(rstd=None),
                dict(grad_normed=None), dict(grad_residual=None), dict(workspace=None), dict(ld_grad_normed=63),
                dict(ld_grad_residual=1), dict(ld_grad_branch=63), dict(ld_grad_residual_out=2),
                dict(grad_branch=call.args["grad_normed"]), dict(grad_residual=call.args["residual_out"]),
                dict(workspace=call.args["grad_residual"]), dict(grad_weight=call.args["grad_bias"]),
                dict(act_dtype=3)):
        assert call(**bad) == INVALID, bad
    assert call(grad_residual=call.args["grad_residual_out"]) == UNSUPPORTED  # in place
    assert call(grad_residual_out=None) == call(weight=None) == call(grad_branch=None) == UNSUPPORTED
    # without sums no workspace is needed
    assert call(grad_weight=None, grad_bias=None, workspace=None, workspace_bytes=0) == UNSUPPORTED
    assert call(grad_bias=None) == call(grad_weight=None) == UNSUPPORTED
    assert call(T=0, grad_weight=None, grad_bias=None) == OK
    assert call(workspace=call.args["workspace"] + 128) == MISALIGNED
    assert call(grad_weight=call.args["grad_weight"] + 2) == MISALIGNED
    assert call(workspace_bytes=call.args["workspace_bytes"] - 1) == WS_SMALL
    assert tune.layer_norm_backward_workspace_size(-1, 64) == 0
    assert tune.layer_norm_backward_workspace_size(8, 16385) == 0


@no_gpu
@pytest.mark.parametrize("T,n", [(100, 4), (100000, 400)])
def test_preference_loss_arguments(lib, T, n):
    a = addresses(8)
    call = Call(lib.lp_preference_loss, logp=a[0], ref_logp=a[1], mask=a[2], cu_seqlens=a[3], T=T, n_sequences=n,
                kind=0, average=1, halves=0, beta=0.1, margin=0.0, label_smoothing=0.1, nll_coef=0.2, stats=a[4],
                rewards=a[5], grad_logp=a[6], workspace=a[7],
                workspace_bytes=tune.preference_loss_workspace_size(T, n), stream=None)
    assert call() == UNSUPPORTED
    for bad in (dict(T=-1), dict(T=1 << 31), dict(n_sequences=3), dict(n_sequences=-2), dict(kind=3), dict(kind=-1),
                dict(beta=0.0), dict(beta=-1.0), dict(beta=NAN), dict(beta=INF), dict(beta=1e39), dict(beta=1e-39),
                dict(beta=1e38 * 3), dict(margin=NAN), dict(margin=1e39), dict(nll_coef=INF),
                dict(label_smoothing=-0.1), dict(label_smoothing=1.1), dict(label_smoothing=NAN), dict(kind=1),
                dict(kind=2), dict(logp=None), dict(cu_seqlens=None), dict(stats=None), dict(rewards=None),
                dict(grad_logp=None), dict(workspace=None), dict(grad_logp=A), dict(rewards=call.args["stats"] + 20),
                dict(workspace=call.args["logp"])):
        assert call(**bad) == INVALID, bad
    assert call(ref_logp=None) == call(mask=None) == call(average=0, halves=1) == UNSUPPORTED
    assert call(kind=1, label_smoothing=0.0) == call(kind=2, label_smoothing=0.0) == UNSUPPORTED
    assert call(cu_seqlens=call.args["cu_seqlens"] + 4) == MISALIGNED
    assert call(logp=A + 2) == MISALIGNED
    assert call(workspace=call.args["workspace"] + 128) == MISALIGNED
    assert call(workspace_bytes=call.args["workspace_bytes"] - 1) == WS_SMALL
    assert call(T=0, logp=None, grad_logp=None) == UNSUPPORTED  # the stats are written all the same
    assert tune.preference_loss_workspace_size(-1, 2) == 0


def matrix(rows, cols, at=0, **kw):
    v = dict(param=A + at, copy=None, grad=A + STEP + at, momentum=A + 2 * STEP + at, rows=rows, cols=cols, lr_scale=1.0,
             weight_decay=0.0, update_scale=1.0, grad_dtype=0)
    return tune._MuonTensor(*{**v, **kw}.values())


def test_muon_plan(lib):
    def plan(*tensors):
        t = (tune._MuonTensor * len(tensors))(*tensors)
        size = lib.lp_muon_plan_size(t, len(tensors))
        if size == 0:
            return INVALID, None
        host = ctypes.create_string_buffer(size)
        return lib.lp_muon_plan(t, len(tensors), host, size), host

    st, host = plan(matrix(300, 200), matrix(0, 5, STEP), matrix(64, 64, 1 << 19))
    assert st == OK
    # two X and G and P of padded sizes, float16 pairs, and 256 bytes before them at least
    least = (2 * 384 * 256 + 2 * 256 * 256 + 4 * 128 * 128) * 4
    assert least < lib.lp_muon_workspace_size(host) < least + 8192
    st, host = plan(matrix(0, 7))
    assert st == OK and lib.lp_muon_workspace_size(host) == 0
    for bad in (dict(rows=-1), dict(cols=65537), dict(param=None), dict(grad=None), dict(momentum=None),
                dict(lr_scale=-1.0), dict(lr_scale=NAN), dict(weight_decay=INF), dict(update_scale=-0.5),
                dict(grad_dtype=2), dict(grad=A), dict(momentum=A + 4), dict(copy=A + 2 * STEP)):
        assert plan(matrix(**{**dict(rows=64, cols=32), **bad}))[0] == INVALID, bad
    assert plan(matrix(8, 8, param=A + 2))[0] == MISALIGNED
    assert plan(matrix(8, 8, grad_dtype=1, grad=A + STEP + 2))[0] == OK
    t = (tune._MuonTensor * 1)(matrix(64, 64))
    host = ctypes.create_string_buffer(4096)
    assert lib.lp_muon_plan(t, 1, host, 16) == WS_SMALL
    assert lib.lp_muon_plan(t, 1, None, 4096) == INVALID
    assert lib.lp_muon_plan_size(None, 1) == 0 and lib.lp_muon_plan_size(t, -1) == 0
    assert lib.lp_muon_workspace_size(None) == 0
    assert lib.lp_muon_workspace_size(ctypes.create_string_buffer(4096)) == 0


def test_muon_batches_bound_the_workspace(lib):
    """Many matrices go through the workspace in batches."""
    n = 40
    t = (tune._MuonTensor * n)(*[matrix(2048, 2048, i << 27, grad=(A + (i << 27)) + (1 << 25),
                                        momentum=(A + (i << 27)) + (1 << 26)) for i in range(n)])
    size = lib.lp_muon_plan_size(t, n)
    host = ctypes.create_string_buffer(size)
    assert lib.lp_muon_plan(t, n, host, size) == OK
    one = 4 * 2048 * 2048 * 4
    assert 16 * one <= lib.lp_muon_workspace_size(host) < 17 * one


@no_gpu
def test_muon_step_arguments(lib):
    t = (tune._MuonTensor * 1)(matrix(300, 200))
    host = ctypes.create_string_buffer(lib.lp_muon_plan_size(t, 1))
    assert lib.lp_muon_plan(t, 1, host, len(host)) == OK
    call = Call(lib.lp_muon_step, plan_host=host, plan=A, lr=0.02, momentum=0.95, nesterov=1, steps=5, eps=1e-7,
                workspace=A + STEP, workspace_bytes=lib.lp_muon_workspace_size(host), stream=None)
    assert call() == UNSUPPORTED
    for bad in (dict(plan_host=None), dict(plan_host=ctypes.create_string_buffer(4096)), dict(plan=None),
                dict(lr=-1.0), dict(lr=NAN), dict(momentum=1.0), dict(momentum=-0.1), dict(steps=0), dict(steps=33),
                dict(eps=0.0), dict(eps=1e-17), dict(eps=INF), dict(eps=1e39), dict(workspace=None)):
        assert call(**bad) == INVALID, bad
    assert call(plan=A + 128) == MISALIGNED
    assert call(workspace=A + STEP + 128) == MISALIGNED
    assert call(workspace_bytes=call.args["workspace_bytes"] - 1) == WS_SMALL
    empty = (tune._MuonTensor * 1)(matrix(0, 200))
    host = ctypes.create_string_buffer(lib.lp_muon_plan_size(empty, 1))
    assert lib.lp_muon_plan(empty, 1, host, len(host)) == OK
    assert call(plan_host=host, plan=None, workspace=None, workspace_bytes=0) == OK


def test_python_refusals():
    """What the Python layer refuses before the library is called."""
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        tune.layer_norm(cpu, cpu, weight=torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        tune.layer_norm_backward(cpu, None, cpu, torch.zeros(4), torch.zeros(4))
    with pytest.raises(TypeError, match="must be a tensor"):
        tune.layer_norm_backward(None, None, cpu, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA"):
        tune.preference_loss(torch.zeros(4), torch.tensor([0, 2, 4]))
    with pytest.raises(ValueError, match="kind"):
        tune.preference_loss(torch.zeros(4), torch.tensor([0, 2, 4]), kind="mean")
    with pytest.raises(ValueError, match="CUDA"):
        tune.Muon([cpu], [cpu.clone()])
    with pytest.raises(ValueError, match="no tensors"):
        tune.Muon([], [])
    with pytest.raises(ValueError, match="scaling"):
        tune.Muon([cpu], [cpu.clone()], scaling="none")
    with pytest.raises(ValueError, match="CUDA"):
        tune.layer_norm(cpu, stream=0)


PROGRAM = r"""
#include <stdio.h>
#include "lp_tune.h"

int main(void) {
  lp_muon_tensor t = {(float*)(uintptr_t)(1u << 20), NULL, (const void*)(uintptr_t)(1u << 24),
                      (float*)(uintptr_t)(1u << 26), 100, 60, 1.0f, 0.0f, 1.0f, LP_FLOAT32};
  static long long plan[1024];
  if (lp_muon_plan_size(&t, 1) == 0 || lp_muon_plan_size(&t, 1) > sizeof(plan)) return 1;
  if (lp_muon_plan(&t, 1, plan, sizeof(plan)) != LP_OK) return 2;
  if (lp_muon_workspace_size(plan) < 4 * 4 * 128 * 128) return 3;
  if (lp_muon_step(plan, plan, 0.1, 2.0, 1, 5, 1e-7, plan, 0, NULL) != LP_ERR_INVALID_ARGUMENT) return 4;
  if (lp_layer_norm_backward_workspace_size(512, 4096) == 0) return 5;
  if (lp_preference_loss_workspace_size(512, 8) == 0) return 6;
  if (lp_preference_loss(NULL, NULL, NULL, NULL, 0, 1, LP_PREFERENCE_HINGE, 0, 0, 0.1, 0.0, 0.0, 0.0, NULL, NULL,
                         NULL, NULL, 0, NULL) != LP_ERR_INVALID_ARGUMENT) return 7;
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
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-I", include, str(src), "-o", str(exe),
                    "-L", os.path.dirname(path), "-l:" + os.path.basename(path),
                    "-Wl,-rpath," + os.path.dirname(path)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.returncode
