"""tune.Muon on the host: what it keeps, refuses and lays out.  The plan is host work; with the check of the
device taken out these tests run on CPU tensors, and no step is taken."""

import pytest
import torch

from invariant_token_logprobs_gb300 import train, tune

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(tune, "_on_one_device", lambda tensors: None)


def matrices(shapes, dtype=F32):
    return [torch.zeros(s, dtype=dtype) for s in shapes]


@pytest.mark.parametrize("default", [BF16, torch.float16, torch.float64, F32])
def test_momenta_are_float32_under_any_default_dtype(on_cpu, default):
    """The kernels take four bytes an element, whatever type torch makes tensors of."""
    shapes = [(256, 256), (5, 7), (0, 3)]
    params, grads, copies = matrices(shapes), matrices(shapes), matrices(shapes, BF16)
    kept = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        opt = tune.Muon(params, grads, copies=copies)
    finally:
        torch.set_default_dtype(kept)
    assert opt.momentum_buffer.dtype == F32
    assert opt.momentum_buffer.untyped_storage().nbytes() == 4 * (256 * 256 + 64)
    views = opt.momenta()
    assert [v.shape for v in views] == [p.shape for p in params] and all(v.dtype == F32 for v in views)
    again = tune.Muon(params, grads, copies=copies, state=opt.state_dict())
    assert again.momentum_buffer is opt.momentum_buffer


@pytest.mark.parametrize("optimizer", [tune.Muon, train.AdamW])
def test_a_plan_is_laid_out_in_host_memory_under_any_default_device(monkeypatch, optimizer):
    """The library writes the plan on the host, wherever torch makes tensors.  (Tensors of "meta" have no memory: a
    plan there is refused, where one on a GPU would be written to from the host.)"""
    for module in (tune, train):
        monkeypatch.setattr(module, "_on_one_device", lambda tensors: None)
    params, grads = matrices([(30, 20)]), matrices([(30, 20)])
    want = optimizer(params, grads)
    torch.set_default_device("meta")
    try:
        opt = optimizer(params, grads, state=want.state_dict())
    finally:
        torch.set_default_device(None)
    assert opt._plan.device.type == "cpu" and opt._plan.shape == want._plan.shape
    assert torch.equal(opt._plan[:56], want._plan[:56])  # AdamW's record of the tensor (what pads it is not set)
