"""train.AdamW on the host: what it keeps, refuses and lays out.  The plan is host work; with the
check of the device taken out these tests run on CPU tensors, and no step is taken."""

import struct

import pytest
import torch

from invariant_token_logprobs_gb300 import train


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(train, "_on_one_device", lambda tensors: None)


def test_refused_gradients_leave_the_optimizer_as_it_was(on_cpu):
    """The plan holds the addresses of the gradients that the optimizer keeps alive."""
    p, g = torch.zeros(300), torch.zeros(300)
    opt = train.AdamW([p], [g])
    plan, elements = opt._plan, opt.state_elements
    for bad, error in (([torch.zeros(299)], ValueError), ([torch.zeros(300).half()], TypeError),
                       ([g, g], ValueError), ([torch.zeros(600)[::2]], ValueError), ([p], train.LpError)):
        with pytest.raises(error):
            opt.set_grads(bad)
        assert len(opt.grads) == 1 and opt.grads[0] is g
        assert opt._plan is plan and opt.state_elements == elements
    other = torch.ones(300)
    opt.set_grads([other])
    assert opt.grads[0] is other and not torch.equal(opt._plan, plan)


def test_gradients_in_the_memory_of_other_params_are_refused(on_cpu):
    """A step takes its tensors in any order, so no gradient may lie in what it writes."""
    flat = torch.zeros(1200)
    p, g = [flat[:300], flat[300:600]], [flat[600:900], flat[900:]]
    opt = train.AdamW(p, g)
    copy = torch.zeros(300, dtype=torch.bfloat16)
    for bad in ([g[0], p[0]], [p[1], g[1]], [flat[450:750], g[1]], [g[0], flat[299:599]]):
        with pytest.raises((ValueError, train.LpError), match="share memory|INVALID"):
            opt.set_grads(bad)
    with pytest.raises(ValueError, match="share memory"):
        train.AdamW(p, [g[0], copy], copies=[copy, None])
    # one gradient of two params, and gradients that touch params without sharing a byte, are fine
    opt.set_grads([g[0], g[0]])
    opt.set_grads([flat[600:900], flat[600:900]])
    train.AdamW([torch.zeros(0), flat[:300]], [torch.zeros(0), g[0]])


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_in_other_memory_of_the_step_are_refused(on_cpu, bits):
    p, g = torch.zeros(4096), torch.zeros(4096)
    kept = train.AdamW([p], [g], state_bits=bits).state_dict()
    for name, spoiled in (("exp_avg", p), ("exp_avg_sq", g), ("exp_avg", kept["exp_avg_sq"])):
        bad = spoiled if bits == 32 or spoiled.dtype == torch.uint8 else spoiled.view(torch.uint8)[:4096]
        with pytest.raises(ValueError, match="share memory"):
            train.AdamW([p], [g], state_bits=bits, state={**kept, name: bad})
    opt = train.AdamW([p], [g], state_bits=bits, state=kept)
    if bits == 32:
        with pytest.raises(ValueError, match="share memory"):
            opt.set_grads([opt.exp_avg])


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses stay off the GPU")
def test_an_eps_that_the_step_would_read_as_zero_is_refused():
    """With both moments zero the step divides by eps: one that is zero or subnormal in float32
    made every such element NaN."""
    a = [(1 << 20) + (i << 24) for i in range(5)]

    def status(eps):
        return train.load().lp_adamw_step(a[0], 1, 2048, 32, a[1], a[2], None, None, 1e-3, 0.9, 0.99,
                                          eps, 1, 0, None, None)
    invalid, unsupported = 1, 3  # the latter is what a valid call answers without a GPU
    for eps in (0.0, -1e-8, 1e-300, 1e-46, 1e-40, 1.17e-38, float("nan"), float("inf")):
        assert status(eps) == invalid, eps
    for eps in (2.0 ** -126, 1.2e-38, 1e-30, 1e-8, 1.0):
        assert status(eps) == unsupported, eps


def test_a_state_brings_its_seed(on_cpu):
    """The rounding of 8-bit moments goes on as it would have."""
    p, g = torch.zeros(300), torch.zeros(300)
    state = train.AdamW([p], [g], state_bits=8, seed=77).state_dict()
    assert train.AdamW([p], [g], state_bits=8, state=state).seed == 77
    assert train.AdamW([p], [g], state_bits=8, state=state, seed=0).seed == 0
    del state["seed"]
    assert train.AdamW([p], [g], state_bits=8, state=state).seed == 0
    assert train.AdamW([p], [g], state_bits=8).seed == 0
    assert train.AdamW([p], [g], state_bits=8, seed=-1).seed == 2 ** 64 - 1


def test_factors_hold_when_they_are_assigned(on_cpu):
    """The factors of each tensor are part of the plan: assigning them lays it out again."""
    def planned(opt):  # (lr_scale, weight_decay) of each record of 56 bytes
        return [struct.unpack_from("ff", bytes(opt._plan.tolist()), 56 * i + 40) for i in range(2)]
    params, grads = [torch.zeros(300), torch.zeros(9)], [torch.zeros(300), torch.zeros(9)]
    opt = train.AdamW(params, grads, weight_decay=0.5)
    assert planned(opt) == [(1.0, 0.5)] * 2 and opt.weight_decay == (0.5, 0.5)
    opt.weight_decay = [0.25, 0]
    opt.lr_scale = 2
    assert planned(opt) == [(2.0, 0.25), (2.0, 0.0)] and opt.lr_scale == (2.0, 2.0)
    for name, bad in (("weight_decay", [0.1]), ("weight_decay", -1.0), ("lr_scale", float("nan"))):
        with pytest.raises((ValueError, train.LpError)):
            setattr(opt, name, bad)
    assert planned(opt) == [(2.0, 0.25), (2.0, 0.0)] and opt.weight_decay == (0.25, 0.0)
    with pytest.raises(TypeError):
        opt.weight_decay[0] = 0.5  # would change nothing
    opt.set_grads([torch.ones(300), grads[1]])
    assert planned(opt) == [(2.0, 0.25), (2.0, 0.0)]
