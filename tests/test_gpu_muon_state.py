"""What Muon's step asks of the buffers that its plan points into, on a GB300."""

import pytest
import torch

from invariant_token_logprobs_gb300 import tune

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_step_refuses_momenta_of_another_type_or_size():
    """The compiled call's own test, before anything is enqueued."""
    shapes = [(70, 90), (5, 7)]
    params = [torch.ones(s, device=DEV) for s in shapes]
    grads = [torch.ones(s, device=DEV) for s in shapes]
    opt = tune.Muon(params, grads, copies=[None, torch.zeros(5, 7, dtype=torch.bfloat16, device=DEV)])
    size = opt.momentum_buffer.numel()
    calls = tune.load_calls()

    def step(momenta):
        calls.muon_step(opt._plan_host, opt._plan, momenta, 0.02, 0.95, True, 5, 1e-7, *opt._given, opt._streams,
                        opt._captured)

    for bad, error in ((torch.zeros(size, device=DEV, dtype=torch.bfloat16), TypeError),
                       (torch.zeros(size, device=DEV, dtype=torch.float64), TypeError),
                       (torch.zeros(size - 64, device=DEV), ValueError), (torch.zeros(size + 1, device=DEV), ValueError),
                       (torch.zeros(2 * size, device=DEV)[::2], ValueError)):
        with pytest.raises(error, match="momenta must be"):
            step(bad)
    assert all((p == 1).all() for p in params) and not opt.momentum_buffer.any()
    step(opt.momentum_buffer)
    assert not any((p == 1).any() for p in params)


def test_a_step_under_another_default_dtype():
    """The same bits as under float32."""
    g = torch.Generator(device=DEV).manual_seed(5)
    params = [torch.randn(256, 200, generator=g, device=DEV), torch.randn(30, 40, generator=g, device=DEV)]
    grads = [torch.randn(p.shape, generator=g, device=DEV) for p in params]
    others = [p.clone() for p in params]
    opt = tune.Muon(params, grads)
    opt.step()
    opt.step()
    kept = torch.get_default_dtype()
    torch.set_default_dtype(torch.bfloat16)
    try:
        same = tune.Muon(others, grads)
        same.step()
        same.step()
    finally:
        torch.set_default_dtype(kept)
    assert torch.equal(opt.momentum_buffer, same.momentum_buffer)
    assert all(torch.equal(a, b) for a, b in zip(params, others))
