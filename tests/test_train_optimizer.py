"""train.AdamW on the host: what it keeps, refuses and lays out.  The plan is host work; with the
check of the device taken out these tests run on CPU tensors, and no step is taken."""

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
