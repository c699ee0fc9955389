"""Which stream a call given one by the caller runs on: host logic, with torch's streams replaced."""

import contextlib

import pytest
import torch

from invariant_token_logprobs_gb300 import train


class Stream:
    def __init__(self, handle, device=None):
        # without a device torch takes the current one
        self.handle, self.device = handle, torch.device("cuda", 0) if device is None else device


class Tensor:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.fixture
def entered(monkeypatch):
    streams = []

    @contextlib.contextmanager
    def stream(s):
        streams.append(s)
        yield
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return streams


def calls(near, stream):
    """Every call that takes a stream, of a tensor `near`."""
    opt = object.__new__(train.AdamW)
    opt.params, opt.exp_avg, opt.state_bits = [near], near, 8
    return [lambda: train.residual_norm(near, stream=stream),
            lambda: train.residual_norm_backward(None, None, near, None, stream=stream),
            lambda: train.policy_loss(near, near, near, stream=stream),
            lambda: opt.step(stream=stream), lambda: opt.state_values(stream=stream)]


def stop(*args):
    raise KeyError("called")


@pytest.mark.parametrize("index", [0, 1])
def test_a_handle_is_a_stream_of_the_tensors_device(monkeypatch, entered, index):
    monkeypatch.setattr(train, "_calls", type("Calls", (), {k: staticmethod(stop) for k in (
        "residual_norm", "residual_norm_backward", "policy_loss", "adamw_step", "adamw_state_values")}))
    for i, call in enumerate(calls(Tensor(index), 77)):
        with pytest.raises((KeyError, AttributeError)):
            call()
        assert len(entered) == i + 1
        assert entered[-1].handle == 77 and entered[-1].device == torch.device("cuda", index)


def test_a_stream_of_another_device_is_refused(entered):
    for call in calls(Tensor(1), Stream(77, torch.device("cuda", 0))):
        with pytest.raises(ValueError, match="another device"):
            call()
    assert not entered


def test_tensors_of_the_host_are_refused(entered):
    cpu = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        train.residual_norm(cpu, weight=torch.ones(8), stream=77)
    assert not entered
