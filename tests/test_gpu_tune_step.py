"""The fine-tuning operators together on a GB300, as a training step uses them: the example, its gradients against
autograd's through plain float32 operations and through the bindings, and a whole step captured in a graph."""

import importlib.util
import math
import os

import pytest
import torch

from invariant_token_logprobs_gb300 import autograd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_preference.py")
    spec = importlib.util.spec_from_file_location("train_preference", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_runs(example):
    stats = example.run(steps=3, pairs=9, hidden=192, vocab=4096, log=None)
    assert len(stats) == 6 and all(math.isfinite(v) for v in stats) and 0 <= stats[3] <= 1


def test_example_steps_repeat(example):
    """The same batches give the same weights, bit for bit, and the copies follow the masters."""
    models = [example.Model(256, 4096, DEV) for _ in range(2)]
    for model in models:
        for step in range(3):
            example.train_step(model, example.pairs_of(model, 12, seed=step))
    for k in models[0].master:
        assert torch.equal(models[0].master[k], models[1].master[k])
        assert torch.equal(models[0].weight[k], models[0].master[k].to(BF16))


def plain_loss(w, batch, beta):
    """The example's loss in float32 torch operations."""
    x = batch["hidden"].float()
    r = x + x @ w["projection"].t()
    off = r - r.mean(1, keepdim=True)
    h = off * torch.rsqrt((off * off).mean(1, keepdim=True) + 1e-5) * w["norm"] + w["norm_bias"]
    z = h @ w["head"].t()
    logp = (z - torch.logsumexp(z, 1, keepdim=True)).gather(1, batch["tokens"].clamp_min(0)[:, None])[:, 0]
    keep = batch["mask"].float()
    cu = batch["cu_seqlens"]
    n = cu.numel() - 1
    sequence = torch.repeat_interleave(torch.arange(n, device=DEV), cu[1:] - cu[:-1])
    fold = lambda v: torch.zeros(n, device=DEV).index_add(0, sequence, v)  # noqa: E731
    score = fold(torch.where(batch["mask"], logp - batch["ref_logp"], torch.zeros_like(logp)))
    gap = beta * (score[0::2] - score[1::2])
    nll = -(fold(logp * keep) / fold(keep))[0::2]
    ln = torch.nn.functional.logsigmoid
    return (-0.95 * ln(gap) - 0.05 * ln(-gap) + 0.1 * nll).mean()


def test_gradients_of_a_step(example):
    """Along the step six tensors are rounded to bfloat16 (the projection's output, the stream, its norm, two
    gradients of them, and the products' operands), each by 2^-9 of it in the mean at most; three times their sum,
    since an error in the norm's gradient meets the head's: 2^-5 in the Frobenius norm."""
    model = example.Model(192, 4096, DEV)
    other = example.Model(192, 4096, DEV, seed=3)
    batch = example.pairs_of(other, 16, seed=7)
    stats = example.gradients(model, batch)
    w = {k: v.float().requires_grad_() for k, v in model.weight.items()}
    loss = plain_loss(w, batch, 0.1)
    loss.backward()
    want = float(loss.detach())
    assert abs(float(stats[0]) - want) <= 2 ** -5 * abs(want)
    for k in w:
        err = torch.linalg.vector_norm(model.grad[k] - w[k].grad) / torch.linalg.vector_norm(w[k].grad)
        assert err <= 2 ** -5, (k, float(err))


def test_the_bindings_give_the_same_step(example):
    """The same step through autograd: the head's gradient is the same call's, the others come by the same kernels."""
    model = example.Model(192, 4096, DEV)
    batch = example.pairs_of(example.Model(192, 4096, DEV, seed=3), 16, seed=7)
    stats = example.gradients(model, batch)
    w = {k: v.clone().requires_grad_() for k, v in model.weight.items()}
    branch = batch["hidden"] @ w["projection"].t()
    h, _ = autograd.layer_norm(batch["hidden"], branch, weight=w["norm"], bias=w["norm_bias"])
    logp, _ = autograd.linear_logprob(h, w["head"], batch["tokens"])
    loss, again, _ = autograd.preference_loss(logp, batch["cu_seqlens"], ref_logp=batch["ref_logp"],
                                              mask=batch["mask"], beta=0.1, label_smoothing=0.05, nll_coef=0.1)
    loss.backward()
    assert torch.equal(again, stats)
    for k in w:
        assert torch.equal(w[k].grad, model.grad[k].to(BF16)), k


def test_a_step_in_a_graph(example):
    """Captured once and replayed: the weights of as many eager steps on the same batch."""
    eager, captured = example.Model(256, 4096, DEV), example.Model(256, 4096, DEV)
    batch = example.pairs_of(eager, 10, seed=1)
    # AdamW's step number is part of a captured step, so the matrices' optimizer is the one that goes on
    for _ in range(3):
        example.gradients(eager, batch)
        eager.muon.step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        example.gradients(captured, batch)  # what torch's products allocate once
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        example.gradients(captured, batch)
        captured.muon.step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k in eager.master:
        assert torch.equal(eager.master[k], captured.master[k]), k
    assert torch.equal(eager.muon.momentum_buffer, captured.muon.momentum_buffer)


def test_the_bindings_in_a_graph(example):
    """Forward and backward through autograd captured together; replays see the inputs of the time."""
    batch = example.pairs_of(example.Model(192, 4096, DEV, seed=3), 16, seed=7)
    model = example.Model(192, 4096, DEV)
    leaves = {k: v.clone().requires_grad_() for k, v in model.weight.items() if k != "projection"}
    hidden = batch["hidden"].clone().requires_grad_()
    leaves["hidden"] = hidden

    def loss_of():
        h, _ = autograd.layer_norm(hidden, weight=leaves["norm"], bias=leaves["norm_bias"])
        logp, _ = autograd.linear_logprob(h, leaves["head"], batch["tokens"])
        loss, stats, rewards = autograd.preference_loss(logp, batch["cu_seqlens"], ref_logp=batch["ref_logp"],
                                                        mask=batch["mask"], beta=0.1)
        loss.backward()
        return stats, rewards

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss_of()
    torch.cuda.current_stream().wait_stream(side)
    for v in leaves.values():
        v.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stats, rewards = loss_of()
    with torch.no_grad():
        hidden.copy_(batch["hidden"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    got = {k: v.grad.clone() for k, v in leaves.items()}
    kept = stats.clone(), rewards.clone()
    for v in leaves.values():
        v.grad = None
    again = loss_of()
    assert torch.equal(kept[0], again[0]) and torch.equal(kept[1], again[1])
    for k, v in leaves.items():
        assert torch.equal(got[k], v.grad), k
