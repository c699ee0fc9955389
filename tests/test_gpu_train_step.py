"""The training-step operators together on a GB300: the example's training, the autograd bindings
against direct calls, and a whole step captured in a graph."""

import importlib.util
import os

import pytest
import torch

from invariant_token_logprobs_gb300 import autograd, lp, train

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_head.py")
    spec = importlib.util.spec_from_file_location("train_head", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bits", [32, 8])
def test_example_learns(example, bits):
    """The rewarded half starts at even odds; both evaluations are on the same rows, so that what
    they differ by is what was learned."""
    before, after = example.run(steps=20, state_bits=bits, log=None)
    assert 0.4 < before < 0.6 and after > before + 0.05


def test_example_steps_repeat(example):
    """The same batches give the same weights, bit for bit."""
    models = [example.Head(256, 4096, 8, 1e-2, DEV) for _ in range(2)]
    for model in models:
        for step in range(3):
            example.train_step(model, example.rollout(model, 300, seed=step))
    for k in models[0].master:
        assert torch.equal(models[0].master[k], models[1].master[k])
        assert torch.equal(models[0].weight[k], models[0].master[k].to(BF16))


def make(T=96, d=256):
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return [r(T, d).to(BF16), r(T, d).to(BF16), (1 + 0.1 * r(d)).to(BF16), (1 + 0.1 * r(d)).to(BF16),
            r(d).to(BF16)], r(T, d).to(BF16), r(T, d).to(BF16)


def test_residual_norm_autograd():
    x, gh, gr = make()
    names = ("branch", "weight", "branch_weight", "gate")
    kw = dict(residual_scale=0.9, branch_scale=0.5)
    t = [v.clone().requires_grad_() for v in x]
    h, new = autograd.residual_norm(t[0], **dict(zip(names, t[1:])), **kw)
    (h.float() * gh.float() + new.float() * gr.float()).sum().backward()
    out = train.residual_norm(x[0], **dict(zip(names, x[1:])), **kw)
    assert torch.equal(h, out.normed) and torch.equal(new, out.residual)
    ref = train.residual_norm_backward(gh, gr, out.residual, out.rstd, branch_rstd=out.branch_rstd,
                                       **dict(zip(names, x[1:])), **kw)
    for v, want in zip(t, ref):
        assert v.grad.dtype == BF16 and torch.equal(v.grad, want.to(BF16))


def test_residual_norm_autograd_of_parts():
    """One output unused, no branch, no weight, frozen weights, an expanded gradient."""
    x, gh, gr = make()
    t = [v.clone().requires_grad_() for v in x]
    _, new = autograd.residual_norm(t[0], t[1], weight=t[2])
    new.sum().backward()  # an expanded gradient of ones, and none of the norm
    assert torch.equal(t[0].grad, torch.ones_like(x[0])) and torch.equal(t[1].grad, torch.ones_like(x[0]))
    assert not t[2].grad.any()
    t = [v.clone().requires_grad_() for v in x]
    h, same = autograd.residual_norm(t[0], weight=x[2])
    assert same is t[0]
    (h.float() * gh.float()).sum().backward()
    out = train.residual_norm(x[0], weight=x[2])
    ref = train.residual_norm_backward(gh, None, x[0], out.rstd, weight=x[2], weight_grads=False)
    assert torch.equal(t[0].grad, ref.residual) and ref.weight is None
    t = [v.clone().requires_grad_() for v in x]
    h, new = autograd.residual_norm(t[0], t[1], gate=t[4])
    assert h is None
    (new.float() * gr.float()).sum().backward()
    assert torch.equal(t[0].grad, gr)


def test_policy_loss_autograd():
    g = torch.Generator(device=DEV).manual_seed(5)
    T = 200
    logp = -torch.rand(T, generator=g, device=DEV)
    old = logp + 0.2 * torch.randn(T, generator=g, device=DEV)
    A = torch.randn(T, generator=g, device=DEV)
    ent = torch.rand(T, generator=g, device=DEV)
    kw = dict(ref_logp=old, kl_coef=0.1, entropy_coef=0.05)
    a, b = logp.clone().requires_grad_(), ent.clone().requires_grad_()
    loss, stats = autograd.policy_loss(a, old, A, entropy=b, **kw)
    (3 * loss).backward()
    ref = train.policy_loss(logp, old, A, entropy=ent, **kw)
    assert torch.equal(stats, ref.stats) and float(loss.detach()) == float(ref.stats[0])
    assert torch.equal(a.grad, 3 * ref.grad_logp) and torch.equal(b.grad, 3 * ref.grad_entropy)
    a = logp.clone().requires_grad_()
    loss, _ = autograd.policy_loss(a, old, A)
    loss.backward()
    assert torch.equal(a.grad, train.policy_loss(logp, old, A).grad_logp)


def test_chain_of_autograd_functions():
    """residual norm -> fused log-probabilities -> policy loss, one backward call: the gradients
    of the direct calls."""
    x, _, _ = make(64, 256)
    g = torch.Generator(device=DEV).manual_seed(6)
    W = (0.05 * torch.randn(4096, 256, generator=g, device=DEV)).to(BF16)
    y = torch.randint(0, 4096, (64,), generator=g, device=DEV)
    A = torch.randn(64, generator=g, device=DEV)
    r, b, w = (v.clone().requires_grad_() for v in x[:3])
    Wg = W.clone().requires_grad_()
    h, _ = autograd.residual_norm(r, b, weight=w)
    logp, ent = autograd.linear_logprob(h, Wg, y)
    loss, _ = autograd.policy_loss(logp, logp.detach(), A, entropy=ent, entropy_coef=0.01)
    loss.backward()
    out = train.residual_norm(x[0], x[1], weight=x[2])
    lp1, e1, lse = lp.linear_logprob_lse(out.normed, W, y)
    p = train.policy_loss(lp1, lp1, A, entropy=e1, entropy_coef=0.01)
    gH, gW = lp.linear_logprob_backward(out.normed, W, y, p.grad_logp, p.grad_entropy, saved_lse=lse,
                                        saved_entropy=e1, grad_W_dtype=BF16)
    n = train.residual_norm_backward(gH.to(BF16), None, out.residual, out.rstd, branch=x[1], weight=x[2])
    assert torch.equal(Wg.grad, gW) and torch.equal(r.grad, n.residual)
    assert torch.equal(b.grad, n.branch) and torch.equal(w.grad, n.weight.to(BF16))


def test_a_step_in_a_graph(example):
    """A captured step (with its step number) does what the eager step does."""
    eager, replayed = (example.Head(256, 4096, 32, 1e-2, DEV) for _ in range(2))
    batch = example.rollout(eager, 256, seed=1)
    example.train_step(example.Head(256, 4096, 32, 1e-2, DEV), batch)  # first calls set kernels up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stats, norm = example.train_step(replayed, batch)
    want, want_norm = example.train_step(eager, batch)
    graph.replay()
    assert torch.equal(stats, want) and torch.equal(norm, want_norm)
    for k in eager.master:
        assert torch.equal(eager.master[k], replayed.master[k])
