"""What the calls of train.py and their autograd forms owe their caller besides the numbers:
what they return where these are not finite, streams, lifetimes, versions, serialisation."""

import pytest
import torch

from invariant_token_logprobs_gb300 import autograd, train  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value,want", [("inf", "inf"), ("-inf", "inf"), ("1e30", "inf"), ("nan", "nan")])
@pytest.mark.parametrize("at", [0, 4321])
def test_norm_of_gradients_that_are_not_finite(bits, value, want, at):
    """An infinite gradient, or squares past float32, have an infinite norm; only a NaN has a NaN."""
    p, g = torch.ones(5000, device=DEV), torch.ones(5000, device=DEV)
    g[at] = float(value)
    norm = train.AdamW([p], [g], state_bits=bits).step(max_norm=1.0)
    assert str(float(norm)) == want
    assert torch.equal(p, torch.ones_like(p))


def make_optimizer(bits, seed=1, sizes=(700, 9000)):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda n: torch.randn(n, generator=g, device=DEV)  # noqa: E731
    return train.AdamW([r(n) for n in sizes], [r(n) for n in sizes],
                       copies=[torch.zeros(n, dtype=BF16, device=DEV) for n in sizes], lr=1e-2, state_bits=bits)


def busy_stream():
    """A stream that is ordered after what was made so far and has some 0.2 s of work ahead."""
    overwrite([512])  # its kernel is loaded before the clock runs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
    return side


def overwrite(sizes):
    """What comes next in memory of these sizes: tensors full of ones bits."""
    return [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(64)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [None, 0.5])
def test_new_gradients_right_after_a_step_on_another_stream(bits, max_norm):
    """Plan and gradients of a step that has not run yet are not handed out again."""
    opt, twin = make_optimizer(bits), make_optimizer(bits)
    twin.step(max_norm=max_norm)
    twin.set_grads([g * 2 for g in twin.grads])
    twin.step(max_norm=max_norm)
    new = [g * 2 for g in opt.grads]
    held = [opt._plan] + opt.grads
    old = {t.data_ptr(): t.numel() * t.element_size() for t in held}
    del held
    side = busy_stream()
    opt.step(max_norm=max_norm, stream=side)
    opt.set_grads(new)
    after = overwrite(old.values())
    assert not side.query(), "the step has run: the test says nothing"
    assert not {t.data_ptr() for t in after} & set(old)
    torch.cuda.current_stream().wait_stream(side)
    opt.step(max_norm=max_norm)
    for a, b in zip(opt.params + opt.copies + list(opt.state_values()),
                    twin.params + twin.copies + list(twin.state_values())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_an_optimizer_that_is_dropped_right_after_a_step_on_another_stream(bits):
    opt, twin = make_optimizer(bits), make_optimizer(bits)
    twin.step()
    params, copies = opt.params, opt.copies
    held = [opt._plan, opt.exp_avg, opt.exp_avg_sq] + opt.grads
    old = {t.data_ptr(): t.numel() * t.element_size() for t in held}
    del held
    side = busy_stream()
    opt.step(stream=side)
    del opt
    after = overwrite(old.values())
    assert not side.query(), "the step has run: the test says nothing"
    assert not {t.data_ptr() for t in after} & set(old)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(params + copies, twin.params + twin.copies):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_keeps_the_plan_that_it_was_captured_with(bits):
    opt, twin = make_optimizer(bits), make_optimizer(bits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(max_norm=0.5)
    held = [opt._plan] + opt.grads
    old = {t.data_ptr(): t.numel() * t.element_size() for t in held}
    del held
    opt.set_grads([g * 2 for g in opt.grads])
    after = overwrite(old.values())
    assert not {t.data_ptr() for t in after} & set(old)
    graph.replay()
    twin.step(max_norm=0.5)
    for a, b in zip(opt.params + opt.copies + list(opt.state_values()),
                    twin.params + twin.copies + list(twin.state_values())):
        assert torch.equal(a, b)


def test_writes_in_place_show_to_autograd():
    """A graph that saved the old values does not go back through the new ones."""
    residual, branch, w = (torch.randn(*s, device=DEV) for s in ((8, 64), (8, 64), (64,)))
    x = torch.randn(8, 64, device=DEV, requires_grad=True)
    y = (x * residual).sum()
    train.residual_norm(residual, branch, weight=w)  # writes none of its inputs
    y.backward(retain_graph=True)
    train.residual_norm(residual, branch, weight=w, in_place=True)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_shows_to_autograd(bits):
    opt = make_optimizer(bits)
    for t in opt.params + opt.copies:
        x = torch.ones_like(t, requires_grad=True)
        y = (x * t).sum()
        opt.step(max_norm=1.0)
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            y.backward()
    # gradients are read, and params may be of inference mode, where nothing is counted
    for g in opt.grads:
        x = torch.ones_like(g, requires_grad=True)
        y = (x * g).sum()
        opt.step()
        y.backward()
    with torch.inference_mode():
        p = torch.ones(300, device=DEV)
        before = p.clone()
        train.AdamW([p], [torch.ones(300, device=DEV)], state_bits=bits).step()
        assert not torch.equal(p, before)


def test_policy_loss_autograd_on_another_stream():
    """The loss is a copy of the call's first statistic: made on the call's stream, after it."""
    g = torch.Generator(device=DEV).manual_seed(3)
    T = 3000
    logp = -torch.rand(T, generator=g, device=DEV)
    old = logp + 0.2 * torch.randn(T, generator=g, device=DEV)
    A, ent = torch.randn(T, generator=g, device=DEV), torch.rand(T, generator=g, device=DEV)
    ref = train.policy_loss(logp, old, A, entropy=ent, entropy_coef=0.1)
    a, b = logp.clone().requires_grad_(), ent.clone().requires_grad_()
    for given in (lambda s: s, lambda s: s.cuda_stream):
        overwrite([512, 4 * T])  # what is left in memory that the outputs may get
        side = busy_stream()
        loss, stats = autograd.policy_loss(a, old, A, entropy=b, entropy_coef=0.1, stream=given(side))
        assert not side.query(), "the call has run: the test says nothing"
        torch.cuda.current_stream().wait_stream(side)
        ga, gb = torch.autograd.grad(3 * loss, (a, b))
        assert torch.equal(stats, ref.stats) and float(loss.detach()) == float(ref.stats[0])
        assert torch.equal(ga, 3 * ref.grad_logp) and torch.equal(gb, 3 * ref.grad_entropy)


def second_order(y, x):
    g, = torch.autograd.grad(y, x, create_graph=True)
    with torch.no_grad():
        g.mul_(1)  # as a clip by the norm does
    with pytest.raises(RuntimeError, match="gradient of a gradient"):
        (g.float().square().sum() + y).backward()  # a penalty on the gradient beside the loss


def test_a_gradient_of_a_gradient_is_refused():
    """The backward calls have no derivative; leaving its terms out in silence would be wrong."""
    x = torch.randn(4, 64, device=DEV, requires_grad=True)
    branch = torch.randn(4, 64, device=DEV, requires_grad=True)
    w = torch.ones(64, device=DEV, requires_grad=True)
    for wanted in (x, branch, w):
        h, new = autograd.residual_norm(x, branch, weight=w)
        second_order((h * new).sum(), wanted)
    logp = (-torch.rand(9, device=DEV)).requires_grad_()
    second_order(autograd.policy_loss(logp, logp.detach(), torch.ones(9, device=DEV))[0], logp)
    H = torch.randn(16, 64, device=DEV).to(BF16).requires_grad_()
    W = torch.randn(512, 64, device=DEV).to(BF16)
    y = torch.arange(16, device=DEV)
    second_order(autograd.linear_logprob(H, W, y)[0].sum(), H)
    z = torch.randn(16, 512, device=DEV, requires_grad=True)
    second_order(autograd.logprob_from_logits(z, y)[0].sum(), z)


@pytest.mark.parametrize("T", [1, 4, 300, 3000])
def test_results_can_be_saved(T, tmp_path):
    """Whatever the sizes, all results of a call go through torch.save, of small calls in little."""
    d = 64
    r, y = (torch.randn(T, d, device=DEV).to(BF16) for _ in range(2))
    w, gate = torch.ones(d, device=DEV), torch.ones(d, device=DEV, dtype=BF16)
    out = train.residual_norm(r, y, weight=w, branch_weight=w, gate=gate)
    grads = train.residual_norm_backward(r, y, out.residual, out.rstd, branch=y, weight=w, branch_weight=w,
                                         branch_rstd=out.branch_rstd, gate=gate)
    logp = -torch.rand(T, device=DEV)
    loss = train.policy_loss(logp, logp, logp, entropy=-logp)
    opt = train.AdamW([torch.ones(9000, device=DEV)], [torch.ones(9000, device=DEV)], state_bits=8)
    step = (opt.step(max_norm=1.0), *opt.state_values())
    for results in (out, grads, loss, step):
        path = tmp_path / "results.pt"
        torch.save(tuple(results), path)
        for a, b in zip(torch.load(path), results):
            assert torch.equal(a, b) and a.dtype == b.dtype
        held = sum({t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in results}.values())
        whole = sum(t.numel() * t.element_size() for t in results)
        assert held <= whole + 256 * (len(results) + 1)  # each rounded up, and next to no scratch


def test_a_workspace_spans_what_it_says():
    """An expanded tensor has more elements than memory; it is refused, not written past."""
    T, d = 2000, 256
    r = torch.randn(T, d, device=DEV)
    w = torch.ones(d, device=DEV)
    rstd = torch.ones(T, device=DEV)
    size = train.residual_norm_backward_workspace_size(T, d)
    ref = train.residual_norm_backward(r, None, r, rstd, weight=w)
    got = train.residual_norm_backward(r, None, r, rstd, weight=w,
                                       workspace=torch.empty(size, dtype=torch.uint8, device=DEV))
    assert torch.equal(got.weight, ref.weight)
    logp = torch.rand(20000, device=DEV)
    need = train.policy_loss_workspace_size(20000, 0)
    loss = train.policy_loss(logp, logp, logp, workspace=torch.empty(need // 4 + 1, device=DEV))
    assert torch.equal(loss.stats, train.policy_loss(logp, logp, logp).stats)
    one = torch.empty(256, dtype=torch.uint8, device=DEV)
    for bad in (one[:1].expand(size), one.expand(size // 256 + 1, 256),
                torch.empty(2 * size, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            train.residual_norm_backward(r, None, r, rstd, weight=w, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            train.policy_loss(logp, logp, logp, workspace=bad)
    with pytest.raises(train.LpError, match="WORKSPACE"):
        train.policy_loss(logp, logp, logp, workspace=one)
