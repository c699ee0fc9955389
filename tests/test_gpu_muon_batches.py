"""Muon's step over more matrices than go through its workspace at once, on a GB300: a matrix has the bits that
it has in a step of its own, whichever batch it is in."""

import pytest
import torch

from invariant_token_logprobs_gb300 import lp, tune

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16

# by elements of whole 128s: three of 2^24 and the small ones; another of 2^24 with its small ones; one of 2^26
SHAPES = [(4096, 4096), (300, 200), (4096, 4096), (0, 5), (17, 400), (4096, 4096),
          (4096, 4096), (100, 60), (5, 0), (2050, 120), (64, 64), (1030, 1100),
          (8192, 8192),
          (31, 33), (257, 140)]
BATCHES = [6, 6, 1, 2]  # the matrices of each


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def matrices(shapes, grad, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return [0.02 * r(*s) for s in shapes], [(1e-3 * (r(s[0], 2) @ r(2, s[1]) + 0.3 * r(*s))).to(grad) for s in shapes]


def batches_of(opt):
    return int(opt._plan_host.view(torch.int64)[3])


@pytest.mark.parametrize("grad", [F32, BF16])
def test_every_matrix_has_its_own_bits(grad):
    params, grads = matrices(SHAPES, grad)
    bad = BATCHES[0] + 1
    grads[bad][3, 3] = float("nan")  # a matrix of the second batch is left as it was
    alone = [p.clone() for p in params]
    copies = [torch.full(p.shape, 7.0, dtype=BF16, device=DEV) for p in params]
    kept = params[bad].clone()
    opt = tune.Muon(params, grads, copies=copies, weight_decay=0.1)
    assert batches_of(opt) == len(BATCHES)
    opt.step()
    opt.step()
    for i, (p, g) in enumerate(zip(alone, grads)):
        one = tune.Muon([p], [g], weight_decay=0.1)
        one.step()
        one.step()
        assert torch.equal(p, params[i]), SHAPES[i]
        assert torch.equal(one.momenta()[0], opt.momenta()[i]), SHAPES[i]
        assert torch.equal(copies[i], torch.full_like(copies[i], 7.0) if i == bad else params[i].bfloat16()), SHAPES[i]
    assert torch.equal(params[bad], kept) and not opt.momenta()[bad].any()


def test_batches_in_a_graph():
    params, grads = matrices(SHAPES, BF16, seed=1)
    others = [p.clone() for p in params]
    a, b = tune.Muon(params, grads), tune.Muon(others, grads)
    for _ in range(2):
        a.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(params, others))
    assert torch.equal(a.momentum_buffer, b.momentum_buffer)


def test_a_wait_that_gives_up_is_its_batchs():
    """A copy of the first batch that is announced and never made: after the bounded waits the params of that batch
    are NaN and the workspace says so; the other batches' have the bits that they have alone."""
    params, grads = matrices(SHAPES, BF16, seed=2)
    start = [p.clone() for p in params]
    opt = tune.Muon(params, grads)
    lp.lp_set_fault_injection(1)
    try:
        ws = tune.load_calls().muon_step(opt._plan_host, opt._plan, opt.momentum_buffer, 0.02, 0.95, True, 5, 1e-7,
                                         *opt._given, opt._streams, opt._captured)
        torch.cuda.synchronize()
    finally:
        lp.lp_set_fault_injection(0)
    assert lp.lp_get_device_error(ws) != 0
    del ws
    for i, (p, g) in enumerate(zip(start, grads)):
        if i < BATCHES[0]:
            assert torch.isnan(params[i]).all(), SHAPES[i]
            continue
        tune.Muon([p], [g]).step()
        assert torch.equal(p, params[i]), SHAPES[i]
    # and the next step clears the word
    for p, s in zip(params, start):
        p.copy_(s)
    opt.step()
    assert not any(torch.isnan(p).any() for p in params)
