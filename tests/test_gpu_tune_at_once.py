"""Calls of the fine-tuning operators at once, on streams and threads of their own, on a GB300: each has workspaces of
its own and the bits that it has alone."""

import threading

import pytest
import torch

from invariant_token_logprobs_gb300 import tune

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def work(seed):
    """Inputs of each operator, and a function that runs them all a few times and returns every output."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    norms = [(r(700, d).to(a), r(700, d).to(b)) for d, a, b in ((1024, BF16, BF16), (515, BF16, BF16), (2048, torch.float32, BF16))]
    lengths = torch.randint(1, 900, (400,), generator=g, device=DEV)
    batches = [torch.cat([lengths.new_zeros(1), n.cumsum(0)]) for n in (lengths, lengths[:8])]
    logps = [-r(int(cu[-1])).abs() for cu in batches]
    shapes = [(256, 300), (1100, 1000), (64, 2050), (700, 700)]
    params, grads = [r(*s) for s in shapes], [r(*s) for s in shapes]

    def run():
        out = []
        optimizer = tune.Muon([p.clone() for p in params], grads)
        for _ in range(4):
            for x, y in norms:
                w = torch.ones(x.shape[1], device=DEV)
                n = tune.layer_norm(x, y, weight=w, bias=w)
                out += n
                out += [t for t in tune.layer_norm_backward(n.normed, None, n.residual, n.mean, n.rstd, weight=w, bias=w,
                                                            branch=True) if t is not None]
            for logp, cu in zip(logps, batches):
                out += tune.preference_loss(logp, cu, ref_logp=0.9 * logp, average=True)
            optimizer.step()
        return out + optimizer.params + [optimizer.momentum_buffer]

    return run


def test_on_streams():
    runs = [work(seed) for seed in range(3)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        got = []
        for run, stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


def test_on_threads():
    runs = [work(seed) for seed in range(3)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    got = [None] * len(runs)

    def call(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = runs[i]()
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=call, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


def test_graphs_at_once():
    """Two captured runs, replayed together."""
    graphs, outs = [], []
    g = torch.Generator(device=DEV).manual_seed(7)
    shapes = [(256, 300), (1100, 1000)]
    for i in range(2):
        params = [torch.randn(s, generator=g, device=DEV) for s in shapes]
        grads = [torch.randn(s, generator=g, device=DEV) for s in shapes]
        alone = [p.clone() for p in params]
        one, captured = tune.Muon(alone, grads), tune.Muon(params, grads)
        x = torch.randn(3000, 1024, generator=g, device=DEV).to(BF16)
        logp, cu = -torch.randn(20000, generator=g, device=DEV).abs(), torch.arange(0, 20001, 2500, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured.step()
            n, p = tune.layer_norm(x, x), tune.preference_loss(logp, cu)
        for _ in range(5):
            one.step()
        graphs.append((graph, captured, x, logp, cu))  # a graph keeps no inputs
        outs.append((params, alone, [*n, *p], [*tune.layer_norm(x, x), *tune.preference_loss(logp, cu)]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for (graph, *_), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for params, alone, got, kept in outs:
        assert all(torch.equal(a, b) for a, b in zip(params, alone))
        assert all(torch.equal(a, b) for a, b in zip(got, kept))
