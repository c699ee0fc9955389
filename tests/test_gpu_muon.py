"""Muon's step on a GB300 against the fp64 oracle, which takes the polynomial of the singular values.

Tolerance of X after the Newton-Schulz steps, in the Frobenius norm, u = 2^-24.  A step's map of
matrices is as steep as p(s) = a s + b s^3 + c s^5 on [0, 1.21]: |p'| <= 4.3.  What a step adds: operands
are held to 2^-22 relatively and their products to 2^-22 (lo lo is left out), and a sum of K products in
float32, of random roundings, to sqrt(K) 2 u of the terms' norm (the tensor core cuts off where it does
not round, hence the 2).  Three products a step, of norms that add up to at most |b| + 2 |c| + a < 13 times
|X|: e = 13 (3 * 2^-22 + 2 sqrt(K) u) |X|.  Five steps multiply what the first adds by 4.3^4; the sum of
the powers is below 450, and |X| does not shrink, so |dX| <= 450 e |X| in all (for K = 512: 0.02 at
the very worst; singular values near 1 are drawn together, so that in fact it is far less).  A second,
much narrower bound comes from the same steps in float32 products by torch: the kernel may err 4 times
as much, and 16 u."""

import math

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import lp, train, tune
from oracle import tune as ot

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return t.double().cpu().numpy()


def matrices(shapes, grad=F32, seed=0, scale=1e-3, copy=True):
    g = torch.Generator(device=DEV).manual_seed(seed + len(shapes))
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    params = [0.02 * r(*s) for s in shapes]
    # a few strong directions over weak ones
    grads = [(scale * (r(s[0], 2) @ r(2, s[1]) + 0.3 * r(*s))).to(grad) for s in shapes]
    copies = [torch.zeros(s, dtype=BF16, device=DEV) for s in shapes] if copy else None
    momenta = [2 * scale * r(*s) for s in shapes]
    return params, grads, copies, momenta


def plain_steps(u, steps, eps):
    """The steps with float32 products."""
    x = u / (torch.linalg.vector_norm(u.double()).float() + eps)
    x = x if x.shape[0] <= x.shape[1] else x.t()
    for _ in range(steps):
        g = x @ x.t()
        x = ot.A * x + (ot.B * g + ot.C * (g @ g)) @ x
    return x if u.shape[0] <= u.shape[1] else x.t()


def run(shapes, grad=F32, steps=5, nesterov=True, scaling="spectral", lr=0.5, weight_decay=0.1, eps=1e-7,
        momentum=0.9, lr_scale=1.0, copy=True, seed=0, scale=1e-3):
    """One step of lr large enough that the update is what the parameters show."""
    params, grads, copies, momenta = matrices(shapes, grad, seed, scale, copy)
    before = [p.clone() for p in params]
    opt = tune.Muon(params, grads, copies=copies, lr=lr, momentum=momentum, nesterov=nesterov, steps=steps,
                    scaling=scaling, weight_decay=weight_decay, lr_scale=lr_scale, eps=eps)
    for view, m in zip(opt.momenta(), momenta):
        view.copy_(m)
    opt.step()
    for i, s in enumerate(shapes):
        if 0 in s:
            continue
        rate = lr * (lr_scale if isinstance(lr_scale, float) else lr_scale[i])
        wd = weight_decay if isinstance(weight_decay, float) else weight_decay[i]
        want, m = ot.muon_step(host(before[i]), host(grads[i]), host(momenta[i]), lr=lr, momentum=momentum,
                               nesterov=nesterov, weight_decay=wd, lr_scale=rate / lr, scaling=scaling,
                               steps=steps, eps=eps)
        got_m = host(opt.momenta()[i])
        size = np.abs(host(momenta[i])) * momentum + np.abs(host(grads[i]))
        assert np.all(np.abs(got_m - m) <= 2 * U * size)
        factor = rate * ot.muon_scale(*s, scaling)
        kept = host(before[i]) * (1 - rate * wd)
        X, got = (kept - want) / factor, (kept - host(params[i])) / factor
        norm = np.linalg.norm(X)
        # p itself is rounded: 3 operations on its parts
        rounding = 4 * U * np.linalg.norm(np.abs(kept) / factor + np.abs(X))
        e = 13 * (3 * 2.0 ** -22 + 2 * math.sqrt(max(s)) * U) * 450 * norm
        err = np.linalg.norm(got - X)
        assert err <= e + rounding, (s, err / norm)
        u = grads[i].float() + momentum * opt.momenta()[i] if nesterov else opt.momenta()[i]
        plain = np.linalg.norm(host(plain_steps(u, steps, eps)) - X)
        assert err <= 4 * plain + 16 * U * norm + rounding, (s, err / norm, plain / norm)
        assert np.all(np.isfinite(host(params[i])))
        if copy:
            assert torch.equal(copies[i], params[i].bfloat16())
    return opt


@pytest.mark.parametrize("grad", [F32, BF16])
@pytest.mark.parametrize("shape", [(128, 128), (1, 1), (1, 300), (300, 1), (2, 2), (64, 64), (127, 129), (65, 200),
                                   (200, 65), (256, 512), (513, 255), (130, 1000), (1000, 130), (640, 640)])
def test_shapes_and_types(shape, grad):
    run([shape], grad)


def test_many_matrices_at_once():
    run([(300, 200), (0, 5), (17, 400), (400, 17), (128, 256), (1, 9), (257, 257), (5, 0), (31, 33)], BF16,
        weight_decay=[0.0, 0.1, 0.2, 0.1, 0.0, 0.1, 0.1, 0.0, 0.3],
        lr_scale=[1.0, 1.0, 0.5, 2.0, 1.0, 1.0, 0.0625, 1.0, 1.0])


@pytest.mark.parametrize("kw", [dict(steps=1), dict(steps=2), dict(steps=7), dict(nesterov=False),
                                dict(scaling="rms"), dict(momentum=0.0), dict(weight_decay=0.0),
                                dict(copy=False), dict(scale=1e8), dict(scale=1e-9), dict(eps=1e-2)])
def test_options(kw):
    run([(200, 333), (333, 200)], **kw)


def test_large():
    run([(1024, 1536), (2100, 1100)], BF16, copy=False)


@pytest.mark.parametrize("shape", [(1024, 1024), (1100, 1000), (130, 4100), (2500, 60), (1023, 1025), (257, 8000)])
def test_split_over_clusters(shape):
    """Few tiles of a long K: a cluster a tile.  K that is no multiple of the segments, and one that only the first
    product has."""
    run([shape], BF16)


def test_several_turns_of_all_ctas():
    """More tiles than there are SMs, of many matrices and of one."""
    run([(300, 200), (129, 1000), (257, 140), (64, 64)] * 25, BF16, copy=False)
    run([(2200, 2300)], lr=0.1)


def test_an_orthogonal_update():
    """Singular values that are all equal: after the division each is 1 / sqrt(m), and X is that
    polynomial's value times the update's directions."""
    q, _ = torch.linalg.qr(torch.randn(256, 256, device=DEV, dtype=torch.float64))
    p, g = torch.zeros(256, 256, device=DEV), (3.0 * q).float().contiguous()
    tune.Muon([p], [g], lr=1.0, momentum=0.0).step()
    s = 1 / 16
    for _ in range(5):
        s = ot.A * s + ot.B * s ** 3 + ot.C * s ** 5
    err = np.linalg.norm(host(p) + s * host(q)) / (16 * s)
    assert err <= 450 * 13 * (3 * 2.0 ** -22 + 2 * 16 * U)
    assert err <= 1e-5  # singular values that agree leave rounding no direction to grow in but p's own slope


def test_steps_go_on_and_a_state_continues():
    shapes = [(96, 160), (160, 96), (50, 50)]
    params, grads, copies, _ = matrices(shapes)
    start = [p.clone() for p in params]
    a = tune.Muon(params, grads, copies=copies, weight_decay=0.01)
    for _ in range(3):
        a.step()
    others = [p.clone() for p in start]
    b = tune.Muon(others, grads, weight_decay=0.01)
    b.step()
    c = tune.Muon(others, grads, weight_decay=0.01, state=b.state_dict())
    c.step()
    c.step()
    assert all(torch.equal(p, q) for p, q in zip(params, others))
    assert torch.equal(a.momentum_buffer, c.momentum_buffer)


def test_a_matrix_has_the_bits_that_it_has_alone():
    """Also where K is split over a cluster's CTAs when few tiles are left to the GPU: alone, not in the batch."""
    shapes = [(300, 140), (129, 1500), (64, 64), (900, 2100), (4000, 100)]
    params, grads, _, _ = matrices(shapes, BF16)
    alone = [p.clone() for p in params]
    tune.Muon(params, grads).step()
    for p, g in zip(alone, grads):
        tune.Muon([p], [g]).step()
    assert all(torch.equal(p, q) for p, q in zip(params, alone))


def test_alignment_does_not_show():
    shapes = [(130, 256), (256, 130)]
    params, grads, _, _ = matrices(shapes, BF16)

    def moved(t):
        base = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        return base[1:].view(t.shape).copy_(t)
    p2, g2, c2 = [moved(p) for p in params], [moved(g) for g in grads], [moved(p.bfloat16()) for p in params]
    tune.Muon(params, grads).step()
    tune.Muon(p2, g2, copies=c2).step()
    assert all(torch.equal(p, q) for p, q in zip(params, p2))
    assert all(torch.equal(p.bfloat16(), q) for p, q in zip(params, c2))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1e30])
def test_a_norm_that_is_not_finite_leaves_its_matrix(bad):
    shapes = [(100, 60), (60, 100), (200, 200)]
    params, grads, copies, _ = matrices(shapes)
    for c in copies:
        c.fill_(7.0)
    good, _, _, _ = matrices(shapes)
    tune.Muon(good, grads).step()
    kept = params[1].clone()
    grads[1][3, 3] = bad
    opt = tune.Muon(params, grads, copies=copies)
    opt.step()
    assert torch.equal(params[1], kept) and (copies[1] == 7).all() and not opt.momenta()[1].any()
    assert torch.equal(params[0], good[0]) and torch.equal(params[2], good[2])


def test_no_gradient_at_all():
    params, grads, _, _ = matrices([(70, 90)])
    grads[0].zero_()
    kept = params[0].clone()
    tune.Muon(params, grads, lr=0.5, weight_decay=0.5).step()
    assert torch.equal(params[0], kept * 0.75)


def test_streams_graphs_and_versions():
    shapes = [(256, 300), (100, 90)]
    params, grads, copies, _ = matrices(shapes)
    ref = [p.clone() for p in params]
    a = tune.Muon(ref, grads)
    for _ in range(4):
        a.step()
    side = torch.cuda.Stream()
    b = tune.Muon(params, grads, copies=copies)
    side.wait_stream(torch.cuda.current_stream())
    version = params[0]._version, copies[1]._version, b.momentum_buffer._version
    b.step(stream=side)
    assert all(x > y for x, y in zip((params[0]._version, copies[1]._version, b.momentum_buffer._version), version))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(params, ref))
    assert all(torch.equal(p.bfloat16(), q) for p, q in zip(params, copies))


def test_another_gradient_and_factors():
    params, grads, _, _ = matrices([(64, 80)])
    same = [p.clone() for p in params]
    opt = tune.Muon(params, grads, weight_decay=0.1)
    other = [2.0 * g for g in grads]
    opt.set_grads(other)
    opt.weight_decay = 0.2
    opt.lr_scale = [0.5]
    opt.step(lr=0.04)
    tune.Muon(same, other, lr=0.04, weight_decay=0.2, lr_scale=0.5).step()
    assert torch.equal(params[0], same[0])
    with pytest.raises(ValueError):
        opt.set_grads([grads[0][:3]])
    assert opt.grads == other


def test_refusals():
    p, g = torch.zeros(8, 16, device=DEV), torch.zeros(8, 16, device=DEV)
    make = lambda *a, **kw: tune.Muon(*(a or ([p], [g])), **kw)  # noqa: E731
    with pytest.raises(ValueError, match="no tensors"):
        make([], [])
    with pytest.raises(TypeError, match="float32 matrices"):
        make([p.bfloat16()], [g])
    with pytest.raises(TypeError, match="float32 matrices"):
        make([p[0]], [g[0]])
    with pytest.raises(TypeError, match="float32 matrices"):
        make([p.t()], [g.t()])
    with pytest.raises(TypeError, match="gradients must be"):
        make([p], [g.half()])
    with pytest.raises(ValueError, match="params' shapes"):
        make([p], [g[:4]])
    with pytest.raises(ValueError, match="share memory"):
        make([p], [p])
    with pytest.raises(ValueError, match="share memory"):
        make([p, p], [g, g])
    with pytest.raises(ValueError, match="scaling"):
        make(scaling="adam")
    with pytest.raises(ValueError, match="steps"):
        make(steps=0)
    with pytest.raises(ValueError, match="momentum must be"):
        make(state={"momentum": torch.zeros(5, device=DEV)})
    with pytest.raises(ValueError, match="CUDA"):
        make([p.cpu()], [g.cpu()])
    with pytest.raises(lp.LpError):
        make(weight_decay=-1.0)
    for kw in (dict(momentum=1.0), dict(momentum=-0.1), dict(eps=0.0), dict(lr=float("nan")), dict(lr=-1.0)):
        with pytest.raises(lp.LpError):
            make(**kw).step()
    with pytest.raises(lp.LpError):
        make([torch.zeros(65537, 1, device=DEV)], [torch.zeros(65537, 1, device=DEV)])


def test_a_wait_that_gives_up_shows():
    """A copy that is announced and never made: the waits end after their bound, the parameters that
    depend on it are NaN, and the next step is right."""
    params, grads, _, _ = matrices([(256, 256)])
    ref = [p.clone() for p in params]
    opt = tune.Muon(params, grads)
    calls = tune.load_calls()
    lp.lp_set_fault_injection(1)
    try:
        ws = calls.muon_step(opt._plan_host, opt._plan, opt.momentum_buffer, 0.02, 0.95, True, 5, 1e-7, *opt._given,
                             opt._streams, opt._captured)
        torch.cuda.synchronize()
    finally:
        lp.lp_set_fault_injection(0)
    assert lp.lp_get_device_error(ws) != 0
    assert torch.isnan(params[0]).any()
    params[0].copy_(ref[0])
    opt.momentum_buffer.zero_()
    opt.step()
    tune.Muon(ref, grads).step()
    assert torch.equal(params[0], ref[0])


def test_beside_adamw():
    """Matrices to Muon, the rest to AdamW, on gradients of one buffer."""
    params, grads, copies, _ = matrices([(64, 128)])
    w, gw = torch.ones(128, device=DEV), torch.full((128,), 0.1, device=DEV)
    a, b = tune.Muon(params, grads, copies=copies), train.AdamW([w], [gw], lr=1e-2)
    before = params[0].clone()
    a.step()
    b.step()
    assert (w < 1).all() and not torch.equal(params[0], before)
