"""AdamW over many tensors on a GB300 against the fp64 oracle, with moments in 32 and in 8 bits.

Tolerances, with u = 2^-24: a moment is two products and a sum, and g^2 one more product: 4 u of
its terms' magnitude (|b1 m| + |(1 - b1) g|), twice that through the float32 rounding of the
factors: 8 u.  The change is a quotient by a root of them and an eps: 32 u relatively where the
first moment does not cancel, so 32 u times its terms' magnitude; a param adds its own rounding."""

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import train
from oracle import train as ot

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8)


def host(t):
    return t.double().cpu().numpy()


def make(sizes, grad=torch.float32, copies=True, shift=0, seed=0, **kw):
    """Params, gradients and copies of these sizes, `shift` elements into their memory."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def one(n, dtype, scale):
        return (torch.randn(n + shift, generator=g, device=DEV) * scale).to(dtype)[shift:]
    params = [one(n, torch.float32, 0.1) for n in sizes]
    grads = [one(n, grad, 1e-2) for n in sizes]
    made = [torch.zeros(n + shift, dtype=torch.bfloat16, device=DEV)[shift:] if copies else None
            for n in sizes]
    return train.AdamW(params, grads, copies=made, **{**HYPER, **kw})


def check_step(opt, step, weight_decay, lr_scale, clip=1.0):
    """One step of `opt` against the oracle, from the moments that it holds."""
    m0, v0 = ([host(x) for x in opt.views(t)] for t in opt.state_values())
    p0, g0 = [host(p) for p in opt.params], [host(g) * clip for g in opt.grads]
    opt.step()
    m1, v1 = ([host(x) for x in opt.views(t)] for t in opt.state_values())
    b1, b2 = HYPER["betas"]
    for i, p in enumerate(opt.params):
        lr = HYPER["lr"] * lr_scale[i]
        want, m, v = ot.adamw_step(p0[i], g0[i], m0[i], v0[i], step, lr, HYPER["betas"], HYPER["eps"],
                                   weight_decay[i])
        mag = np.abs(b1 * m0[i]) + np.abs((1 - b1) * g0[i])
        change = lr / (1 - b1 ** step) * mag / (np.sqrt(v / (1 - b2 ** step)) + HYPER["eps"])
        assert np.all(np.abs(host(p) - want) <= 32 * U * change + 4 * U * np.abs(p0[i])), i
        if opt.copies[i] is not None:
            assert torch.equal(opt.copies[i], p.to(torch.bfloat16))
        if opt.state_bits == 32:
            assert np.all(np.abs(m1[i] - m) <= 8 * U * mag), i
            assert np.all(np.abs(v1[i] - v) <= 8 * U * v), i
        else:
            # what is rounded to a code is the float32 moment (one that cancels is further off
            # than a code's edge allows for), itself within the bounds above
            f = np.float32
            m32 = (f(b1) * m0[i].astype(f) + f(1 - b1) * g0[i].astype(f)).astype(np.float64)
            assert np.all(np.abs(m32 - m) <= 8 * U * mag), i
            for x, held, signed in ((m32, m1[i], True), (np.sqrt(v), np.sqrt(v1[i]), False)):
                check_codes(x, held, signed)


def check_codes(x, held, signed):
    """Every held value is one of the two code values around x (a relative 2^-20 of slack for x in
    float32 and for the square root taken here)."""
    for a in range(0, len(x), 256):
        part, got = x[a:a + 256], held[a:a + 256]
        scale = np.float32(np.max(np.abs(part)))
        scale = np.float64(scale) if scale >= 2.0 ** -100 else 0.0
        slack = 2.0 ** -20 * np.abs(part)
        low, _, _ = ot.moment_neighbours(np.abs(part) - slack, scale, signed)
        _, high, _ = ot.moment_neighbours(np.abs(part) + slack, scale, signed)
        size = np.abs(got)
        assert np.all(size >= low * (1 - 2.0 ** -20)) and np.all(size <= high * (1 + 2.0 ** -20))
        assert np.all((size == 0) | (np.sign(got) == np.sign(part)))


SIZES = [1, 255, 256, 257, 2047, 2048, 2049, 0, 5000, 70000]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("copies,shift", [(True, 0), (False, 0), (True, 1), (True, 2)])
def test_steps(bits, grad, copies, shift):
    decay = [0.1 if i % 2 else 0.0 for i in range(len(SIZES))]
    scale = [1.0 if i % 3 else 0.25 for i in range(len(SIZES))]
    opt = make(SIZES, grad, copies, shift, weight_decay=decay, lr_scale=scale, state_bits=bits)
    for step in range(1, 5):
        check_step(opt, step, decay, scale)
        for g in opt.grads:
            g.mul_(-0.7 if step % 2 else 1.3)


def test_alignment_and_grouping_keep_the_bits():
    for bits in (32, 8):
        a, b = make([5000, 3000], state_bits=bits), make([5000, 3000], state_bits=bits, shift=1)
        for x, y in zip(a.params + a.grads, b.params + b.grads):
            y.copy_(x)
        for _ in range(3):
            a.step()
            b.step()
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
        assert all(torch.equal(x, y) for x, y in zip(a.state_values(), b.state_values()))


def test_random_rounding_uses_the_stated_words():
    """Each code against the rounding by the published generator's words, where the element is not
    within 2^-10 of a code step of its threshold."""
    opt = make([3000], state_bits=8, seed=3)
    opt.seed = (5 << 32) | 9
    g = host(opt.grads[0])
    opt.step()
    m = (1 - 0.9) * g
    u = np.sqrt((1 - 0.99) * g * g)
    held = [host(opt.views(t)[0]) for t in opt.state_values()]
    checked = 0
    for a in range(0, 3000, 256):
        for x, values, signed, at in ((m, held[0], True, 0), (u, np.sqrt(held[1]), False, 16)):
            part = np.abs(x[a:a + 256])
            scale = float(np.float32(part.max()))
            low, high, share = ot.moment_neighbours(part, scale, signed)
            for e in range(0, len(part), 7):
                flat = a + e
                word = ot.philox_4x32_7((flat // 4, 0, 1, 0), (9, 5))[flat % 4] >> at & 0xFFFF
                if abs(share[e] + word / 65536 - 1) < 2.0 ** -10:
                    continue
                want = high[e] if share[e] + word / 65536 >= 1 else low[e]
                assert abs(abs(values[a + e]) - want) <= 2.0 ** -20 * scale
                checked += 1
    assert checked > 800


def test_rounding_is_unbiased():
    """A gradient of zero decays the moments by b1 and b2 a step; over N = 65536 equal elements the
    mean of m after k steps is b1^k within the rounding's noise.  One rounding errs by at most a
    step, 2^-3 of the value, with a standard deviation of at most half: 2^-4 / sqrt(N) = 2.4e-4 of
    the mean, and k = 20 of them at most 20^0.5 times that: 1.1e-3; five deviations are asked."""
    n = 65536
    opt = make([n], state_bits=8, copies=False, weight_decay=0.0)
    opt.grads[0].zero_()
    # every block: one element of 1 to hold the scale, the others at a value between codes
    m = torch.full((n // 256, 256), 0.37, device=DEV)
    m[:, 0] = 1.0
    codes = ot.moment_values(True)
    c = int(np.searchsorted(codes, 0.37))
    opt.exp_avg.copy_(torch.full((n,), c, dtype=torch.uint8, device=DEV))
    opt.exp_avg.view(-1, 256)[:, 0] = 127
    opt.exp_avg_scale.fill_(1.0)
    start = codes[c]
    for _ in range(20):
        opt.step()
    mean = float(opt.state_values()[0].view(-1, 256)[:, 1:].double().mean())
    assert abs(mean / (start * 0.9 ** 20) - 1) < 5 * 1.1e-3


@pytest.mark.parametrize("bits", [32, 8])
def test_special_values(bits):
    opt = make([1024, 1024], state_bits=bits, weight_decay=0.0)
    opt.grads[0][300] = float("nan")
    opt.grads[0][600] = float("inf")
    opt.grads[1][:256] = 0.0
    opt.grads[1][256:512] = 1e-35
    before = opt.params[1].clone()
    opt.step()
    bad = torch.isnan(opt.params[0])
    assert bad[300] and bad[600] and int(bad.sum()) == 2
    assert torch.isfinite(opt.params[1]).all()
    assert torch.equal(opt.params[1][:256], before[:256])
    m, v = (opt.views(t) for t in opt.state_values())
    if bits == 8:
        # the two blocks with them read back as NaN, the others are whole
        assert torch.isnan(m[0][256:768]).all() and torch.isnan(v[0][256:768]).all()
        assert torch.isfinite(m[0][:256]).all() and torch.isfinite(m[0][768:]).all()
        # a block below 2^-100 holds zeros
        assert not m[1][:512].any() and not v[1][:512].any()
    opt.grads[0].zero_()
    opt.step()
    assert torch.isfinite(opt.params[0][:256]).all()


@pytest.mark.parametrize("bits,grad", [(32, torch.float32), (8, torch.bfloat16)])
def test_clip(bits, grad):
    """The norm: squares are rounded once and summed in chains of at most 2048: 2100 u of it, and
    the root halves that; then the step is that of the scaled gradients."""
    opt = make([5000, 12, 2049, 100000], grad, state_bits=bits)
    want = np.sqrt(sum(np.sum(host(g) ** 2) for g in opt.grads))
    twin = make([5000, 12, 2049, 100000], torch.float32, state_bits=bits)
    for a, b in zip(opt.grads, twin.grads):
        b.copy_(a)
    norm = opt.step(max_norm=0.5)
    assert norm.dim() == 0 and abs(float(norm) - want) <= 1050 * U * want
    for g in twin.grads:
        g.mul_(torch.clamp_max(0.5 / (norm + 1e-6), 1.0))
    twin.step()
    assert all(torch.equal(a, b) for a, b in zip(opt.params, twin.params))
    # a norm below the limit changes nothing
    opt.step(max_norm=1e9)
    for a, b in zip(opt.grads, twin.grads):
        b.copy_(a)
    twin.step()
    assert all(torch.equal(a, b) for a, b in zip(opt.params, twin.params))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30])
def test_norm_that_is_not_finite_skips_the_step(bits, value):
    opt = make([300, 4000], state_bits=bits)
    opt.step()
    kept = [t.clone() for t in opt.params + opt.copies + list(opt.state_values())]
    opt.grads[1][77] = value
    norm = opt.step(max_norm=1.0)
    assert not torch.isfinite(norm)
    for a, b in zip(opt.params + opt.copies + list(opt.state_values()), kept):
        assert torch.equal(a, b)
    assert opt.step_count == 2


@pytest.mark.parametrize("bits", [32, 8])
def test_streams_graphs_state_and_new_gradients(bits):
    a, b = (make([700, 9000], state_bits=bits, seed=8) for _ in range(2))
    for _ in range(3):
        a.step(max_norm=0.1)
        b.step(max_norm=0.1)
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    # continuing from a state dictionary
    state = {k: v.clone() if torch.is_tensor(v) else v for k, v in b.state_dict().items()}
    c = train.AdamW([p.clone() for p in b.params], b.grads, **HYPER, state_bits=bits, state=state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(max_norm=0.1, lr=1e-2)
    b.step(max_norm=0.1, lr=1e-2, stream=side)
    c.step(max_norm=0.1, lr=1e-2)
    side.synchronize()
    for x, y, z in zip(a.params, b.params, c.params):
        assert torch.equal(x, y) and torch.equal(x, z)
    # a captured step is the step with that number
    held = [t.clone() for t in a.params + [a.exp_avg, a.exp_avg_sq]]
    scales = [t.clone() for t in (a.exp_avg_scale, a.exp_avg_sq_scale) if t is not None]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(max_norm=0.1)
    for t, k in zip(a.params + [a.exp_avg, a.exp_avg_sq], held):
        assert torch.equal(t, k)
    graph.replay()
    b.step(max_norm=0.1)
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    assert all(torch.equal(x, y) for x, y in zip(a.state_values(), b.state_values()))
    assert len(scales) == (2 if bits == 8 else 0)
    # other gradient tensors, of the other type
    b.set_grads([g.bfloat16() for g in b.grads])
    a.set_grads([g.bfloat16().float() for g in a.grads])
    a.step()
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


def test_elements_past_32_bits():
    """A tensor of more than 2^32 elements: its ends are those of small tensors with the same
    values and, for the rounding, the same flat index."""
    n = (1 << 32) + 4096 + 13
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(4096 + 13, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    p[-4109:], g[-4109:] = tail, tail.bfloat16()
    opt = train.AdamW([p], [g], **HYPER, state_bits=8, seed=3)
    norm = opt.step(max_norm=1e9)
    ref = train.AdamW([tail.clone()], [g[-4109:].clone()], **HYPER, state_bits=8, seed=3)
    ref_norm = ref.step(max_norm=1e9)
    assert torch.equal(p[-4109:], ref.params[0]) and not p[:4096].any()
    assert float(norm) == float(ref_norm)
    m = opt.exp_avg[-6144:].cpu().numpy()
    want = (1 - 0.9) * host(g[-4109:])
    for e in range(0, 4109, 411):
        flat = (1 << 32) + e
        a = e // 256 * 256
        scale = float(np.float32(np.abs(want[a:a + 256]).max()))
        low, high, share = ot.moment_neighbours(np.abs(want[e:e + 1]), scale, True)
        word = ot.philox_4x32_7((flat // 4 & 0xFFFFFFFF, flat // 4 >> 32, 1, 0), (3, 0))[flat % 4] & 0xFFFF
        if abs(share[0] + word / 65536 - 1) > 2.0 ** -10:
            value = ot.moment_values(True)[m[e] & 127] * scale
            assert abs(value - (high[0] if share[0] + word / 65536 >= 1 else low[0])) <= 2.0 ** -20 * scale


def test_refusals():
    p, g = torch.zeros(8, device=DEV), torch.zeros(8, device=DEV)
    with pytest.raises(TypeError, match="params"):
        train.AdamW([p.half()], [g])
    with pytest.raises(TypeError, match="params"):
        train.AdamW([torch.zeros(4, 4, device=DEV).t()[:, :2]], [g])
    with pytest.raises(ValueError, match="shapes"):
        train.AdamW([p], [g[:4]])
    with pytest.raises(TypeError, match="gradients"):
        train.AdamW([p], [g.half()])
    with pytest.raises(TypeError, match="copies"):
        train.AdamW([p], [g], copies=[torch.zeros(8, device=DEV)])
    with pytest.raises(ValueError, match="share memory"):
        train.AdamW([p, p[4:]], [g, g[4:]])
    with pytest.raises(ValueError, match="weight_decay"):
        train.AdamW([p], [g], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError, match="exp_avg"):
        train.AdamW([p], [g], state={"step": 0, "exp_avg": g, "exp_avg_sq": g})
    with pytest.raises(train.LpError, match="INVALID"):
        train.AdamW([p], [g], betas=(0.9, 1.0)).step()
    with pytest.raises(train.LpError, match="INVALID"):
        train.AdamW([p], [p])
