"""The layer norm and its backward pass on a GB300 against the fp64 oracle.

Tolerances, with u = 2^-24 (float32 arithmetic).  A row's sum is a tree whose longest chain is at most
17 + 9 additions (a thread's 16 pairs, then lanes and warps), 32 u of its terms' magnitudes.  So the
mean is within em = 36 u mean|r'| (r' is rounded once, the mean twice more); a deviation within
ed = u |r'| + em + u |dev|; the variance within 36 u of itself, what the deviations' errors add
(2 mean(|dev| u |r'|), the mean's error entering squared), so the root within half of that relatively,
and 4 u.  h adds three operations and the rounding of its type (bfloat16: 2^-8 of the value).  The
backward's sums have the same chains; its products add up to 6 u of each term.  A sum over T rows is a
chain of at most T + 64 additions."""

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import autograd, tune
from oracle import tune as ot

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def half_ulp(dtype):
    return 2.0 ** -8 if dtype == BF16 else U


def host(t):
    return None if t is None else t.double().cpu().numpy()


def rows(g, T, d, dtype, pad=0, scale=1.0, shift=0):
    """[T, d] with a row stride of d + pad, starting `shift` elements into its memory."""
    base = torch.randn(T * (d + pad) + shift + 8, generator=g, device=DEV) * scale
    return base.to(dtype)[shift:shift + T * (d + pad)].view(T, d + pad)[:, :d]


def make(T, d, residual=BF16, act=BF16, weight=F32, branch=True, affine="wb", pad=0, shift=0, offset=0.5):
    g = torch.Generator(device=DEV).manual_seed(1000 * T + d)
    x = {"residual": (rows(g, T, d, residual, pad, shift=shift) + offset).to(residual)}
    if pad or shift:
        x["residual"] = rows(g, T, d, residual, pad, shift=shift).add_(offset)
    if branch:
        x["branch"] = rows(g, T, d, act, pad, 0.8, shift)
    else:
        act = residual
    if "w" in affine:
        x["weight"] = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(weight)
    if "b" in affine:
        x["bias"] = (0.3 * torch.randn(d, generator=g, device=DEV)).to(weight)
    return x, (rows(g, T, d, act, pad, 0.1, shift), rows(g, T, d, residual, pad, 0.1, shift))


def check_forward(x, eps=1e-5):
    out = tune.layer_norm(eps=eps, **x)
    ref = ot.layer_norm(**{k: host(v) for k, v in x.items()}, eps=eps)
    act = x.get("branch", x["residual"]).dtype
    assert out.normed.dtype == act and out.residual.dtype == x["residual"].dtype
    size = np.abs(host(x["residual"])) + (np.abs(host(x["branch"])) if "branch" in x else 0.0)
    if "branch" in x:
        err = np.abs(host(out.residual) - ref[1])
        assert np.all(err <= (U + half_ulp(out.residual.dtype) * 1.01) * np.abs(ref[1]))
    else:
        assert out.residual is x["residual"]
    em = 36 * U * size.mean(1)
    assert np.all(np.abs(host(out.mean) - ref[2]) <= em)
    dev = np.abs(ref[1] - ref[2][:, None])
    ed = U * size + em[:, None] + U * dev
    var = (dev * dev).mean(1)
    ev = 36 * U * var + 2 * (dev * U * size).mean(1) + em * em
    er = 0.51 * ev / (var + eps) + 4 * U  # relative, of the root
    assert np.all(np.abs(host(out.rstd) - ref[3]) <= er * ref[3])
    w = np.abs(host(x["weight"])) if "weight" in x else 1.0
    b = np.abs(host(x["bias"])) if "bias" in x else 0.0
    hat = dev * ref[3][:, None] * w
    near = ed * ref[3][:, None] * w * 1.01 + hat * (er[:, None] + 4 * U) + U * (hat + b)
    assert np.all(np.abs(host(out.normed) - ref[0]) <= near + half_ulp(act) * 1.01 * (np.abs(ref[0]) + near))
    return out


def check_backward(x, grads, out, with_residual=True, weight_grads=True):
    dh, dr = grads
    dr = dr if with_residual else None
    got = tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd, weight=x.get("weight"),
                                   bias=x.get("bias"), branch="branch" in x, weight_grads=weight_grads)
    ref = ot.layer_norm_backward(host(dh), host(dr), host(out.residual), host(out.mean), host(out.rstd),
                                 weight=host(x.get("weight")))
    root = host(out.rstd)[:, None]
    xh = np.abs((host(out.residual) - host(out.mean)[:, None]) * root)
    dx = np.abs(host(dh)) * (np.abs(host(x["weight"])) if "weight" in x else 1.0)
    m0, m1 = dx.mean(1, keepdims=True), (dx * xh).mean(1, keepdims=True)
    near = root * (44 * U * (m0 + xh * m1) + 6 * U * dx) + (0 if dr is None else 4 * U * np.abs(host(dr)))
    for g, dtype in ((got.residual, out.residual.dtype), (got.branch, dh.dtype)):
        if g is None:
            assert "branch" not in x
            continue
        assert g.dtype == dtype
        assert np.all(np.abs(host(g) - ref[0]) <= near + half_ulp(dtype) * 1.01 * (np.abs(ref[0]) + near))
    if "branch" in x:
        assert (got.branch is got.residual) == (dh.dtype == out.residual.dtype)
    T = dh.shape[0]
    for name, g, want, terms in (("weight", got.weight, ref[1], np.abs(host(dh)) * xh),
                                 ("bias", got.bias, ref[2], np.abs(host(dh)))):
        assert (g is not None) == (name in x and weight_grads)
        if g is not None:
            assert g.dtype == F32
            assert np.all(np.abs(host(g) - want) <= (T + 68) * U * terms.sum(0))
    return got


@pytest.mark.parametrize("residual,act", [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 2), (2, 8), (5, 255), (7, 256), (1, 4096), (40, 264), (9, 4104),
                                 (3, 8192), (2, 8200), (5, 16384), (3, 12295)])
def test_types_and_sizes(T, d, residual, act):
    x, grads = make(T, d, residual, act)
    check_backward(x, grads, check_forward(x))


@pytest.mark.parametrize("affine", ["", "w", "b", "wb"])
@pytest.mark.parametrize("branch", [False, True])
@pytest.mark.parametrize("weight", [F32, BF16])
def test_optional_parts(affine, branch, weight):
    x, grads = make(33, 520, F32 if branch else BF16, BF16, weight, branch, affine)
    out = check_forward(x, eps=1e-3)
    check_backward(x, grads, out, with_residual=False)
    check_backward(x, grads, out, weight_grads=False)


@pytest.mark.parametrize("residual,act", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,d,pad,shift", [(17, 1000, 8, 8), (17, 1000, 3, 0), (17, 1001, 0, 0), (17, 1001, 3, 1),
                                           (300, 77, 2, 2), (6, 9001, 0, 3), (6, 5001, 1, 1), (11, 2048, 0, 4)])
def test_strides_and_alignment(T, d, pad, shift, residual, act):
    x, grads = make(T, d, residual, act, pad=pad, shift=shift)
    check_backward(x, grads, check_forward(x))


@pytest.mark.parametrize("T,d,dtype", [(1300, 1024, BF16), (2100, 256, F32), (700, 4096, BF16), (400, 6000, BF16),
                                       (320, 9000, F32), (5000, 40, BF16), (611, 2047, BF16)])
def test_several_turns(T, d, dtype):
    """Several rows of a team, the last turn ragged."""
    x, grads = make(T, d, dtype, dtype)
    check_backward(x, grads, check_forward(x))


@pytest.mark.parametrize("d", [1, 7, 4096, 10000])
def test_rows_without_spread(d):
    """Rows whose elements are all equal: the deviations are what rounding of the mean leaves, and the
    root is eps's."""
    x = torch.full((3, d), 2.5, device=DEV)
    out = tune.layer_norm(x, eps=1e-2, weight=torch.ones(d, device=DEV), bias=torch.full((d,), 0.25, device=DEV))
    assert np.all(np.abs(host(out.rstd) - 10.0) <= 10 * 8 * U + 10 * (36 * U * 2.5) ** 2 / 1e-2)
    assert np.all(np.abs(host(out.normed) - 0.25) <= 10 * 36 * U * 2.5 * 1.01 + 4 * U)


def test_offset_far_above_the_spread():
    """A row's mean a thousand times its spread: the squares are of the deviations, so the root keeps
    the precision that check_forward derives."""
    x, grads = make(8, 4096, F32, F32, offset=1000.0)
    check_backward(x, grads, check_forward(x))


@pytest.mark.parametrize("d", [1000, 4096, 9000])
def test_a_row_has_the_bits_that_it_has_alone(d):
    x, (dh, dr) = make(37, d)
    out = tune.layer_norm(**x)
    grads = tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd, weight=x["weight"])
    for t in (0, 5, 36):
        one = {k: v[t:t + 1] if v.dim() == 2 else v for k, v in x.items()}
        alone = tune.layer_norm(**one)
        for a, b in zip(out, alone):
            assert torch.equal(a[t:t + 1], b)
        g = tune.layer_norm_backward(dh[t:t + 1], dr[t:t + 1], alone.residual, alone.mean, alone.rstd,
                                     weight=x["weight"])
        assert torch.equal(grads.residual[t:t + 1], g.residual)


def test_not_finite_rows_stay_their_own():
    x, (dh, dr) = make(20, 600)
    good = tune.layer_norm(**x)
    good_g = tune.layer_norm_backward(dh, dr, good.residual, good.mean, good.rstd, weight=x["weight"])
    x["residual"][3, 7] = float("nan")
    x["branch"][11, 0] = float("inf")
    out = tune.layer_norm(**x)
    got = tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd, weight=x["weight"])
    others = [t for t in range(20) if t not in (3, 11)]
    assert torch.equal(out.normed[others], good.normed[others])
    assert torch.equal(got.residual[others], good_g.residual[others])
    assert torch.isnan(out.normed[3]).all() and torch.isnan(out.mean[3])
    assert torch.isnan(out.rstd[11])


def test_in_place_and_repeats():
    x, (dh, dr) = make(70, 1500, F32, BF16)
    ref = tune.layer_norm(**x)
    again = tune.layer_norm(**x)
    assert all(torch.equal(a, b) for a, b in zip(ref, again))
    stream, version = x["residual"].clone(), None
    version = stream._version
    out = tune.layer_norm(stream, x["branch"], weight=x["weight"], bias=x["bias"], in_place=True)
    assert out.residual is stream and stream._version > version
    assert torch.equal(stream, ref.residual) and torch.equal(out.normed, ref.normed)
    kw = dict(weight=x["weight"], bias=x["bias"], branch=True)
    a = tune.layer_norm_backward(dh, dr, ref.residual, ref.mean, ref.rstd, **kw)
    b = tune.layer_norm_backward(dh, dr, ref.residual, ref.mean, ref.rstd, **kw)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_no_rows():
    x = torch.zeros(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    out = tune.layer_norm(x, x, weight=w, bias=w)
    assert out.normed.shape == (0, 64) and out.mean.shape == (0,)
    g = tune.layer_norm_backward(x, None, out.residual, out.mean, out.rstd, weight=w, bias=w, branch=True)
    assert g.residual.shape == (0, 64) and not g.weight.any() and not g.bias.any()


def test_another_stream_and_a_graph():
    x, (dh, dr) = make(130, 2048)
    kw = dict(weight=x["weight"], bias=x["bias"], branch=True)
    ref = tune.layer_norm(**x)
    ref_g = tune.layer_norm_backward(dh, dr, ref.residual, ref.mean, ref.rstd, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = tune.layer_norm(stream=side, **x)
    got = tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip((*ref, *ref_g), (*out, *got)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tune.layer_norm(**x)
        got = tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd, **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*ref, *ref_g), (*out, *got)))


def test_given_workspace():
    x, (dh, dr) = make(300, 512)
    out = tune.layer_norm(**x)
    kw = dict(weight=x["weight"], bias=x["bias"])
    ref = tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd, **kw)
    size = tune.layer_norm_backward_workspace_size(300, 512)
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        got = tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd, workspace=ws, **kw)
        assert torch.equal(got.weight, ref.weight) and torch.equal(got.bias, ref.bias)
    with pytest.raises(tune.LpError):
        tune.layer_norm_backward(dh, dr, out.residual, out.mean, out.rstd,
                                 workspace=torch.empty(size - 256, dtype=torch.uint8, device=DEV), **kw)


def test_refusals():
    x, (dh, dr) = make(6, 64)
    out = tune.layer_norm(**x)
    back = lambda **kw: tune.layer_norm_backward(  # noqa: E731
        **{**dict(grad_normed=dh, grad_residual=dr, residual=out.residual, mean=out.mean, rstd=out.rstd), **kw})
    with pytest.raises(ValueError, match="2-D"):
        tune.layer_norm(x["residual"][0])
    with pytest.raises(ValueError, match="branch must have the shape"):
        tune.layer_norm(x["residual"], x["branch"][:3])
    with pytest.raises(ValueError, match="contiguous rows"):
        tune.layer_norm(x["residual"].t().contiguous().t())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        tune.layer_norm(x["residual"].half())
    with pytest.raises(TypeError, match="one dtype"):
        tune.layer_norm(x["residual"], weight=x["weight"], bias=x["bias"].bfloat16())
    with pytest.raises(ValueError, match="weight must be"):
        tune.layer_norm(x["residual"], weight=x["weight"][:32])
    with pytest.raises(tune.LpError):
        tune.layer_norm(x["residual"], eps=-1.0)
    with pytest.raises(tune.LpError):  # rows that share memory, written in place
        tune.layer_norm(x["residual"][:1].expand(6, 64), x["branch"], in_place=True)
    with pytest.raises(tune.LpError):
        tune.layer_norm(torch.zeros(1, 16385, device=DEV))
    with pytest.raises(TypeError, match="without a branch"):
        back(grad_normed=dh.float())
    with pytest.raises(TypeError, match="grad_residual must be"):
        back(grad_residual=dr.float())
    with pytest.raises(ValueError, match="mean must be"):
        back(mean=out.mean[:3])
    with pytest.raises(ValueError, match="CUDA"):
        back(rstd=out.rstd.cpu())
    with pytest.raises(TypeError, match="mean must be a tensor"):
        back(mean=None)


@pytest.mark.parametrize("branch", [False, True])
def test_autograd(branch):
    """The binding's gradients are the call's, in the inputs' dtypes, and those of differences."""
    x, grads = make(12, 96, F32, F32, F32, branch)
    leaves = {k: v.clone().requires_grad_() for k, v in x.items()}
    h, r = autograd.layer_norm(leaves["residual"], leaves.get("branch"), weight=leaves["weight"], bias=leaves["bias"])
    torch.autograd.backward((h, r), grads)
    out = tune.layer_norm(**x)
    want = tune.layer_norm_backward(*grads, out.residual, out.mean, out.rstd, weight=x["weight"], bias=x["bias"],
                                    branch=branch)
    if branch:
        assert torch.equal(leaves["residual"].grad, want.residual)
        assert torch.equal(leaves["branch"].grad, want.residual)
        assert leaves["branch"].grad.data_ptr() != leaves["residual"].grad.data_ptr()
    assert torch.equal(leaves["weight"].grad, want.weight) and torch.equal(leaves["bias"].grad, want.bias)
    # central differences of the oracle's loss along a direction, its error of order step^2
    at = {k: host(v) for k, v in x.items()}

    def loss(v):
        n, new, _, _ = ot.layer_norm(**v)
        return (n * host(grads[0])).sum() + (new * host(grads[1])).sum()

    rng = np.random.default_rng(3)
    for k in at:
        way, step = rng.standard_normal(at[k].shape), 1e-5
        slope = (loss({**at, k: at[k] + step * way}) - loss({**at, k: at[k] - step * way})) / (2 * step)
        assert abs((host(leaves[k].grad) * way).sum() - slope) <= 1e-5 * np.abs(host(leaves[k].grad) * way).sum()


def test_autograd_dtypes_and_second_order():
    x, _ = make(9, 128, F32, BF16, BF16)
    leaves = {k: v.clone().requires_grad_() for k, v in x.items()}
    h, r = autograd.layer_norm(leaves["residual"], leaves["branch"], weight=leaves["weight"], bias=leaves["bias"])
    h.float().sum().backward()
    assert all(v.grad.dtype == v.dtype and v.grad.shape == v.shape for v in leaves.values())
    h, r = autograd.layer_norm(leaves["residual"], leaves["branch"], weight=leaves["weight"])
    r.sum().backward()  # the norm's gradient is zero: the stream's passes through
    g, = torch.autograd.grad(autograd.layer_norm(leaves["residual"])[0].sum(), leaves["residual"], create_graph=True)
    with pytest.raises(RuntimeError, match="gradient of a gradient"):
        g.sum().backward()


@pytest.mark.parametrize("branch", [False, True])
@pytest.mark.parametrize("residual,act", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,d", [(3, 8), (700, 248), (5, 512), (333, 520), (2500, 1024), (411, 4096), (401, 5000),
                                 (200, 8192), (160, 8200)])
def test_alignment_does_not_show(T, d, residual, act, branch):
    """Rows of whole groups and the same rows at an odd pitch, one column on: the same bits, whichever kernel."""
    if not branch and residual != act:
        return
    g = torch.Generator(device=DEV).manual_seed(T + d)
    r = torch.randn(T, d, generator=g, device=DEV).to(residual)
    y = torch.randn(T, d, generator=g, device=DEV).to(act) if branch else None
    w, b = torch.randn(2, d, generator=g, device=DEV)

    def odd(t):
        if t is None:
            return None
        wide = torch.zeros(T, d + 3, device=DEV, dtype=t.dtype)
        wide[:, 1:d + 1] = t
        return wide[:, 1:d + 1]

    for affine in (dict(weight=w, bias=b), dict(weight=w.to(BF16)), dict(bias=b), dict()):
        want = tune.layer_norm(r, y, **affine)
        got = tune.layer_norm(odd(r), odd(y), **{k: torch.cat([v[:1], v])[1:] for k, v in affine.items()})
        for u, v in zip(got, want):
            assert torch.equal(u, v)
