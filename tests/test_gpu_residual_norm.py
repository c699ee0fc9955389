"""The residual norm and its backward pass on a GB300 against the fp64 oracle.

Tolerances, with u = 2^-24 (float32 arithmetic): a sum of squares is a tree whose longest
chain is at most 64 + 16 additions (the elements of one thread, then shuffles and warps) of terms
rounded once, so rstd is within (80 + 4) / 2 u < 64 u relatively.  An element of the new stream
is four rounded operations on its two terms: 8 u (|a r| + |b g n|), the branch's root adding 64 u
of the second.  h adds rstd's 64 u and two products: 72 u |h|.  A bfloat16 output adds half a unit
in its last place, 2^-8 relatively.  The gradients' bounds follow the same terms in magnitude."""

import numpy as np
import pytest
import torch

from invariant_token_logprobs_gb300 import train
from oracle import train as ot

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


def make(T, d, residual, act, weight, post, gate, norm=True, branch=True, pad=0, shift=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000 * T + d)
    x = {"residual": rows(g, T, d, residual, pad, shift=shift)}
    if branch:
        x["branch"] = rows(g, T, d, act, pad, 0.8, shift)
    if norm:
        x["weight"] = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(weight)
    if post:
        x["branch_weight"] = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(weight)
    if gate == "channel":
        x["gate"] = torch.randn(d, generator=g, device=DEV).to(act)
    elif gate == "token":
        x["gate"] = rows(g, T, d, act, pad, shift=shift)
    x["grads"] = (rows(g, T, d, act, pad, 0.1, shift), rows(g, T, d, residual, pad, 0.1, shift))
    return x


def split(x):
    kw = {k: v for k, v in x.items() if k not in ("residual", "grads")}
    return x["residual"], kw


def check_forward(x, a, b, eps):
    residual, kw = split(x)
    out = train.residual_norm(residual, residual_scale=a, branch_scale=b, eps=eps, **kw)
    ref = ot.residual_norm(host(residual), **{k: host(v) for k, v in kw.items()}, residual_scale=a,
                           branch_scale=b, eps=eps)
    terms = np.abs(a * host(residual)) + np.abs(ref[1] - a * host(residual))
    if "branch" in kw:
        err = np.abs(host(out.residual) - ref[1])
        assert np.all(err <= 72 * U * terms + half_ulp(residual.dtype) * np.abs(ref[1]))
    else:
        assert out.residual is residual
    if "weight" in kw:
        act = kw.get("branch", residual).dtype
        assert out.normed.dtype == act
        near = 72 * U * np.abs(ref[0]) + \
            72 * U * terms * ref[2][:, None] * np.abs(host(kw["weight"]))
        # what the stream's own error adds to the row's root
        near = near + np.abs(ref[0]) * 72 * U * np.max(terms * ref[2][:, None], axis=1, keepdims=True)
        assert np.all(np.abs(host(out.normed) - ref[0]) <= near + half_ulp(act) * np.abs(ref[0]) * 1.01)
        limit = 64 * U * ref[2] * (1 + 2 * np.max(terms * ref[2][:, None], axis=1))
        assert np.all(np.abs(host(out.rstd) - ref[2]) <= limit)
    else:
        assert out.normed is None and out.rstd is None
    if "branch_weight" in kw:
        assert np.all(np.abs(host(out.branch_rstd) - ref[3]) <= 64 * U * ref[3])
    else:
        assert out.branch_rstd is None
    return out


def check_backward(x, out, a, b, with_residual=True):
    residual, kw = split(x)
    gh, gr = x["grads"]
    gh = gh if "weight" in kw else None
    gr = gr if with_residual else None
    got = train.residual_norm_backward(gh, gr, out.residual, out.rstd, branch_rstd=out.branch_rstd,
                                       residual_scale=a, branch_scale=b, **kw)
    # the oracle takes what the kernel took: the kept stream and roots
    h = {k: host(v) for k, v in kw.items()}
    ref = ot.residual_norm_backward(host(gh), host(gr), host(out.residual), host(out.rstd),
                                    branch_rstd=host(out.branch_rstd), residual_scale=a,
                                    branch_scale=b, **h)
    T, d = residual.shape
    # magnitudes of the terms: D, then what each gradient sums or multiplies
    D = 0.0 if gr is None else np.abs(host(gr))
    if gh is not None:
        x_hat = np.abs(host(out.residual) * host(out.rstd)[:, None])
        v = np.abs(host(gh) * h["weight"])
        D = D + host(out.rstd)[:, None] * (v + x_hat * np.mean(x_hat * v, axis=1, keepdims=True))
    mags = [np.abs(a) * D]
    if "branch" in kw:
        y_hat = np.abs(h["branch"])
        if "branch_weight" in kw:
            y_hat = y_hat * host(out.branch_rstd)[:, None]
        n = y_hat * np.abs(h.get("branch_weight", 1.0))
        e = b * D * np.abs(h.get("gate", 1.0))
        v = e * np.abs(h.get("branch_weight", 1.0))
        m = v
        if "branch_weight" in kw:
            m = host(out.branch_rstd)[:, None] * (v + y_hat * np.mean(v * y_hat, axis=1, keepdims=True))
        mags += [m]
    # a row's elements pass at most ~30 roundings and two sums of 80 (the sum over the branch
    # holds the first inside it): 256 u of the terms; sums over T rows add a chain of T
    for name, grad, want, mag in zip(("residual", "branch"), (got.residual, got.branch), ref, mags):
        assert np.all(np.abs(host(grad) - want) <= 256 * U * mag + half_ulp(grad.dtype) * np.abs(want)), name
    if "branch" not in kw:
        assert got.branch is None
    sums = {"weight": (None if gh is None else np.sum(np.abs(host(gh)) * x_hat, axis=0), ref[2])}
    if "branch" in kw:
        sums["branch_weight"] = (np.sum(e * y_hat, axis=0) if "branch_weight" in kw else None, ref[3])
        if "gate" in kw:
            terms = b * D * n
            sums["gate"] = (terms if kw["gate"].dim() == 2 else terms.sum(axis=0), ref[4])
    for name, (mag, want) in sums.items():
        grad = getattr(got, name)
        if mag is None or want is None:
            assert grad is None, name
            continue
        limit = (256 + (T if grad.dim() == 1 else 0)) * U * mag
        assert np.all(np.abs(host(grad) - want) <= limit + half_ulp(grad.dtype) * np.abs(want)), name
    return got


PARTS = [  # post norm, gate, norm
    (False, None, True), (True, "channel", True), (True, "token", True), (False, "channel", False),
    (True, None, False), (False, "token", True),
]


@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (5, 64), (2, 255), (33, 256), (7, 1000), (9, 2047),
                                 (4, 2560), (160, 4096), (3, 5000), (5, 8192), (3, 12288), (2, 16384),
                                 (3, 16383)])
@pytest.mark.parametrize("post,gate,norm", PARTS)
def test_sizes_and_parts(T, d, post, gate, norm):
    x = make(T, d, BF16, BF16, BF16, post, gate, norm)
    check_backward(x, check_forward(x, 1.0, 0.5, 1e-6), 1.0, 0.5)


@pytest.mark.parametrize("residual,act,weight", [(F32, F32, F32), (F32, BF16, BF16), (BF16, F32, BF16),
                                                 (BF16, BF16, F32)])
@pytest.mark.parametrize("T,d", [(6, 264), (70, 1536), (2, 9000)])
def test_types(residual, act, weight, T, d):
    x = make(T, d, residual, act, weight, True, "channel")
    check_backward(x, check_forward(x, 0.9, 0.7, 1e-5), 0.9, 0.7)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_strides_and_alignment_keep_the_bits(pad, shift, gate):
    plain = make(19, 520, BF16, BF16, BF16, True, gate, seed=4)
    ref = check_forward(plain, 1.0, 0.5, 1e-6)
    grads = check_backward(plain, ref, 1.0, 0.5)
    x = {}
    for k, v in plain.items():
        def moved(t):
            if t.dim() == 1:
                out = torch.empty(520 + shift, dtype=t.dtype, device=DEV)[shift:]
            else:
                out = torch.empty(19 * (520 + pad) + shift, dtype=t.dtype, device=DEV)[shift:] \
                    .view(19, 520 + pad)[:, :520]
            return out.copy_(t)
        x[k] = tuple(moved(t) for t in v) if k == "grads" else moved(v)
    out = check_forward(x, 1.0, 0.5, 1e-6)
    for a, b in zip(out, ref):
        assert torch.equal(a, b)
    for a, b in zip(check_backward(x, out, 1.0, 0.5), grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("residual", [BF16, F32])
@pytest.mark.parametrize("d", [1, 7, 255, 257, 1031, 4099])
def test_rows_in_the_middle_of_a_word(d, residual):
    """Rows at odd places, between NaN, have the bits that they have on boundaries of 16 columns."""
    x = make(9, d, residual, BF16, BF16, True, "channel", seed=5)

    def placed(t, ld, shift):
        rows_of = t.view(1, -1) if t.dim() == 1 else t
        out = torch.full((rows_of.shape[0] * ld + shift,), float("nan"), dtype=t.dtype, device=DEV)
        out = out[shift:].view(-1, ld)[:, :d]
        out.copy_(rows_of)
        return out[0] if t.dim() == 1 else out

    def run(ld, shift):
        at = {k: tuple(placed(t, ld, shift) for t in v) if k == "grads" else placed(v, ld, shift)
              for k, v in x.items()}
        out = check_forward(at, 1.0, 0.5, 1e-6)
        return list(out) + list(check_backward(at, out, 1.0, 0.5))

    boundaries = run((d + 15) // 16 * 16, 0)
    for ld, shift in ((d | 1, 0), (d | 1, 1), (d + 3 & ~1, 1)):
        for a, b in zip(run(ld, shift), boundaries):
            assert (a is None and b is None) or torch.equal(a, b)


def test_without_branch_and_without_residual_gradient():
    x = make(11, 768, BF16, BF16, F32, False, None, branch=False)
    check_backward(x, check_forward(x, 1.0, 1.0, 1e-6), 1.0, 1.0, with_residual=False)
    x = make(11, 768, F32, BF16, F32, True, None)
    check_backward(x, check_forward(x, 1.0, 1.0, 1e-6), 1.0, 1.0, with_residual=False)


def test_no_rows():
    x = make(0, 96, BF16, BF16, BF16, True, "channel")
    residual, kw = split(x)
    out = train.residual_norm(residual, **kw)
    assert out.normed.shape == out.residual.shape == (0, 96) and out.rstd.shape == (0,)
    got = train.residual_norm_backward(*x["grads"], out.residual, out.rstd,
                                       branch_rstd=out.branch_rstd, **kw)
    assert got.residual.shape == (0, 96)
    for s in (got.weight, got.branch_weight, got.gate):
        assert torch.equal(s, torch.zeros(96, device=DEV))


def test_rows_do_not_depend_on_the_batch():
    """A row's bits are those it has alone, forward and backward (the framework's property)."""
    for d in (96, 1000, 4096, 9000):
        x = make(40, d, BF16, BF16, BF16, True, "token", seed=9)
        residual, kw = split(x)
        out = train.residual_norm(residual, **kw)
        grads = train.residual_norm_backward(*x["grads"], out.residual, out.rstd,
                                             branch_rstd=out.branch_rstd, **kw)
        for first, last in ((0, 1), (39, 40), (7, 24)):
            cut = lambda t: t[first:last] if t.shape[0] == 40 else t  # noqa: E731
            k = {n: cut(v) for n, v in kw.items()}
            part = train.residual_norm(cut(residual), **k)
            for a, b in zip(part, out):
                assert torch.equal(a, cut(b))
            g = train.residual_norm_backward(*map(cut, x["grads"]), part.residual, part.rstd,
                                             branch_rstd=part.branch_rstd, **k)
            for a, b in ((g.residual, grads.residual), (g.branch, grads.branch), (g.gate, grads.gate)):
                assert torch.equal(a, cut(b))


def test_gradients_against_differences():
    """The summed gradients and a few elements of the others against central differences of the
    forward pass in float32: with a step h the quotient carries ~d u |loss| / h of rounding and
    ~h^2 of curvature, 2e-3 of the gradient's scale at h = 1e-2 for these sizes."""
    T, d, h = 4, 48, 1e-2
    x = make(T, d, F32, F32, F32, True, "channel", seed=2)
    residual, kw = split(x)
    gh, gr = (10 * t for t in x["grads"])

    def loss():
        o = train.residual_norm(residual, **kw, eps=1e-3)
        return float((o.normed.double() * gh.double()).sum() + (o.residual.double() * gr.double()).sum())

    o = train.residual_norm(residual, **kw, eps=1e-3)
    g = train.residual_norm_backward(gh, gr, o.residual, o.rstd, branch_rstd=o.branch_rstd, **kw)
    for t, grad in ((residual, g.residual), (kw["branch"], g.branch), (kw["weight"], g.weight),
                    (kw["branch_weight"], g.branch_weight), (kw["gate"], g.gate)):
        scale = float(grad.abs().max())
        for i in range(0, t.numel(), 17):
            at = (i // d, i % d) if t.dim() == 2 else i % d
            kept = float(t[at])
            t[at] = kept + h
            up, high = loss(), float(t[at])
            t[at] = kept - h
            down, low = loss(), float(t[at])
            t[at] = kept
            assert abs((up - down) / (high - low) - float(grad[at])) < 2e-3 * max(scale, 1.0)


def test_in_place_streams_graphs_and_repeats():
    x = make(64, 1024, F32, BF16, BF16, True, "channel", seed=3)
    residual, kw = split(x)
    ref = train.residual_norm(residual, **kw)
    grads = train.residual_norm_backward(*x["grads"], ref.residual, ref.rstd,
                                         branch_rstd=ref.branch_rstd, **kw)
    again = residual.clone()
    out = train.residual_norm(again, **kw, in_place=True)
    assert out.residual is again and torch.equal(again, ref.residual)
    assert torch.equal(out.normed, ref.normed)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        out = train.residual_norm(residual, **kw, stream=s)
        g = train.residual_norm_backward(*x["grads"], out.residual, out.rstd,
                                         branch_rstd=out.branch_rstd, **kw, stream=s)
        side.synchronize()
        for a, b in zip(out + g, ref + grads):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train.residual_norm(residual, **kw)
        g = train.residual_norm_backward(*x["grads"], out.residual, out.rstd,
                                         branch_rstd=out.branch_rstd, **kw)
    for _ in range(2):
        for t in out + g:
            t.zero_()
        graph.replay()
        for a, b in zip(out + g, ref + grads):
            assert torch.equal(a, b)


def test_special_values_stay_in_their_row():
    x = make(9, 640, F32, F32, F32, True, "token", seed=6)
    residual, kw = split(x)
    ref = train.residual_norm(residual, **kw)
    residual[2, 5] = float("nan")
    kw["branch"][4, 639] = float("inf")
    residual[6] = 0
    kw["branch"][6] = 0
    out = train.residual_norm(residual, **kw)
    assert torch.isnan(out.normed[2]).all() and torch.isnan(out.normed[4]).any()
    # a row of zeros norms to zero, its roots are those of eps
    assert torch.equal(out.normed[6], torch.zeros(640, device=DEV))
    assert abs(float(out.rstd[6]) - 1e3) < 1e-2 and abs(float(out.branch_rstd[6]) - 1e3) < 1e-2
    for t in (0, 1, 3, 5, 7, 8):
        assert torch.equal(out.normed[t], ref.normed[t]) and torch.equal(out.residual[t], ref.residual[t])


def test_offsets_past_32_bits():
    """Row offsets beyond 2^31 elements: the last rows are those of a call of their own."""
    T, d = 140001, 16384
    residual = torch.zeros(T, d, dtype=BF16, device=DEV)
    branch = torch.zeros(T, d, dtype=BF16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.rand(d, generator=g, device=DEV).to(BF16)
    for t in (residual, branch):
        t[-3:] = torch.randn(3, d, generator=g, device=DEV).to(BF16)
    out = train.residual_norm(residual, branch, weight=w)
    ref = train.residual_norm(residual[-3:], branch[-3:], weight=w)
    assert torch.equal(out.normed[-3:], ref.normed) and torch.equal(out.residual[-3:], ref.residual)
    assert float(out.normed[:-3].abs().max()) == 0.0
    got = train.residual_norm_backward(out.normed, out.residual, out.residual, out.rstd,
                                       branch=branch, weight=w)
    part = train.residual_norm_backward(ref.normed, ref.residual, ref.residual, ref.rstd,
                                        branch=branch[-3:], weight=w)
    assert torch.equal(got.residual[-3:], part.residual) and torch.equal(got.branch[-3:], part.branch)


@pytest.mark.parametrize("T", [1, 5, 700])
@pytest.mark.parametrize("skipped", [("gate",), ("weight", "gate"), ("branch_weight",)])
def test_sums_that_are_not_asked_for(T, skipped):
    """Through the C entry: a null sum is left out and the others keep their bits."""
    d = 520
    x = make(T, d, BF16, BF16, F32, True, "channel")
    residual, kw = split(x)
    out = train.residual_norm(residual, **kw)
    gh, gr = x["grads"]
    ref = train.residual_norm_backward(gh, gr, out.residual, out.rstd, branch_rstd=out.branch_rstd, **kw)
    sums = {k: torch.full((d,), 7.0, device=DEV) for k in ("gate", "branch_weight", "weight")}
    ptr = {k: None if k in skipped else v.data_ptr() for k, v in sums.items()}
    g, gb = torch.empty_like(residual), torch.empty_like(residual)
    size = train.residual_norm_backward_workspace_size(T, d)
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    status = train.load().lp_residual_norm_backward(
        out.residual.data_ptr(), d, 1, kw["branch"].data_ptr(), d, kw["gate"].data_ptr(), 0, 1,
        kw["branch_weight"].data_ptr(), kw["weight"].data_ptr(), 0, T, d, 1.0, 1.0,
        out.branch_rstd.data_ptr(), out.rstd.data_ptr(), gh.data_ptr(), d, gr.data_ptr(), d,
        g.data_ptr(), d, gb.data_ptr(), d, ptr["gate"], 0, ptr["branch_weight"], ptr["weight"],
        work.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    assert torch.equal(g, ref.residual) and torch.equal(gb, ref.branch)
    for k, v in sums.items():
        assert torch.equal(v, torch.full_like(v, 7.0) if k in skipped else getattr(ref, k)), k


def test_refusals():
    x = make(4, 64, BF16, BF16, BF16, True, "channel")
    residual, kw = split(x)
    with pytest.raises(ValueError, match="shape"):
        train.residual_norm(residual, kw["branch"][:3], weight=kw["weight"])
    with pytest.raises(ValueError, match="contiguous rows"):
        train.residual_norm(residual, kw["branch"].t().contiguous().t(), weight=kw["weight"])
    with pytest.raises(TypeError, match="gate"):
        train.residual_norm(residual, kw["branch"], weight=kw["weight"], gate=kw["gate"].float())
    with pytest.raises(TypeError, match="one dtype"):
        train.residual_norm(residual, kw["branch"], weight=kw["weight"].float(),
                            branch_weight=kw["branch_weight"])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        train.residual_norm(residual.half(), weight=kw["weight"])
    with pytest.raises(ValueError, match="overlap"):
        train.residual_norm(residual, kw["branch"], weight=kw["weight"],
                            gate=kw["gate"].expand(4, 64))
    with pytest.raises(train.LpError, match="INVALID"):
        train.residual_norm(residual)
    with pytest.raises(train.LpError, match="INVALID"):
        train.residual_norm(torch.zeros(1, 16385, device=DEV), weight=torch.ones(16385, device=DEV))
    with pytest.raises(TypeError, match="grad_normed"):
        train.residual_norm_backward(x["grads"][0].float(), None, residual,
                                     torch.ones(4, device=DEV), weight=kw["weight"])
