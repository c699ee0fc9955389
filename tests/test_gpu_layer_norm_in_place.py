"""The layer norm over its own inputs, and its backward's bits by alignment, on a GB300.

The in-place forms have the bits of the others: residual_out over residual in both of the forward's kernels, rows of
whole groups and others, grad_residual over grad_residual_out, with more rows than the CTAs take in one turn.  The
backward's results do not depend on how rows lie either."""

import ctypes

import pytest
import torch

from invariant_token_logprobs_gb300 import lp, tune

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)]
# several turns of every kernel, and one
SIZES = [(2500, 1024), (5000, 256), (700, 4096), (500, 8192), (400, 9000), (330, 16384), (3, 4096), (1, 640),
         (400, 2047), (3000, 77), (340, 9001), (2, 1001)]


def rows(g, T, d, dtype, pad=0, shift=0):
    """[T, d] with a row stride of d + pad, starting `shift` elements into its memory."""
    base = torch.randn(T * (d + pad) + shift + 8, generator=g, device=DEV).to(dtype)
    return base[shift:shift + T * (d + pad)].view(T, d + pad)[:, :d]


def whole(t):
    """The memory that t's rows lie in, what is between them too."""
    return t.as_strided((t.untyped_storage().nbytes() // t.element_size(),), (1,), 0)


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 0), (3, 1), (2, 2)])
@pytest.mark.parametrize("residual,act", TYPES)
@pytest.mark.parametrize("T,d", SIZES)
def test_forward(T, d, residual, act, pad, shift):
    g = torch.Generator(device=DEV).manual_seed(T + d)
    r, y = rows(g, T, d, residual, pad, shift), rows(g, T, d, act, pad, shift)
    w, b = torch.randn(2, d, generator=g, device=DEV)
    want = tune.layer_norm(r, y, weight=w, bias=b)
    before = whole(r).clone()
    got = tune.layer_norm(r, y, weight=w, bias=b, in_place=True)
    assert got.residual is r
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    r.copy_(torch.as_strided(before, r.shape, r.stride(), r.storage_offset()))
    assert torch.equal(whole(r), before)  # nothing between the rows was written


def backward(x, out, mean, rstd, dh, dr, grad, branch, weight_grads, workspace):
    """lp_layer_norm_backward into `grad` and, where it is one, `branch`."""
    code = lambda t: 1 if t.dtype == BF16 else 0  # noqa: E731
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    ld = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    T, d = out.shape
    status = tune.load().lp_layer_norm_backward(
        at(out), ld(out), code(out), code(dh), at(x["weight"]), code(x["weight"]), T, d, at(mean), at(rstd), at(dh), ld(dh),
        at(dr), ld(dr), at(grad), ld(grad), at(branch), ld(branch), at(weight_grads[0]), at(weight_grads[1]), at(workspace),
        workspace.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    lp._check("lp_layer_norm_backward", status)


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 0), (3, 1), (2, 2)])
@pytest.mark.parametrize("residual,act", TYPES)
@pytest.mark.parametrize("T,d", SIZES)
def test_backward(T, d, residual, act, pad, shift):
    g = torch.Generator(device=DEV).manual_seed(T + d)
    out, dh, dr = rows(g, T, d, residual, pad, shift), rows(g, T, d, act, pad, shift), rows(g, T, d, residual, pad, shift)
    x = {"weight": torch.randn(d, generator=g, device=DEV)}
    mean, rstd = out.float().mean(1), 1 / (out.float().std(1, unbiased=False) + 0.1)
    want = tune.layer_norm_backward(dh, dr, out, mean, rstd, weight=x["weight"], bias=x["weight"], branch=True)
    before = whole(dr).clone()
    sums = torch.empty(2, d, device=DEV)
    branch = None if act == residual else torch.empty_like(dh)
    ws = torch.empty(tune.layer_norm_backward_workspace_size(T, d), dtype=torch.uint8, device=DEV)
    backward(x, out, mean, rstd, dh, dr, dr, branch, sums, ws)
    assert torch.equal(dr, want.residual)
    assert branch is None or torch.equal(branch, want.branch)
    assert torch.equal(sums[0], want.weight) and torch.equal(sums[1], want.bias)
    dr.copy_(torch.as_strided(before, dr.shape, dr.stride(), dr.storage_offset()))
    assert torch.equal(whole(dr), before)


@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("residual,act", TYPES)
@pytest.mark.parametrize("T,d", [(3, 8), (700, 248), (5, 512), (333, 520), (2500, 1024), (411, 4096), (401, 5000), (200, 8192),
                                 (160, 8200), (1, 640), (330, 16384)])
def test_backward_alignment_does_not_show(T, d, residual, act, with_residual):
    """Rows of whole groups and the same rows at odd pitches and places: the same bits, the sums over rows too."""
    g = torch.Generator(device=DEV).manual_seed(T + d)
    out, dh = torch.randn(T, d, generator=g, device=DEV).to(residual), torch.randn(T, d, generator=g, device=DEV).to(act)
    dr = torch.randn(T, d, generator=g, device=DEV).to(residual) if with_residual else None
    w, b = torch.randn(2, d, generator=g, device=DEV)
    mean, rstd = out.float().mean(1), 1 / (out.float().std(1, unbiased=False) + 0.1)

    def moved(t, pad, shift):
        if t is None:
            return None
        wide = torch.zeros(T, d + pad, device=DEV, dtype=t.dtype)
        wide[:, shift:d + shift] = t
        return wide[:, shift:d + shift]

    for affine in (dict(weight=w, bias=b), dict(weight=w.to(BF16)), dict(bias=b), dict()):
        want = tune.layer_norm_backward(dh, dr, out, mean, rstd, branch=True, **affine)
        for pad, shift in ((3, 1), (2, 2), (1, 0)):
            got = tune.layer_norm_backward(moved(dh, pad, shift), moved(dr, pad, shift), moved(out, pad, shift), mean, rstd,
                                           branch=True, **{k: torch.cat([v[:1], v])[1:] for k, v in affine.items()})
            for u, v in zip(got, want):
                assert (u is None) == (v is None) and (u is None or torch.equal(u, v))
