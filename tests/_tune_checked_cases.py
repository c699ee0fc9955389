"""Small cases of the fine-tuning operators for the checked-build test: run with the normal library in the test
process and with the checked one in a child."""

from __future__ import annotations

import torch

DEV = "cuda:0"


def run_cases(tune) -> dict:
    out = {}

    def keep(name, *ts):
        for i, t in enumerate(ts):
            if t is not None:
                out[f"{name}.{i}"] = t.detach().contiguous().view(-1).view(torch.uint8).cpu()

    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    for T, d, pad, kinds in [(9, 264, 0, "bb"), (5, 101, 3, "ff"), (3, 5000, 0, "fb"), (2, 9001, 0, "ff"),
                             (700, 64, 8, "bb"), (400, 1200, 0, "fb"), (1, 4096, 0, "bf"), (311, 515, 0, "bb")]:
        types = [torch.bfloat16 if k == "b" else torch.float32 for k in kinds]
        rows = lambda k: r(T, d + pad).to(types[k])[:, :d]  # noqa: E731
        x, y, w, b = rows(0), rows(1), r(d), r(d)
        o = tune.layer_norm(x, y, weight=w, bias=b)
        keep(f"norm{T}x{d}", *o)
        keep(f"norm{T}x{d}.back", *tune.layer_norm_backward(rows(1), rows(0), o.residual, o.mean, o.rstd, weight=w,
                                                            bias=b, branch=True))
        keep(f"norm{T}x{d}.alone", *tune.layer_norm(y))
    for lengths in ([3, 0, 60, 5], [3000, 17, 9000, 1], [1] * 5000, [40000, 700]):
        cu = torch.tensor([0] + lengths, device=DEV).cumsum(0) + 3
        T = int(cu[-1]) + 5
        logp, mask = -r(T).abs(), r(T) > -0.5
        for kind in ("sigmoid", "hinge", "square"):
            keep(f"preference{T}.{kind}", *tune.preference_loss(logp, cu, ref_logp=logp + 0.1 * r(T), mask=mask,
                                                                kind=kind, nll_coef=0.1))
        keep(f"preference{T}.halves", *tune.preference_loss(logp, cu, halves=True, average=True))
    cu = torch.tensor([50, -7, 1 << 40, 3, 20000, 11, 9], device=DEV)  # no offsets: the call ends
    tune.preference_loss(-r(12000).abs(), cu)
    for shapes, cut in [([(130, 200), (64, 64), (1, 9), (300, 40), (0, 3)], 0), ([(130, 200), (257, 31)], 1),
                        ([(1030, 1100)], 0), ([(120, 2050), (2050, 120)], 0), ([(256, 256)] * 70, 0)]:
        flat = lambda n: r(n + cut)[cut:]  # noqa: E731
        params = [0.02 * flat(a * b).view(a, b) for a, b in shapes]
        grads = [r(a * b + cut).bfloat16()[cut:].view(a, b) for a, b in shapes]
        copies = [torch.zeros(a * b + cut, device=DEV, dtype=torch.bfloat16)[cut:].view(a, b) for a, b in shapes]
        opt = tune.Muon(params, grads, copies=copies, weight_decay=0.1)
        opt.step()
        opt.step()
        keep(f"muon{shapes[0]}{len(shapes)}.{cut}", opt.momentum_buffer, *params[:8], *copies[:8])
    torch.cuda.synchronize()
    return out
