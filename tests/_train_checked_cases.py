"""Small cases of the training-step operators for the checked-build test: run with the normal
library in the test process and with the checked one in a child."""

from __future__ import annotations

import torch

DEV = "cuda:0"


def run_cases(train) -> dict:
    out = {}

    def keep(name, *ts):
        for i, t in enumerate(ts):
            if t is not None:
                out[f"{name}.{i}"] = t.detach().contiguous().view(-1).view(torch.uint8).cpu()

    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    for T, d, pad, dtype in [(9, 264, 0, torch.bfloat16), (5, 101, 3, torch.float32), (3, 5000, 0, torch.bfloat16),
                             (2, 9001, 0, torch.float32), (40, 64, 8, torch.bfloat16)]:
        rows = lambda: r(T, d + pad).to(dtype)[:, :d]  # noqa: E731
        w, wb, row_gate = r(d), r(d), r(d).to(dtype)
        for gate in (None, row_gate, rows()):
            x, y = rows(), rows()
            o = train.residual_norm(x, y, weight=w, branch_weight=wb, gate=gate)
            keep(f"norm{T}x{d}.{0 if gate is None else gate.dim()}", *o)
            keep(f"norm{T}x{d}.{0 if gate is None else gate.dim()}.bwd", *train.residual_norm_backward(
                rows(), rows(), o.residual, o.rstd, branch=y, weight=w, branch_weight=wb,
                branch_rstd=o.branch_rstd, gate=gate))
    for lengths in ([3, 0, 60], [3000, 17, 9000], [1] * 5000):
        cu = torch.tensor([0] + lengths, device=DEV).cumsum(0)
        T = int(cu[-1])
        logp, mask = -r(T).abs(), r(T) > -0.5
        keep(f"policy{T}", *train.policy_loss(logp, logp + 0.2 * r(T), r(len(lengths)), mask=mask,
                                              ref_logp=logp + 0.1 * r(T), entropy=r(T), cu_seqlens=cu,
                                              reduction="sequence", per_sequence=True, kl_coef=0.1,
                                              entropy_coef=0.1))
    for bits in (32, 8):
        sizes, shift = [1, 700, 2048, 9000], 1
        for cut in (0, shift):
            params = [r(n + cut)[cut:] for n in sizes]
            grads = [r(n + cut).bfloat16()[cut:] for n in sizes]
            copies = [torch.zeros(n + cut, device=DEV, dtype=torch.bfloat16)[cut:] for n in sizes]
            opt = train.AdamW(params, grads, copies=copies, state_bits=bits)
            norm = opt.step(max_norm=1.0)
            opt.step()
            keep(f"adamw{bits}.{cut}", norm, *params, *copies, *opt.state_values())
    torch.cuda.synchronize()
    return out
