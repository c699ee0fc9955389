"""More cases of the fine-tuning operators for the checked build: long sequences among short ones, runs of empty ones,
Muon's batches and an eps above the norm, the layer norm in place.  As a program it runs them with the library that
LP_LIBRARY names and saves the outputs, the backend id and the check word."""

from __future__ import annotations

import os
import sys

import torch

DEV = "cuda:0"


def run_cases(tune) -> dict:
    out = {}

    def keep(name, *ts):
        for i, t in enumerate(ts):
            out[f"{name}.{i}"] = t.detach().contiguous().view(-1).view(torch.uint8).cpu()

    g = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    for name, lengths in {"long": [16] * 601 + [200000] + [16] * 398, "last": [40] * 999 + [70001],
                          "side": [9] * 800 + [30000, 9000, 20000, 1] + [9] * 196, "empty": [700, 5] + [0] * 5002 + [9000, 40],
                          "runs": ([90, 90] + [0] * 70) * 50, "around": [0] * 3000 + [9000, 800, 7, 1] + [0] * 200}.items():
        cu = torch.tensor([0] + lengths, device=DEV).cumsum(0) + 2
        logp = -r(int(cu[-1]) + 3).abs()
        mask = r(logp.shape[0]) > -1.0
        keep(name, *tune.preference_loss(logp, cu, ref_logp=0.9 * logp, mask=mask))
        keep(name + ".halves", *tune.preference_loss(logp, cu, halves=True, average=True))
    cu = torch.randint(-3000, 30000, (2001,), generator=g, device=DEV)  # no offsets: the call ends
    tune.preference_loss(-r(20000).abs(), cu)
    for eps in (1e-7, 1e3, 1e12):
        shapes = [(4096, 4096)] * 4 + [(300, 200), (2050, 120), (1030, 1100), (64, 64)]
        params, grads = [0.02 * r(*s) for s in shapes], [r(*s) for s in shapes]
        opt = tune.Muon(params, grads, eps=eps)
        opt.step()
        keep(f"muon{eps}", *(p[:64] for p in params))
    for T, d in ((900, 1024), (400, 2047), (20, 9001)):
        x, y, w = r(T, d).bfloat16(), r(T, d).bfloat16(), r(d)
        keep(f"place{d}", *tune.layer_norm(x, y, weight=w, in_place=True))
    torch.cuda.synchronize()
    return out


if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from invariant_token_logprobs_gb300 import lp, tune as module

    lp.load(build_if_needed=False)
    cases = run_cases(module)
    torch.save({"out": cases, "backend": lp.lp_backend_id(), "word": lp.lp_get_check_word()}, sys.argv[1])
