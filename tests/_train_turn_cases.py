"""Calls of the training-step operators where a CTA or a warp takes several turns, shared by the
normal and the checked build (test_gpu_train_checked_turns.py).  As a program: runs them with the
library that LP_LIBRARY names and saves the outputs, the backend id and the check word."""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def run_cases(train):
    g = torch.Generator(device=DEV).manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    out = {}

    def keep(name, *tensors):
        for i, t in enumerate(tensors):
            if t is not None:
                out[f"{name}.{i}"] = t.clone()

    # aligned rows; whole words; a ragged last group; the middle of a word, at the same place in every
    # row and at changing ones; two groups a thread; rows wider than the team kernels'
    for T, d, pad, shift in ((1301, 4096, 0, 0), (5003, 264, 8, 0), (1301, 2048, 2, 0), (1301, 2044, 4, 0),
                             (1301, 2047, 1, 1), (1301, 2047, 0, 0), (4001, 263, 0, 1), (501, 6000, 0, 0),
                             (501, 5001, 0, 1), (401, 9000, 0, 0), (401, 9001, 0, 1)):
        for residual, act in ((BF16, BF16), (F32, BF16), (F32, F32)):
            def rows(dtype):
                flat = r(T * (d + pad) + shift).to(dtype)[shift:]
                return flat.view(T, d + pad)[:, :d]
            for post, gate in ((True, "token"), (False, "channel")):
                w = r(d)
                kw = dict(branch=rows(act), weight=w, gate=rows(act) if gate == "token" else r(d).to(act),
                          branch_weight=w if post else None)
                o = train.residual_norm(rows(residual), **kw, branch_scale=0.5)
                b = train.residual_norm_backward(rows(act), rows(residual), o.residual, o.rstd,
                                                 branch_rstd=o.branch_rstd, **kw, branch_scale=0.5)
                keep(f"norm.{T}.{d}.{pad}.{shift}.{residual}.{act}.{post}", *o, *b)
    cpu = torch.Generator().manual_seed(32)
    for name, lengths in (("long", torch.tensor([700_001, 3, 900_000, 5])),
                          ("short", torch.randint(1, 3, (1_060_000,), generator=cpu)),
                          ("empty", torch.randint(-800, 900, (9000,), generator=cpu).clamp(min=0)),
                          ("few", torch.randint(0, 30, (300,), generator=cpu))):
        cu = torch.zeros(len(lengths) + 1, dtype=torch.int64)
        cu[1:] = lengths.cumsum(0)
        T = int(cu[-1]) + 7
        logp = -r(T).abs()
        mask = r(T) < 0.5
        for reduction in ("token", "sequence"):
            for per_sequence in (False, True):
                keep(f"policy.{name}.{reduction}.{per_sequence}", *train.policy_loss(
                    logp, logp + 0.2 * r(T), r(len(lengths) if per_sequence else T), mask=mask,
                    ref_logp=logp + r(T), entropy=logp, cu_seqlens=cu.to(DEV), reduction=reduction,
                    per_sequence=per_sequence, kl_coef=0.1, entropy_coef=0.1))
    sizes, shifts = [7_000_001, 0, 255, 2047, 4_194_304, 3_000_003, 1, 2_000_000], [0, 0, 1, 2, 0, 1, 0, 3]
    for bits in (8, 32):
        one = lambda n, s, dtype: r(n + s).to(dtype)[s:]  # noqa: E731
        params = [one(n, s, F32) for n, s in zip(sizes, shifts)]
        opt = train.AdamW(params, [one(n, s, BF16) for n, s in zip(sizes, shifts)],
                          copies=[one(n, s, BF16) for n, s in zip(sizes, shifts)], state_bits=bits)
        norm = opt.step(max_norm=1.0)
        opt.step()
        keep(f"adamw{bits}", norm, *params, *opt.copies, *opt.state_values())
    torch.cuda.synchronize()
    return out


if __name__ == "__main__":
    from invariant_token_logprobs_gb300 import lp, train

    lp.load(build_if_needed=False)
    outputs = run_cases(train)
    torch.save({"out": outputs, "backend": lp.lp_backend_id(), "word": lp.lp_get_check_word()}, sys.argv[1])
