"""Policy-gradient training of the end of a language model: the last block's output is added to
the residual stream and normed, the LM head scores the sampled tokens, and the clipped policy
loss is propagated back into the head, the norms' weights and the gate.

    python examples/train_head.py [--steps N] [--rows T] [--hidden d] [--vocab V] [--state-bits 8]

Every step runs in liblp: train.residual_norm, lp.linear_logprob_lse, train.policy_loss,
lp.linear_logprob_backward into float32 main gradients, train.residual_norm_backward and one
train.AdamW step with the gradients clipped by their global norm, which also writes the bfloat16
weights of the next step.  The data are synthetic: rows of random hidden states, with one channel
that is always on, and sampled tokens, those from the lower half of the vocabulary rewarded.  What
the trainer is to learn is therefore to put less weight on the upper half.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from invariant_token_logprobs_gb300 import lp, train  # noqa: E402

BF16 = torch.bfloat16


class Head:
    """The trained weights: float32 masters, bfloat16 copies that the passes read, and main
    gradients."""

    def __init__(self, hidden: int, vocab: int, state_bits: int, lr: float, device, seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = {
            "head": 0.02 * torch.randn(vocab, hidden, generator=g, device=device),
            "norm": torch.ones(hidden, device=device),
            "branch_norm": torch.ones(hidden, device=device),
            "gate": torch.full((hidden,), 0.5, device=device),
        }
        self.weight = {k: v.to(BF16) for k, v in self.master.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items()}
        names = list(self.master)
        self.optimizer = train.AdamW(
            [self.master[k] for k in names], [self.grad[k] for k in names],
            copies=[self.weight[k] for k in names], lr=lr, betas=(0.9, 0.95),
            weight_decay=[0.01 if k == "head" else 0.0 for k in names], state_bits=state_bits)


def forward(model: Head, residual, branch):
    """The residual stream after the last block, and its norm: the LM head's input."""
    return train.residual_norm(residual, branch, weight=model.weight["norm"],
                               branch_weight=model.weight["branch_norm"], gate=model.weight["gate"])


def train_step(model: Head, batch: dict, clip: float = 0.2, entropy_coef: float = 1e-3,
               max_norm: float = 1.0):
    """One step; (stats of the loss, norm of the gradients), on the device."""
    out = forward(model, batch["residual"], batch["branch"])
    logp, entropy, lse = lp.linear_logprob_lse(out.normed, model.weight["head"], batch["tokens"])
    loss = train.policy_loss(logp, batch["old_logp"], batch["advantages"], mask=batch["mask"],
                             entropy=entropy, cu_seqlens=batch["cu_seqlens"], reduction="sequence",
                             clip_low=clip, clip_high=clip, entropy_coef=entropy_coef)
    model.grad["head"].zero_()
    grad_h, _ = lp.linear_logprob_backward(
        out.normed, model.weight["head"], batch["tokens"], loss.grad_logp, loss.grad_entropy,
        saved_lse=lse, saved_entropy=entropy, accumulate_into=model.grad["head"])
    g = train.residual_norm_backward(
        grad_h.to(BF16), None, out.residual, out.rstd, branch=batch["branch"],
        weight=model.weight["norm"], branch_weight=model.weight["branch_norm"],
        branch_rstd=out.branch_rstd, gate=model.weight["gate"])
    for name, grad in (("norm", g.weight), ("branch_norm", g.branch_weight), ("gate", g.gate)):
        model.grad[name].copy_(grad)
    return loss.stats, model.optimizer.step(max_norm=max_norm)


def rollout(model: Head, rows: int, seed: int) -> dict:
    """A batch of ragged sequences whose tokens are drawn from the head itself."""
    device = model.weight["norm"].device
    vocab, hidden = model.weight["head"].shape
    g = torch.Generator(device=device).manual_seed(seed)
    batch = {"residual": torch.randn(rows, hidden, generator=g, device=device).to(BF16),
             "branch": torch.randn(rows, hidden, generator=g, device=device).to(BF16)}
    batch["residual"][:, 0] = 8.0
    normed = forward(model, batch["residual"], batch["branch"]).normed
    p = torch.softmax(normed.float() @ model.weight["head"].float().t(), dim=1)
    tokens = torch.multinomial(p, 1, generator=g)[:, 0]
    # four sequences, the first rows of each a prompt: its tokens are no targets
    cu = torch.tensor([0, rows // 8, rows // 2, rows - rows // 4, rows], device=device)
    place = torch.arange(rows, device=device)
    start = cu[torch.searchsorted(cu[1:], place, right=True)]
    batch["mask"] = place - start >= rows // 32
    batch["tokens"] = torch.where(batch["mask"], tokens, torch.full_like(tokens, -1))
    batch["advantages"] = torch.where(tokens < vocab // 2, 1.0, -1.0)
    batch["old_logp"], _ = lp.linear_logprob(normed, model.weight["head"], batch["tokens"])
    batch["cu_seqlens"] = cu
    return batch


def lower_half(model: Head, seed: int, rows: int = 256) -> float:
    """The mean probability of the rewarded tokens on rows that were not trained on."""
    batch = rollout(model, rows, seed)
    normed = forward(model, batch["residual"], batch["branch"]).normed
    p = torch.softmax(normed.float() @ model.weight["head"].float().t(), dim=1)
    return float(p[:, :p.shape[1] // 2].sum(1).mean())


def run(steps: int = 20, rows: int = 512, hidden: int = 256, vocab: int = 8192, state_bits: int = 32,
        lr: float = 1e-2, device: str = "cuda:0", log=print) -> tuple[float, float]:
    """Trains and returns lower_half before and after."""
    model = Head(hidden, vocab, state_bits, lr, device)
    before = lower_half(model, seed=10**6)
    for step in range(steps):
        stats, norm = train_step(model, rollout(model, rows, seed=1 + step))  # the weights have seed 0
        if log is not None and step % max(1, steps // 10) == 0:
            loss, policy, _, entropy, clipped = stats.tolist()
            log(f"step {step:4d}  loss {loss:+.4f}  entropy {entropy:.3f}  clipped {clipped:.3f}  "
                f"gradient norm {float(norm):.3g}")
    after = lower_half(model, seed=10**6)
    if log is not None:
        log(f"probability of the rewarded half: {before:.3f} -> {after:.3f}")
    return before, after


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=20)
    parser.add_argument("--rows", type=int, default=512)
    parser.add_argument("--hidden", type=int, default=256)
    parser.add_argument("--vocab", type=int, default=8192)
    parser.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    args = parser.parse_args()
    run(args.steps, args.rows, args.hidden, args.vocab, args.state_bits)
