"""Preference training of the end of a language model: a block's projection is added to the residual
stream and layer-normed, the LM head scores the tokens of pairs of answers, and the preference loss
against a frozen reference is propagated back into the head, the norm and the projection.

    python examples/train_preference.py [--steps N] [--pairs P] [--hidden d] [--vocab V]

A step is tune.layer_norm, lp.linear_logprob_lse, tune.preference_loss, lp.linear_logprob_backward into
float32 main gradients, tune.layer_norm_backward, one tune.Muon step of the projection and one
train.AdamW step of the rest; torch multiplies by the projection.  The data are synthetic: rows of
random hidden states, the chosen answers' tokens from the lower half of the vocabulary and the
rejected ones' from the upper.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from invariant_token_logprobs_gb300 import lp, train, tune  # noqa: E402

BF16 = torch.bfloat16


class Model:
    """The trained weights: float32 masters, bfloat16 copies that the passes read, and main gradients."""

    def __init__(self, hidden: int, vocab: int, device, seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = {
            "projection": torch.randn(hidden, hidden, generator=g, device=device) / hidden ** 0.5,
            "head": 0.02 * torch.randn(vocab, hidden, generator=g, device=device),
            "norm": torch.ones(hidden, device=device),
            "norm_bias": torch.zeros(hidden, device=device),
        }
        self.weight = {k: v.to(BF16) for k, v in self.master.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items()}
        rest = [k for k in self.master if k != "projection"]
        self.muon = tune.Muon([self.master["projection"]], [self.grad["projection"]],
                              copies=[self.weight["projection"]], lr=0.01, weight_decay=0.01, scaling="rms")
        self.adamw = train.AdamW([self.master[k] for k in rest], [self.grad[k] for k in rest],
                                 copies=[self.weight[k] for k in rest], lr=1e-3, betas=(0.9, 0.95),
                                 weight_decay=[0.01 if k == "head" else 0.0 for k in rest])


def score(model: Model, batch: dict):
    """The layer norm's outputs, and the tokens' log-probabilities, entropies and log Z."""
    branch = batch["hidden"] @ model.weight["projection"].t()
    out = tune.layer_norm(batch["hidden"], branch, weight=model.weight["norm"], bias=model.weight["norm_bias"])
    return out, lp.linear_logprob_lse(out.normed, model.weight["head"], batch["tokens"])


def gradients(model: Model, batch: dict, beta: float = 0.1) -> torch.Tensor:
    """The loss's stats; its gradients are written into the main gradients."""
    out, (logp, entropy, lse) = score(model, batch)
    loss = tune.preference_loss(logp, batch["cu_seqlens"], ref_logp=batch["ref_logp"], mask=batch["mask"],
                                beta=beta, label_smoothing=0.05, nll_coef=0.1)
    model.grad["head"].zero_()
    grad_h, _ = lp.linear_logprob_backward(out.normed, model.weight["head"], batch["tokens"], loss.grad_logp, None,
                                           saved_lse=lse, saved_entropy=entropy, accumulate_into=model.grad["head"])
    g = tune.layer_norm_backward(grad_h.to(BF16), None, out.residual, out.mean, out.rstd, weight=model.weight["norm"],
                                 bias=model.weight["norm_bias"], branch=True)
    model.grad["norm"].copy_(g.weight)
    model.grad["norm_bias"].copy_(g.bias)
    model.grad["projection"].copy_(g.branch.t() @ batch["hidden"])
    return loss.stats


def train_step(model: Model, batch: dict) -> torch.Tensor:
    """One step; the loss's stats, on the device."""
    stats = gradients(model, batch)
    model.muon.step()
    model.adamw.step(max_norm=1.0)
    return stats


def pairs_of(model: Model, pairs: int, seed: int) -> dict:
    """A batch of pairs of answers of 8 to 31 tokens behind a prompt of 4, with the model's present
    log-probabilities as the reference's."""
    device = model.weight["norm"].device
    vocab, hidden = model.weight["head"].shape
    g = torch.Generator(device=device).manual_seed(seed)
    lengths = torch.randint(12, 36, (2 * pairs,), generator=g, device=device)
    cu = torch.zeros(2 * pairs + 1, dtype=torch.int64, device=device)
    cu[1:] = lengths.cumsum(0)
    rows = int(cu[-1])
    sequence = torch.repeat_interleave(torch.arange(2 * pairs, device=device), lengths)
    place = torch.arange(rows, device=device) - cu[sequence]
    batch = {"hidden": torch.randn(rows, hidden, generator=g, device=device).to(BF16), "cu_seqlens": cu,
             "mask": place >= 4}
    tokens = torch.randint(0, vocab // 2, (rows,), generator=g, device=device) + (sequence % 2) * (vocab // 2)
    batch["tokens"] = torch.where(batch["mask"], tokens, torch.full_like(tokens, -1))  # a prompt's are no targets
    batch["ref_logp"] = score(model, batch)[1][0]
    return batch


def run(steps: int = 20, pairs: int = 32, hidden: int = 256, vocab: int = 8192, device: str = "cuda:0", log=print):
    """Trains, and returns the last step's stats."""
    model = Model(hidden, vocab, device)
    reference = Model(hidden, vocab, device)
    stats = None
    for step in range(steps):
        batch = pairs_of(reference, pairs, seed=1 + step)  # the weights have seed 0
        stats = train_step(model, batch).tolist()
        if log is not None and step % max(1, steps // 10) == 0:
            log(f"step {step:4d}  loss {stats[0]:.4f}  accuracy {stats[3]:.2f}  rewards {stats[4]:+.3f} {stats[5]:+.3f}")
    return stats


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=20)
    parser.add_argument("--pairs", type=int, default=32)
    parser.add_argument("--hidden", type=int, default=256)
    parser.add_argument("--vocab", type=int, default=8192)
    args = parser.parse_args()
    run(args.steps, args.pairs, args.hidden, args.vocab)
