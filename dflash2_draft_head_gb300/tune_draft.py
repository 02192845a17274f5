"""Tunes a draft head on what its drafts are worth, the stage behind distillation.

A target (a fixed linear head) and a draft head read the same hidden states.  Every step samples
drafts from the draft's logits (sample, whose share of a token is its old probability) and
tokens from the target's, and a drafted token is worth 1 where it is the target's.  By
method "policy" every position is a sample with the advantage of its worth over the mean
(policy_loss); by "preference" two drafts of every block make a pair, the one with more
tokens confirmed being the chosen one (preference_loss).  Both hold the head near the one it
began with: by a KL term at the drawn tokens, or by log ratios to it.  The weight moves by
AdamW with clipped gradients (grad_norm, adamw).

    python -m dflash2_draft_head_gb300.tune_draft --steps 60 --method policy
"""
from __future__ import annotations

import argparse

import torch

from . import binding as df2
from .train_draft import AdamW, accepted


def token_logp(logits, tokens):
    """log-probabilities of tokens: those that policy_loss() returns, nothing being
    weighed."""
    none = torch.zeros(tokens.shape, device=logits.device)
    return df2.policy_loss(logits, tokens, none, none)[1]


def tune(steps: int = 60, blocks: int = 256, n: int = 16, d: int = 64, V: int = 4096,
         method: str = "policy", bits: int = 32, lr: float = 0.0005, kl_coef: float = 0.02,
         seed: int = 0) -> dict:
    """{"loss": [first, last], "accepted": [before, after], "norm": last gradient's} of a run on
    synthetic states."""
    if method not in ("policy", "preference"):
        raise ValueError(f"method must be policy or preference, got {method}")
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows = blocks * n

    def noise(*shape):
        return torch.randn(shape, device=dev, generator=g)

    def uniform():
        return torch.rand((rows,), device=dev, generator=g)

    def logits(h, w):
        return (h @ w.t()).to(torch.bfloat16)

    target = noise(V, d) * (4.0 / d ** 0.5)
    draft = target * 0.6 + noise(V, d) * (1.0 / d ** 0.5)
    first = draft.clone()
    adam = AdamW([draft], lr, bits, seed=seed)
    held, drawn = noise(rows, d), uniform()
    before = accepted(logits(held, draft), logits(held, target), drawn, n)
    weight = torch.full((rows,), 1.0 / rows, device=dev)
    losses, norm = [], None
    for _ in range(steps):
        h = noise(rows, d)
        z = logits(h, draft)
        want, _ = df2.sample(logits(h, target), uniform())
        reference = logits(h, first)
        if method == "policy":
            tokens, share = df2.sample(z, uniform())
            worth = (tokens == want).float()
            loss, _, _, grad = df2.policy_loss(
                z, tokens, share.log(), worth - worth.mean(), weight=weight, kl_coef=kl_coef,
                ref_logp=token_logp(reference, tokens), grad=z)  # in place
            slope = grad.float().t() @ h
        else:
            two = [df2.sample(z, uniform())[0].view(blocks, n) for _ in range(2)]
            hits = [(t == want.view(blocks, n)).sum(1) for t in two]
            better = (hits[0] >= hits[1])[:, None]
            # the chosen draft of every block, then the rejected ones; equal pairs weigh nothing
            tokens = torch.cat([torch.where(better, two[0], two[1]),
                                torch.where(better, two[1], two[0])]).view(-1)
            offsets = torch.arange(0, 2 * rows + 1, n, dtype=torch.int32, device=dev)
            both = z.repeat(2, 1)
            ref = token_logp(reference.repeat(2, 1), tokens).view(2 * blocks, n).sum(1)
            loss, _, _, _, grad = df2.preference_loss(
                both, tokens, offsets, ref_logp=ref, beta=0.2,
                weight=(hits[0] != hits[1]).float() / blocks, grad=both)  # in place
            slope = grad.float().t() @ h.repeat(2, 1)
        norm = adam.step([slope])
        losses.append(loss.sum())
    after = accepted(logits(held, draft), logits(held, target), drawn, n)
    return {"loss": [losses[0].item(), losses[-1].item()], "accepted": [before, after],
            "norm": norm.item()}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--method", choices=("policy", "preference"), default="policy")
    ap.add_argument("--bits", type=int, choices=(32, 8), default=32)
    a = ap.parse_args()
    r = tune(steps=a.steps, seed=a.seed, method=a.method, bits=a.bits)
    print(f"loss {r['loss'][0]:.4f} -> {r['loss'][1]:.4f}, accepted tokens of 16: "
          f"{r['accepted'][0]:.2f} -> {r['accepted'][1]:.2f}")


if __name__ == "__main__":
    main()
