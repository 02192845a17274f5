"""Trains a small draft head on a teacher's top logits and verifies its drafts by sampling.

A teacher (a fixed linear head) and a draft head of the same size read the same hidden
states.  Every step extracts the teacher's top-K logits (topk), takes the draft's loss
and gradient on them in one pass over its logits (distill), and moves the draft's weight
along it.  Before and after, the draft proposes the best token of every position of
a block (topk with K = 1), the target's rows are sampled with temperature, top-k and
top-p (sample), and a draft stands up to the first token that is not the sampled one.

    python -m dflash2_draft_head_gb300.train_draft --steps 60
"""
from __future__ import annotations

import argparse

import torch

from . import binding as df2


def accepted(draft_logits, teacher_logits, uniform, n: int) -> float:
    """Mean number of leading drafted tokens of a block of n that the target's samples
    confirm."""
    drafted = df2.topk(draft_logits, 1)[0].view(-1, n)
    tokens, _ = df2.sample(teacher_logits, uniform, temperature=1.0, top_k=20, top_p=0.95)
    return (drafted == tokens.view(-1, n)).int().cumprod(1).sum(1).float().mean().item()


def train(steps: int = 60, blocks: int = 64, n: int = 16, d: int = 64, V: int = 4096,
          K: int = 16, lr: float = 120.0, seed: int = 0) -> dict:
    """{"loss": [first, last], "accepted": [before, after]} of a run on synthetic states."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows = blocks * n

    def states():
        return torch.randn((rows, d), device=dev, generator=g)

    teacher = torch.randn((V, d), device=dev, generator=g) * (4.0 / d ** 0.5)
    draft = torch.randn((V, d), device=dev, generator=g) * (0.1 / d ** 0.5)
    # later positions of a block count less; the losses' mean
    weight = (0.95 ** (torch.arange(rows, device=dev) % n)) / rows
    held, uniform = states(), torch.rand((rows,), device=dev, generator=g)

    def logits(h, w):
        return (h @ w.t()).to(torch.bfloat16)

    before = accepted(logits(held, draft), logits(held, teacher), uniform, n)
    losses = []
    for _ in range(steps):
        h = states()
        ids, top = df2.topk(logits(h, teacher), K)
        z = logits(h, draft)
        loss, _, grad = df2.distill(z, ids, top, weight=weight, grad=z)  # in place
        draft -= lr * (grad.float().t() @ h)
        losses.append(loss.sum())
    after = accepted(logits(held, draft), logits(held, teacher), uniform, n)
    return {"loss": [losses[0].item(), losses[-1].item()], "accepted": [before, after]}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    r = train(steps=a.steps, seed=a.seed)
    print(f"loss {r['loss'][0]:.3f} -> {r['loss'][1]:.3f}, accepted tokens of 16: "
          f"{r['accepted'][0]:.2f} -> {r['accepted'][1]:.2f}")


if __name__ == "__main__":
    main()
