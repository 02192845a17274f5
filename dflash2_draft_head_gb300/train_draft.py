"""Trains a small draft head on a teacher's top logits and verifies its drafts by sampling.

A teacher (a fixed linear head) and a draft head of the same size read the same hidden
states.  Every step extracts the teacher's top-K logits (topk), takes the draft's loss
and gradient on them in one pass over its logits (distill), and moves the draft's weight
along it: by plain gradient descent, or by AdamW with clipped gradients (grad_norm, adamw)
and states in 32 or 8 bits.  Before and after, the draft proposes the best token of every
position of a block (topk with K = 1), the target's rows are sampled with temperature, top-k
and top-p (sample), and a draft stands up to the first token that is not the sampled one.

    python -m dflash2_draft_head_gb300.train_draft --steps 60
    python -m dflash2_draft_head_gb300.train_draft --steps 60 --optimizer adamw8
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


class AdamW:
    """Weights in one list with their AdamW states, clipped by the gradients' norm: fp32
    states, or 8 bits an element with stochastic rounding from `seed`.  Steps are counted on the
    device: one that is left out, as its norm is not finite, does not count."""

    def __init__(self, params, lr: float, bits: int = 32, max_norm: float | None = 1.0,
                 weight_decay: float = 0.0, seed: int = 0):
        self.params, self.lr, self.max_norm, self.seed = params, lr, max_norm, seed
        self.weight_decay = weight_decay
        self.step_number = torch.zeros(1, dtype=torch.int32, device=params[0].device)

        def zeros(size, dtype):
            return [torch.zeros(size(p), dtype=dtype, device=p.device) for p in params]

        kind = torch.uint8 if bits == 8 else torch.float32
        self.exp_avg = zeros(lambda p: p.shape, kind)
        self.exp_avg_sq = zeros(lambda p: p.shape, kind)
        self.scales = {}
        if bits == 8:
            for name in ("exp_avg_scale", "exp_avg_sq_scale"):
                self.scales[name] = zeros(lambda p: ((p.numel() + 31) // 32,), torch.uint8)

    def step(self, grads) -> torch.Tensor:
        """One step; the gradients' norm [1] before it is clipped."""
        norm = df2.grad_norm(grads)
        self.step_number += torch.isfinite(norm)
        df2.adamw(self.params, grads, self.exp_avg, self.exp_avg_sq, step=self.step_number,
                  lr=self.lr, weight_decay=self.weight_decay, norm=norm, max_norm=self.max_norm,
                  seed=self.seed if self.scales else None, **self.scales)
        return norm


def train(steps: int = 60, blocks: int = 64, n: int = 16, d: int = 64, V: int = 4096,
          K: int = 16, lr: float | None = None, seed: int = 0, optimizer: str = "sgd") -> dict:
    """{"loss": [first, last], "accepted": [before, after]} of a run on synthetic states.
    optimizer: "sgd" (lr 120 by default), "adamw" or "adamw8" (states in 8 bits; lr 0.02)."""
    if optimizer not in ("sgd", "adamw", "adamw8"):
        raise ValueError(f"optimizer must be sgd, adamw or adamw8, got {optimizer}")
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
    adam = None
    if optimizer == "sgd":
        lr = 120.0 if lr is None else lr
    else:
        adam = AdamW([draft], 0.02 if lr is None else lr, 8 if optimizer == "adamw8" else 32,
                     seed=seed)

    def logits(h, w):
        return (h @ w.t()).to(torch.bfloat16)

    before = accepted(logits(held, draft), logits(held, teacher), uniform, n)
    losses = []
    for _ in range(steps):
        h = states()
        ids, top = df2.topk(logits(h, teacher), K)
        z = logits(h, draft)
        loss, _, grad = df2.distill(z, ids, top, weight=weight, grad=z)  # in place
        slope = grad.float().t() @ h
        if adam is None:
            draft -= lr * slope
        else:
            adam.step([slope])
        losses.append(loss.sum())
    after = accepted(logits(held, draft), logits(held, teacher), uniform, n)
    return {"loss": [losses[0].item(), losses[-1].item()], "accepted": [before, after]}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--optimizer", choices=("sgd", "adamw", "adamw8"), default="sgd")
    a = ap.parse_args()
    r = train(steps=a.steps, seed=a.seed, optimizer=a.optimizer)
    print(f"loss {r['loss'][0]:.3f} -> {r['loss'][1]:.3f}, accepted tokens of 16: "
          f"{r['accepted'][0]:.2f} -> {r['accepted'][1]:.2f}")


if __name__ == "__main__":
    main()
