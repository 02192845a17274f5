"""Cuts by top_p on rows made for the turns of the kernel's cut search.  Tokens are compared
with the rule in whole numbers (see test_sample_gpu.py)."""
import math

import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_sample_gpu import _built, _place, _rule, _u  # noqa: F401

pytestmark = pytest.mark.gpu

P = 0.9
GROUPS, BINS = 256, 2048  # of the kernel: groups of a row, bins of depth


def _one_sided_rows(rows, side, seed, levels=600, copies=240, tops=4000):
    """fp32 rows in which every depth bin's entries stand on the same side of its middle:
    above it (side 1) a cut by the middles' weights comes too late, below it (-1) too early.
    `tops` entries share the maximum, so that it is the largest of every group of the row,
    and with it the bins' width is known: the deepest one ends where an entry weighs less
    than an even share of what top_p leaves of the groups' weight."""
    V = tops + levels * copies
    share = (1 - P) * 0.999 * GROUPS * 2.0 ** 40 / V - 1
    width = -(math.log2(share) - 40.1) / (BINS - 1)
    at = (torch.arange(1, levels + 1, dtype=torch.float64) - 0.4 * side) * width
    depth = torch.cat([torch.zeros(tops, dtype=torch.float64), at.repeat_interleave(copies)])
    x = (-depth * math.log(2)).float()
    g = torch.Generator().manual_seed(seed)
    return torch.stack([x[torch.randperm(V, generator=g)] for _ in range(rows)])


@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("rows", [3, 16, 64])
def test_likely_cuts_that_miss_on_every_row(rows, side):
    """The first list misses the cut on every row, so that the search turns again, on
    clusters of 8.  With side 1 the exact weight before that list is past the limit: the CTAs
    learn of it from one exchange of sums, and the next turn's exchange follows without
    a list in between.  Many runs have to agree."""
    x = _place(_one_sided_rows(rows, side, rows), torch.float32)
    u = _u(rows, rows)
    tok, prob = df2.sample(x, u, top_p=P)
    for r in range(0, rows, max(1, rows // 8)):
        rt, rp = _rule(x[r], u[r].item(), 1.0, 0, P, 0.0)
        assert tok[r].item() == rt and abs(prob[r].item() - rp) <= 2.0 ** -23 * rp
    for _ in range(25):
        again = df2.sample(x, u, top_p=P)
        assert torch.equal(again[0], tok) and torch.equal(again[1], prob)
