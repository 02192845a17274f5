"""Cuts by top_p on rows made for the turns of the kernel's cut search, and on splits of
a row that other tests do not reach.  Tokens are compared with the rule in whole numbers
(see test_sample_gpu.py)."""
import math

import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_sample_gpu import TOL, _built, _order, _place, _rule, _u  # noqa: F401

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


def _in_64_bits_near_a_cut(x32, u, p, token, prob):
    """The rule in 64 bits without a gap round the cut: the entries that are kept for
    p - TOL are kept, those that are not for p + TOL are not, and what lies between moves
    the shares by at most `slack`."""
    x = x32.double().cpu().numpy()
    order = _order(x)
    w = np.exp(x - x.max())[order]
    w /= w.sum()
    before = np.cumsum(w) - w
    sure, may = before < p - TOL, before < p + TOL
    sure[0] = may[0] = True
    kept = np.zeros(len(x), bool)
    kept[order[may]] = True
    share = np.zeros(len(x))
    share[order[sure]] = w[sure]
    total = share.sum()
    slack = 2 * (w[may].sum() - total + TOL) / total + TOL
    share /= total
    hi = np.cumsum(share)
    own = np.exp(x[token] - x.max()) / np.exp(x - x.max()).sum() / total
    return kept[token] and hi[token] - own - slack <= u <= hi[token] + slack and \
        abs(prob - own) <= own * (2 * TOL + slack)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,p", [(151936, 0.95), (151935, 0.5), (32000, 0.9), (262144, 0.99)])
def test_flat_rows_in_64_bits(V, p, dtype):
    """On a flat row the running weights near the cut are closer together than fp32's
    rounding of them, so that no row is far from a cut; every row is compared."""
    g = torch.Generator().manual_seed(V)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = _place(torch.randn((4, V), generator=g) * torch.tensor([[0.1], [0.5], [1.0], [1.5]]), dt)
    u = _u(4, V)
    tok, prob = df2.sample(x, u, top_p=p)
    pf = float(np.float32(p))
    for r in range(4):
        rt, _ = _rule(x[r].float(), u[r].item(), 1.0, 0, p, 0.0)
        assert tok[r].item() == rt
        assert _in_64_bits_near_a_cut(x[r].float(), u[r].item(), pf, tok[r].item(),
                                      prob[r].item()), r


@pytest.mark.parametrize("V,dtype,rows", [
    (110_001, "f32", 470),    # 430 KB a row, one CTA each
    (160_007, "f32", 470),    # 625 KB
    (200_003, "f32", 470),    # 781 KB, clusters of two although the GPU is full
    (400_009, "f32", 460),    # 1.5 MB, clusters of four
])
def test_wide_slices_in_a_full_batch(V, dtype, rows):
    """A row alone and in a batch that fills the GPU are split in different ways."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn((rows, V), device="cuda", generator=g)
    x[::3] *= 3
    u = _u(rows, V)
    for s in (dict(top_p=0.9), dict(top_k=2000, top_p=0.8), dict()):
        tok, prob = df2.sample(x, u, **s)
        for r in range(0, rows, 23):
            one = df2.sample(x[r:r + 1], u[r:r + 1], **s)
            assert one[0].item() == tok[r].item() and one[1].item() == prob[r].item()
        r = rows - 1
        rt, rp = _rule(x[r], u[r].item(), 1.0, s.get("top_k", 0), s.get("top_p", 1.0), 0.0)
        assert tok[r].item() == rt and abs(prob[r].item() - rp) <= 2.0 ** -23 * rp
