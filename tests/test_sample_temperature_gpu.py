"""Sampling at temperatures whose factor log2(e) / T is 0 or infinite in fp32 (T = +inf, and T
below 4.3e-39), and at those next to them, against the rule in whole numbers (see
test_sample_gpu.py).  At T = +inf every finite entry weighs the same."""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_sample_gpu import INF, NAN, _built, _one_of, _place, _rows, _rule, _u  # noqa: F401

pytestmark = pytest.mark.gpu

TEMPERATURES = [INF, 3e38, 1e38, 4.3e-39, 4.2e-39, 1e-40, 1e-45]
CUTS = [dict(k=1), dict(k=20), dict(p=0.9), dict(k=300, p=0.5), dict(k=50, p=0.3, mp=0.2),
        dict(p=0.4, mp=1.0)]


def _check(x, u, T, k=0, p=1.0, mp=0.0):
    tok = torch.full(x.shape[:1], -9, dtype=torch.int32, device="cuda")
    tok, prob = df2.sample(x, u, temperature=T, top_k=k, top_p=p, min_p=mp, tokens=tok)
    tok, prob = tok.cpu().numpy(), prob.cpu().numpy()
    for r in range(x.shape[0]):
        t = np.float32(_one_of(T, r)).item()
        rt, rp = _rule(x[r].float(), u[r].item(), t, k, p, mp)
        assert tok[r] == rt, (r, t, k, p, mp, tok[r], rt)
        assert abs(prob[r] - rp) <= 2.0 ** -23 * rp, (r, t, k, p, mp, prob[r], rp)
    return tok, prob


def _inputs(V, dtype, masked, seed):
    x = _rows(4, V, dtype, seed, pad=seed % 4, offset=seed % 3)
    if masked:
        g = torch.Generator().manual_seed(seed)
        gone = (torch.rand((4, V), generator=g) < 0.7).cuda()
        x.masked_fill_(gone, -INF)
        x[1, ::5] = NAN
        x[2, -1] = 3.0                      # at least this one is left
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("V", [1, 7, 1003, 20011, 151935])
def test_temperature_alone(V, masked, dtype):
    x = _inputs(V, dtype, masked, V)
    for i, T in enumerate(TEMPERATURES):
        _check(x, _u(4, i), T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("V", [7, 1003, 20011, 151935])
def test_with_cuts(V, masked, dtype):
    x = _inputs(V, dtype, masked, V + 1)
    for i, T in enumerate(TEMPERATURES if V < 100000 else (INF, 1e-40)):
        for s in CUTS:
            _check(x, _u(4, i), T, **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_by_row(dtype):
    x = _inputs(5003, dtype, True, 3)
    T = torch.tensor([INF, 1e-40, 1.0, INF]).cuda()
    for s in [dict()] + CUTS:
        _check(x, _u(4, 9), T, **s)


def test_the_largest_entry_stands_apart():
    """+inf entries are the only ones kept, and a difference that leaves fp32's range is
    still that of an entry above -inf."""
    x = torch.randn((3, 2000), generator=torch.Generator().manual_seed(2))
    x[0, 5] = x[0, 900] = INF
    x[1, ::2] = -3e38
    x[1, 1::2] = 3e38
    x[2] = torch.finfo(torch.float32).min
    x[2, 3] = 2.0
    x = _place(x, torch.float32, pad=1)
    u = torch.tensor([0.7, 0.25, 0.5]).cuda()
    tok, prob = df2.sample(x, u, temperature=INF)
    assert tok.tolist() == [900, 500, 1000]
    assert prob.tolist() == [0.5, np.float32(1 / 2000), np.float32(1 / 2000)]
    tok, prob = df2.sample(x, u, temperature=1e-40)
    assert tok.tolist() == [900, 501, 3] and prob.tolist() == [0.5, np.float32(1 / 1000), 1.0]


def test_frequencies_are_even_at_infinity():
    n, V = 8192, 60
    x = _rows(1, V, "f32", 21)
    x[0, 10:14] = -INF
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    tok, prob = df2.sample(x.expand(n, V).contiguous(), u, temperature=INF)
    count = torch.bincount(tok.long(), minlength=V).double()
    want = torch.full((V,), n / 56, dtype=torch.float64, device="cuda")
    want[10:14] = 0
    assert (count - want).abs().max() <= 2 and torch.equal(prob, torch.full_like(prob, 1 / 56))
