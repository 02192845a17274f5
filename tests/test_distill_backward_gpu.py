"""The gradient alone on rows whose logits are far from 0, against the formula in 64 bits and
against the gradient that comes with the loss (see test_distill_gpu.py).

Bound: the fused gradient's (1e-5 and q's, times |grad_loss * weight| / T).  A row with |lse| below 256
takes exp(z/T - lse) from the rounded lse, whose half unit is at most 2^-17, so that a share,
which is at most 1, is off by less than 2^-16; other rows take their sum again and have no
such term.  Nothing in the bound grows with the logits."""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_distill_gpu import INF, NAN, _bounds, _built, _formula, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.bfloat16).min


def _check(z, ids, y, T, w=None):
    rows = z.shape[0]
    bf = z.dtype == torch.bfloat16
    _, lse, grad = df2.distill(z, ids, y, temperature=T, weight=w, grad=True)
    up = torch.linspace(0.5, 2, rows, device="cuda")
    back = df2.distill_backward(up, z, ids, y, lse, temperature=T, weight=w)
    for r in range(rows):
        wr = 1.0 if w is None else w[r].item()
        _, _, rg = _formula(z[r], ids[r], y[r], T, wr)
        gb = _bounds(z[r], y[r], T, 0.0)[2] + 2.0 ** -16
        rnd = 2.0 ** -8 * np.abs(rg) if bf else 0
        for got, s in ((grad, 1.0), (back, up[r].item())):
            err = np.abs(got[r].double().cpu().numpy() - rg * s)
            assert (err <= abs(wr * s) / T * gb + rnd * s).all(), (r, s, err.max())
    return grad, back


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 0.5, 2.0])
@pytest.mark.parametrize("V,rows", [(1, 2), (700, 6), (40_003, 6), (151936, 6), (3000, 640)])
def test_rows_of_one_large_value(V, rows, T, dtype):
    """Rows masked by the type's lowest value all over: every share is 1 / V."""
    K = min(V, 9)
    z, ids, y = _inputs(rows, V, K, dtype, V + 1, pad=1)
    z[0] = LOWEST
    z[1] = -LOWEST
    if rows > 2:
        z[2] = LOWEST
        z[2, ::7] = 1.5                    # a row of which every seventh entry is left
        z[3] = -1e30
        z[4, ids[4, 0].long()] = 3e38      # one entry far above the others
        z[-1] = LOWEST
    w = torch.linspace(0.5, 1.5, rows, device="cuda")
    _check(z, ids, y, T)
    _check(z, ids, y, T, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [-200.0, 250.0, 300.0, -5000.0, 70000.0, 1e7])
def test_shifted_rows(offset, dtype):
    """A shift of a row's logits changes nothing but their own rounding."""
    z, ids, y = _inputs(5, 5003, 17, dtype, 8, pad=3, offset=1)
    z.add_(offset)
    _check(z, ids, y, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1003, 151936])
def test_in_place_and_on_another_grid(V, dtype):
    z, ids, y = _inputs(4, V, 6, dtype, 5, pad=2, offset=1)
    z[::2] -= 9000.0
    lse = df2.distill(z, ids, y)[1]
    up = torch.ones(4, device="cuda")
    want = df2.distill_backward(up, z, ids, y, lse)
    other = torch.full((4 * V + 5,), NAN, dtype=z.dtype, device="cuda")
    other = other[3:3 + 4 * V].view(4, V)
    assert torch.equal(df2.distill_backward(up, z, ids, y, lse, grad=other), want)
    assert torch.isnan(other._base[:3].float()).all() and torch.isnan(other._base[-2:].float()).all()
    assert torch.equal(df2.distill_backward(up, z, ids, y, lse, grad=z), want)


def test_what_else_a_row_can_hold():
    z, ids, y = _inputs(6, 900, 5, "f32", 5)
    z -= 4000.0
    z[0, 800] = NAN                        # lse is NaN, and with it the gradient
    z[1] = -INF                            # lse is -inf: the softmax is 0 everywhere
    ids[2] = -1                            # no teacher
    z[4, 1:] = -INF
    loss, lse, grad = df2.distill(z, ids, y, grad=True)
    up = torch.tensor([1.0, 1.0, 1.0, 0.0, 1.0, 1.0], device="cuda")
    back = df2.distill_backward(up, z, ids, y, lse)
    assert torch.isnan(lse[0]) and torch.isnan(back[0]).all()
    assert lse[1] == -INF and torch.equal(back[1], grad[1])
    q = torch.zeros(900, device="cuda")
    q[ids[1].long()] = -torch.softmax(y[1], 0)
    assert (back[1] - q).abs().max() < 1e-5
    assert not back[2].any() and not back[3].any()
    for r in (4, 5):
        assert (back[r] - grad[r]).abs().max() <= 2.2e-5 and torch.isfinite(back[r]).all()
    one = back[4].clone()
    one[ids[4].long()] += torch.softmax(y[4], 0)
    want = torch.zeros(900, device="cuda")
    want[0] = 1.0
    assert (one - want).abs().max() < 1e-5
