"""The distillation loss and its gradient on rows whose logits are large next to their
differences, against the formula in 64 bits (see test_distill_gpu.py).

Bounds: a row's shares, and with them the loss and the gradient, depend on differences
of its logits only.  With D the largest |z - max z| / T of an entry with a share above
2^-40: loss 8e-6 + 2^-22 * (D + log V) + q's part, gradient 1e-5 and q's, times |weight| / T; lse 8e-6
and 2^-22 of itself.  Only the last one grows with the logits."""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_distill_gpu import _bounds, _built, _formula, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu

# log2(e) * 11629080 is 2^24
VALUES = [1e6, 1.16e7, 1.17e7, 1e9, 3e9, 1e10, 7.7e11, 1e20, 1e30, 1e37, 3e38]


def _check(z, ids, y, T=1.0, w=None):
    rows, V = z.shape
    loss, lse, none = df2.distill(z, ids, y, temperature=T, weight=w)
    loss2, lse2, grad = df2.distill(z, ids, y, temperature=T, weight=w, grad=True)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    for r in range(rows):
        wr = 1.0 if w is None else w[r].item()
        rl, rs, rg = _formula(z[r], ids[r], y[r], T, wr)
        zt = z[r].double().cpu().numpy() / T
        d = zt.max() - zt
        D = d[d < 40 * np.log(2)].max() + np.log(V)
        gb = _bounds(z[r], y[r], T, 0.0)[2]
        tb = np.abs(d[ids[r].cpu().numpy()]).max()      # the teacher's tokens, any share
        ym = np.abs(y[r].double().cpu().numpy()).max() / T
        lb = 8e-6 + 2.0 ** -22 * (D + tb) + (gb - 1e-5) * (2 + ym + D + tb)
        assert abs(loss[r].item() - rl) <= abs(wr) * lb + 2.0 ** -23 * abs(rl), (r, loss[r], rl)
        with np.errstate(over="ignore"):
            rs32 = np.float32(rs)
        if np.isinf(rs32):                              # beyond fp32
            assert lse[r].item() == rs32
        else:
            assert abs(lse[r].item() - rs) <= 8e-6 + 2.0 ** -22 * abs(rs), (r, lse[r], rs)
        rnd = 2.0 ** -8 * np.abs(rg) if z.dtype == torch.bfloat16 else 0
        err = np.abs(grad[r].double().cpu().numpy() - rg)
        assert (err <= abs(wr) / T * gb + rnd).all(), (r, err.max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 0.5, 3.0])
@pytest.mark.parametrize("V", [5, 700, 60_001, 151936])
def test_rows_of_one_value(V, T, dtype):
    """Every share is 1 / V, whatever the value."""
    values = VALUES if V < 100_000 else VALUES[1::3]
    z, ids, y = _inputs(2 * len(values), V, min(V, 9), dtype, V, pad=1)
    for i, v in enumerate(values):
        z[2 * i], z[2 * i + 1] = -v, v
    _check(z, ids, y, T)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("V", [3000, 40_000])
def test_parts_of_a_row_on_both_sides_of_a_limit(V, sign):
    """fp32 logits are whole numbers near 2^24 / log2(e): eighths of the row whose largest ones
    lie a few units apart, with the shares that follow from them."""
    rows = 9
    z, ids, y = _inputs(rows, V, 9, "f32", V + 3)
    g = torch.Generator().manual_seed(V)
    part = (torch.arange(V) * 8 // V).float()
    for r in range(rows):
        lift = part if r % 2 == 0 else 7 - part
        near = torch.randint(0, 2, (V,), generator=g).float()
        z[r] = (sign * 11629080 + (r - 4) + lift - 4 + near).cuda()
    _check(z, ids, y, w=torch.linspace(0.5, 1.5, rows, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_masked_by_large_numbers(dtype):
    """One in 16 entries is left of a row, or none: what masks the others is far below."""
    z, ids, y = _inputs(12, 5000, 6, dtype, 4, pad=3, offset=1)
    g = torch.Generator().manual_seed(1)
    gone = (torch.rand((12, 5000), generator=g) > 1 / 16).cuda()
    gone.scatter_(1, ids.long(), False)                 # the teacher's tokens stay
    for r, low in enumerate((-1e4, -1e9, -1e10, -1e20, -1e30, -3e38)):
        z[2 * r].masked_fill_(gone[2 * r], low)
        z[2 * r + 1] = low
    _check(z, ids, y)
