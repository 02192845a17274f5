"""More of the distillation loss: rows without a teacher whose logits are not finite, and
one row in batches that split it in different ways."""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_distill_gpu import INF, NAN, _bounds, _built, _formula, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 900, 151936])
def test_no_teacher_hides_what_is_not_finite(V, dtype):
    """Without a teacher the loss and the gradient are 0, whatever the row holds; with the
    loss, alone, in place, and on another grid."""
    z, ids, y = _inputs(5, V, 4, dtype, 3, pad=1)
    z[0, V // 2] = NAN
    z[1, 0] = INF
    z[2] = INF
    z[3] = NAN
    ids[:4] = -1
    y[0] = NAN
    y[2] = -INF
    ids[2] = 1
    loss, lse, grad = df2.distill(z, ids, y, grad=True)
    assert not loss[:4].any() and not grad[:4].any()
    assert torch.isnan(lse[:4]).all()
    assert torch.isfinite(loss[4]) and torch.isfinite(grad[4]).all() and grad[4].any()
    back = df2.distill_backward(torch.ones(5, device="cuda"), z, ids, y, lse)
    assert not back[:4].any()
    other = torch.full((5 * V + 9,), NAN, dtype=z.dtype, device="cuda")[5:5 + 5 * V].view(5, V)
    assert torch.equal(df2.distill(z, ids, y, grad=other)[2], grad)
    assert torch.equal(df2.distill(z, ids, y, grad=z)[2], grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3000, 151936])
def test_a_row_in_batches_of_other_sizes(V, dtype):
    """The number of rows decides how a row is split, and with it the order of its fp32 sums:
    each result is inside its bound, and a batch's rows are the same bits."""
    z, ids, y = _inputs(1, V, 32, dtype, 12)
    rl, rs, rg = _formula(z[0], ids[0], y[0], 1.0, 1.0)
    lb, ob, gb = _bounds(z[0], y[0], 1.0, rs)
    rnd = 2.0 ** -8 * np.abs(rg) if dtype == "bf16" else 0
    for rows in (1, 64, 640, 1300):
        loss, lse, grad = df2.distill(z.expand(rows, V).contiguous(), ids.expand(rows, 32).contiguous(),
                                      y.expand(rows, 32).contiguous(), grad=True)
        for t in (loss, lse, grad):
            assert (t == t[:1]).all()
        assert abs(lse[0].item() - rs) <= lb and abs(loss[0].item() - rl) <= ob + 2.0 ** -23 * abs(rl)
        assert (np.abs(grad[0].double().cpu().numpy() - rg) <= gb + rnd).all()
