"""More of the distillation loss: rows without a teacher whose logits are not finite."""
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_distill_gpu import INF, NAN, _built, _inputs  # noqa: F401

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
