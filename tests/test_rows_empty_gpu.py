"""Sampling and distillation of batches without rows, of any shape."""
import pytest
import torch

import dflash2_draft_head_gb300 as df2

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lead", [(0,), (5, 0), (0, 5), (5, 0, 3), (0, 0)])
def test_no_rows(lead):
    df2.build_library()
    z = torch.empty(lead + (100,), device="cuda")
    one = torch.empty(lead, device="cuda")
    tok, prob = df2.sample(z, one, top_p=0.9)
    assert tok.shape == prob.shape == lead and tok.dtype == torch.int32
    ids = torch.empty(lead + (4,), dtype=torch.int32, device="cuda")
    y = torch.empty(lead + (4,), device="cuda")
    loss, lse, grad = df2.distill(z, ids, y, grad=True)
    assert loss.shape == lse.shape == lead and grad.shape == z.shape
    assert df2.distill_backward(one, z, ids, y, lse).shape == z.shape
    assert df2.distill(z, ids, y, grad=z)[2] is z
