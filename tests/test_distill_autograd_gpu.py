"""How distill() and distill_backward() stand beside PyTorch's autograd: they make no graph,
their gradient is handed on by the caller, and autograd learns of a gradient that was
written over the logits."""
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from test_distill_gpu import _built, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu


def _head(rows=6, V=500, d=8):
    g = torch.Generator().manual_seed(1)
    h = torch.randn((rows, d), generator=g).cuda()
    w = torch.randn((V, d), generator=g).cuda().requires_grad_()
    _, ids, y = _inputs(rows, V, 4, "f32", 2)
    return h, w, ids, y


def test_the_gradient_is_handed_on():
    h, w, ids, y = _head()
    z = h @ w.t()
    loss, _, grad = df2.distill(z, ids, y, grad=True)
    assert not loss.requires_grad and not grad.requires_grad
    z.backward(grad)
    assert torch.allclose(w.grad, grad.t() @ h, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("alone", [False, True])
def test_autograd_sees_a_gradient_over_saved_logits(alone):
    h, w, ids, y = _head()
    z = h @ w.t()
    later = (z * z).sum()                  # keeps z for its own backward
    lse = df2.distill(z.detach(), ids, y)[1]
    before = z._version
    if alone:
        df2.distill_backward(torch.ones(6, device="cuda"), z, ids, y, lse, grad=z)
    else:
        df2.distill(z, ids, y, grad=z)
    assert z._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        later.backward()


def test_tensors_of_inference_mode_are_taken():
    h, w, ids, y = _head()
    with torch.inference_mode():
        z = h @ w.t()
        want = df2.distill(z, ids, y, grad=True)[2]
        assert torch.equal(df2.distill(z, ids, y, grad=z)[2], want)
