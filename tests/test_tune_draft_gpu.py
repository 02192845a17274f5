"""The operators of training together: the examples run, can be repeated, and their weights'
gradients are those of the formulas; a whole step is captured into a graph beside an eager one."""
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from dflash2_draft_head_gb300 import train_draft, tune_draft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()
    assert df2.take_device_faults() == 0


@pytest.mark.parametrize("optimizer", ["adamw", "adamw8"])
def test_training_by_adamw_runs_and_can_be_repeated(optimizer):
    a, b = (train_draft.train(steps=4, blocks=4, optimizer=optimizer) for _ in range(2))
    assert a == b and all(v == v for v in a["loss"] + a["accepted"])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("method", ["policy", "preference"])
def test_tuning_runs_and_can_be_repeated(method, bits):
    a, b = (tune_draft.tune(steps=4, blocks=4, method=method, bits=bits) for _ in range(2))
    assert a == b and all(v == v for v in a["loss"] + a["accepted"]) and a["norm"] >= 0


def test_unknown_settings_are_refused():
    with pytest.raises(ValueError):
        train_draft.train(optimizer="adam")
    with pytest.raises(ValueError):
        tune_draft.tune(method="reward")


def _head(rows=24, V=300, d=16):
    g = torch.Generator().manual_seed(3)
    h, w = torch.randn((rows, d), generator=g).cuda(), torch.randn((V, d), generator=g).cuda()
    tokens = torch.randint(0, V, (rows,), generator=g).to(torch.int32).cuda()
    return h, w, tokens, g


def test_the_weights_gradient_of_a_policy_step():
    """Through the logits, against autograd on the formula in 64 bits.  Off by the product's
    rounding and the share's 1e-5: 2e-5 of the sum of |h| over the rows is a bound on both."""
    h, w, tokens, g = _head()
    A = torch.randn(24, generator=g).cuda()
    x = w.double().requires_grad_()
    logp = torch.log_softmax(h.double() @ x.t(), 1).gather(1, tokens.long()[:, None]).squeeze(1)
    old, ref = (logp.detach() + 0.1).float(), (logp.detach() - 0.2).float()
    rho, d = torch.exp(logp - old.double()), ref.double() - logp
    (0.1 * (torch.exp(d) - d - 1) - torch.minimum(rho * A, rho.clamp(0.8, 1.2) * A)).sum().backward()
    z = h @ w.t()
    grad = df2.policy_loss(z, tokens, old, A, ref_logp=ref, kl_coef=0.1, grad=True)[3]
    got = grad.t() @ h
    assert (got - x.grad).abs().max() <= 2e-5 * h.abs().sum(0).max() * (1 + A.abs().max())


def test_the_weights_gradient_of_a_preference_step():
    h, w, tokens, _ = _head()
    offsets = torch.tensor([0, 5, 12, 20, 24], dtype=torch.int32, device="cuda")
    x = w.double().requires_grad_()
    logp = torch.log_softmax(h.double() @ x.t(), 1).gather(1, tokens.long()[:, None]).squeeze(1)
    S = torch.stack([p.sum() for p in logp.split([5, 7, 8, 4])])
    ref = (S.detach() + torch.tensor([1.0, -2.0, 0.5, 3.0]).cuda()).float()
    r = S - ref.double()
    torch.nn.functional.softplus(-0.3 * (r[:2] - r[2:])).sum().backward()
    grad = df2.preference_loss(h @ w.t(), tokens, offsets, ref_logp=ref, beta=0.3, grad=True)[4]
    got = grad.t() @ h
    assert (got - x.grad).abs().max() <= 2e-5 * h.abs().sum(0).max() * 2


@pytest.mark.parametrize("method", ["policy", "preference"])
def test_a_whole_step_in_a_graph_beside_an_eager_one(method):
    """Loss, weights' gradient, norm and AdamW with 8-bit states, replayed with other inputs, between
    eager steps on the same gradient function; both sides give the same bits."""
    h, w, tokens, g = _head(rows=32)
    A, old = torch.randn(32, generator=g).cuda(), torch.full((32,), -4.0, device="cuda")
    offsets = torch.arange(0, 33, 8, dtype=torch.int32, device="cuda")
    step = torch.ones(1, dtype=torch.int32, device="cuda")

    def new_state():
        n = w.numel()
        codes = [torch.zeros_like(w, dtype=torch.uint8) for _ in range(2)]
        scales = [torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
        return [w.clone().bfloat16(), codes, scales]

    def one(state, h, tokens):
        p, codes, scales = state
        z = (h @ p.float().t()).bfloat16()
        if method == "policy":
            grad = df2.policy_loss(z, tokens, old, A, grad=z)[3]
        else:
            grad = df2.preference_loss(z, tokens, offsets, grad=z)[4]
        slope = grad.float().t() @ h
        norm = df2.grad_norm([slope])
        df2.adamw([p], [slope], [codes[0]], [codes[1]], step=step, lr=1e-2, norm=norm, max_norm=0.5,
                  exp_avg_scale=[scales[0]], exp_avg_sq_scale=[scales[1]], seed=7)
        return norm

    # a first step outside of capture, on a stream of its own, sets the libraries up
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one(new_state(), h, tokens)
    torch.cuda.current_stream().wait_stream(side)
    eager, captured = new_state(), new_state()
    hh, tt = h.clone(), tokens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graph_norm = one(captured, hh, tt)
    for k in range(3):
        hh.copy_(h.roll(k, 0))
        tt.copy_(tokens.roll(k, 0))
        graph.replay()
        norm = one(eager, hh, tt)
        assert torch.equal(norm, graph_norm)
        assert torch.equal(eager[0], captured[0])
        for a, b in zip(eager[1] + eager[2], captured[1] + captured[2]):
            assert torch.equal(a, b)
        step += 1
