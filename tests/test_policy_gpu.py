"""The clipped policy loss, its gradient in the same call and the gradient alone, against the
formulas in 64 bits.  The bounds are derived in loss_rows.py."""
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from loss_rows import (INF, NAN, by_numbers, equal_bits, gradient_bound, linspace, logp64,
                       logp_bound, lse_bound, place, policy64_like, rows_of, same)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()
    assert df2.take_device_faults() == 0


RATIOS = [0.3, 0.7, 0.9, 1.0, 1.1, 1.35, 4.0]  # none near 0.8 or 1.2, where the slope jumps


def _around(z, tokens, T, g):
    """old, advantage, ref around the tokens' log-probabilities."""
    rows = z.shape[0]
    logp = torch.nan_to_num(logp64(z, tokens, T)[0], 0, 0, -8).clamp(min=-30)
    rho = torch.tensor(RATIOS).repeat(rows // len(RATIOS) + 1)[:rows].cuda()
    old = (logp - rho.double().log()).float()
    A = (torch.randn(rows, generator=g) * 2).cuda()
    return old, A, (logp + torch.randn(rows, generator=g).cuda() * 0.5).float()


def _check(z, tokens, old, A, ref=None, w=None, T=1.0, lo=0.2, hi=0.2, kl=0.0):
    rows, V = z.shape
    bf = z.dtype == torch.bfloat16
    kw = dict(ref_logp=ref, temperature=T, clip_low=lo, clip_high=hi, kl_coef=kl, weight=w)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, logp, lse, none = df2.policy_loss(z, tokens, old, A, err_flag=flag, **kw)
    assert none is None
    loss2, logp2, lse2, grad = df2.policy_loss(z, tokens, old, A, grad=True, **kw)
    assert equal_bits(loss, loss2) and equal_bits(logp, logp2) and equal_bits(lse, lse2)
    ones = torch.ones(rows, device="cuda") if w is None else w
    rl, rp, rs, rg, g, lb, gb = policy64_like(grad, z, tokens, old, A, ref, ones, T, lo, hi,
                                                kl)
    same(logp, rp, logp_bound(rp), "logp")
    same(lse, rs, lse_bound(rs), "lse")
    same(loss, rl, torch.nan_to_num(lb, 0, 0, 0), "loss")
    same(grad, rg, torch.nan_to_num(gradient_bound(rg, g, gb, T, bf), 0, 0, 0), "grad")
    up = linspace(0.5, 2, rows)
    back = df2.policy_loss_backward(up, z, tokens, old, A, logp, lse, **kw)
    # from the rounded lse and the logp that the loss returned
    _, _, _, rb, g, _, gb = policy64_like(back, z, tokens, old, A, ref, ones, T, lo, hi, kl, up)
    gb = gb + 2.0 ** -23 * g.abs() * torch.nan_to_num(rs, 0, 0, 0).abs()
    same(back, rb, torch.nan_to_num(gradient_bound(rb, g, gb, T, bf), 0, 0, 0), "backward")
    return loss, logp, lse, grad, int(flag)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 257, 1000, 4099, 20011, 151936])
def test_formula(V, dtype):
    for i, T in enumerate((1.0, 0.5, 2.0)):
        z, tokens, g = rows_of(7, V, dtype, V + i, pad=i, offset=(0, 1, 3)[i])
        old, A, ref = _around(z, tokens, T, g)
        w = None if i == 0 else by_numbers([0.3, 0.0, -2.0, 1.0, 0.1, 5.0, 0.7])[0]
        _check(z, tokens, old, A, ref, w, T, kl=(0.04, 0.0, 0.5)[i])


@pytest.mark.parametrize("rows", [1, 2, 77, 600])
def test_row_counts(rows):
    z, tokens, g = rows_of(rows, 2999, "bf16", rows)
    old, A, ref = _around(z, tokens, 1.0, g)
    _check(z, tokens, old, A, ref, 0.9 ** (torch.arange(rows) % 16).float().cuda(), kl=0.1)


@pytest.mark.parametrize("V,dtype", [(500_001, "f32"), (1_000_003, "bf16")])
def test_rows_too_wide_for_shared_memory(V, dtype):
    z, tokens, g = rows_of(2, V, dtype, 9, pad=1)
    old, A, ref = _around(z, tokens, 1.0, g)
    grad = _check(z, tokens, old, A, ref, kl=0.1)[3]
    assert df2.policy_loss(z, tokens, old, A, ref_logp=ref, kl_coef=0.1, grad=z)[3] is z
    assert torch.equal(z, grad)


def test_no_rows():
    z = torch.empty((0, 50), device="cuda")
    e, t = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    loss, logp, lse, grad = df2.policy_loss(z, t, e, e, grad=True)
    assert loss.shape == logp.shape == lse.shape == (0,) and grad.shape == (0, 50)
    assert df2.policy_loss_backward(e, z, t, e, e, logp, lse).shape == (0, 50)


@pytest.mark.parametrize("lo,hi", [(0.2, 0.2), (0.0, 0.0), (0.1, 0.3), (1.0, 5.0), (INF, INF)])
def test_both_sides_of_the_clamp(lo, hi):
    """Every ratio with both signs of the advantage, and none: the slope is 0 exactly where the
    clamp lowers the loss' gain."""
    ratios = torch.tensor([r for r in RATIOS if r != 1.0] * 3).cuda()
    rows = ratios.numel()
    z, tokens, _ = rows_of(rows, 501, "f32", 3)
    A = torch.tensor([1.5] * (rows // 3) + [-0.5] * (rows // 3) + [0.0] * (rows // 3)).cuda()
    old = (logp64(z, tokens, 1.0)[0] - ratios.double().log()).float()
    loss, _, _, grad, _ = _check(z, tokens, old, A, lo=lo, hi=hi)
    held = (A > 0) & (ratios > 1 + hi) | (A < 0) & (ratios < 1 - lo) | (A == 0)
    # 0.9 lies on the edge of 1 - 0.1: both slopes are right there
    edge = (A < 0) & ((ratios.double() - (1 - lo)).abs() < 1e-4)
    assert torch.equal((grad == 0).all(1)[~edge], held[~edge])
    assert not loss[A == 0].any()


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_gradient_against_differences(T):
    """Central differences of the loss in 64 bits of its fp32 values, h = 2^-6: the remainder is
    at most h^2/6 of the third derivative (below 2/T^3 for |A| rho and kl_coef exp(d) below
    0.5 each), and twice the loss' bound of 2e-5 over 2h."""
    V, h = 19, 2.0 ** -6
    z, tokens, g = rows_of(1, V, "f32", 4)
    logp = logp64(z, tokens, T)[0].float()
    old, A, ref = logp - 0.05, torch.tensor([0.4]).cuda(), logp + 0.3

    def loss(x):
        n = x.shape[0]
        return df2.policy_loss(x.contiguous(), tokens.expand(n).contiguous(),
                               old.expand(n).contiguous(), A.expand(n).contiguous(),
                               ref_logp=ref.expand(n).contiguous(), temperature=T, kl_coef=0.3)[0]

    grad = df2.policy_loss(z, tokens, old, A, ref_logp=ref, temperature=T, kl_coef=0.3,
                           grad=True)[3][0]
    step = torch.eye(V, device="cuda") * h
    diff = (loss(z + step).double() - loss(z - step).double()) / (2 * h)
    bound = h * h / 6 * 2 / T ** 3 + 2e-5 / h
    assert (diff - grad.double()).abs().max().item() <= bound
    assert grad.abs().max().item() > 20 * bound
    assert abs(grad.double().sum().item()) < 1e-5  # shifting all logits changes nothing


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_a_token(dtype):
    z, tokens, g = rows_of(6, 301, dtype, 2, pad=1)
    old, A, ref = _around(z, tokens, 1.0, g)
    tokens[1], tokens[3] = -1, -7
    z[1], z[4] = NAN, NAN                     # not read
    w = by_numbers([1.0, 1.0, 2.0, 1.0, 0.0, 0.5])[0]
    old[1] = A[3] = NAN
    assert _check(z, tokens, old, A, ref, w, kl=0.1)[4] == 0
    tokens[5] = 301                           # outside: not counted, and flagged
    loss, logp, lse, grad, flag = _check(z, tokens, old, A, ref, w, kl=0.1)
    assert flag == 1
    for r in (1, 3, 4, 5):
        assert loss[r] == 0 and logp[r] == 0 and lse[r] == 0 and not grad[r].any()
    tokens[5] = 2 ** 31 - 1
    assert _check(z, tokens, old, A, ref, w, kl=0.1)[4] == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_logits(dtype):
    z, tokens, g = rows_of(6, 700, dtype, 3, pad=1)
    old, A, ref = _around(z, tokens, 1.0, g)
    mask = torch.ones(700, dtype=torch.bool, device="cuda")
    mask[tokens[0].long()] = False
    z[0, mask] = -INF                              # the token alone is left
    z[1, tokens[1].long()] = -INF                  # the token is masked away
    z[2] = -INF                                    # nothing is left
    z[3] = torch.finfo(torch.bfloat16).min         # the type's lowest value everywhere
    z[4, :350] = torch.finfo(torch.bfloat16).min
    A[:] = 1.0
    loss, logp, lse, grad, _ = _check(z, tokens, old, A)
    # the bound of logp near 0: the multiply-add leaves the base's rounding in both its terms
    assert -8e-6 <= logp[0].item() <= 0 and logp[1] == -INF and logp[2] == -INF and lse[2] == -INF
    assert abs(logp[3].item() + torch.tensor(700.0).log().item()) < 1e-5
    assert loss[1] == 0 and loss[2] == 0 and torch.isfinite(grad).all()
    A[:] = -1.0                                    # the clamp holds a ratio of 0
    loss = _check(z, tokens, old, A)[0]
    assert abs(loss[1].item() - 0.8) < 1e-6
    # the divergence from a reference that gives a masked token a share is infinite
    loss, *_ = df2.policy_loss(z, tokens, old, A, ref_logp=ref, kl_coef=0.1)
    # (exp(d) is infinite as well where the token of row 4 is among those at the lowest value)
    low = tokens[4] < 350
    assert loss[1] == INF and torch.isfinite(loss[[0, 3, 5]]).all()
    assert torch.isfinite(loss[4]) != low


@pytest.mark.parametrize("bad", [NAN, INF])
def test_what_is_not_a_number_stays_visible(bad):
    z, tokens, g = rows_of(3, 1500, "f32", 5)
    old, A, ref = _around(z, tokens, 1.0, g)
    z[1, 777] = bad
    tokens[1] = 777
    for kl in (0.0, 0.1):
        loss, logp, lse, grad = df2.policy_loss(z, tokens, old, A, ref_logp=ref, kl_coef=kl,
                                                grad=True)
        assert torch.isnan(loss[1]) and torch.isnan(logp[1]) and torch.isnan(grad[1]).all()
        assert torch.isfinite(grad[[0, 2]]).all() and torch.isfinite(loss[[0, 2]]).all()


def test_ratios_beyond_fp32():
    """exp(logp - old) overflows: the clamp holds it for A > 0, and A = 0 leaves it out."""
    z, tokens, g = rows_of(3, 400, "f32", 6)
    logp = logp64(z, tokens, 1.0)[0].float()
    old = logp - 200
    A = by_numbers([2.0, 0.0, -1.0])[0]
    loss, _, _, grad = df2.policy_loss(z, tokens, old, A, grad=True)
    assert abs(loss[0].item() + 2.4) < 1e-6 and loss[1] == 0 and loss[2] == INF
    assert not grad[:2].any()


@pytest.mark.parametrize("shift", [300.0, -1e4, 1e6])
def test_logits_far_from_zero(shift):
    """A common shift of a row changes nothing but lse: what of the logits' spacing at the shift is
    lost is lost before the call."""
    z, tokens, g = rows_of(5, 5000, "f32", 7, std=2.0)
    z.copy_(((z + shift) * 4).round() / 4)        # exact at any of the shifts
    old, A, ref = _around(z, tokens, 1.0, g)
    loss, logp, lse, grad, _ = _check(z, tokens, old, A, ref, kl=0.1)
    near = df2.policy_loss((z - shift).contiguous(), tokens, old, A, ref_logp=ref, kl_coef=0.1,
                           grad=True)
    assert (near[3] - grad).abs().max() <= 4e-5 * A.abs().max() * 4
    back = df2.policy_loss_backward(torch.ones(5, device="cuda"), z, tokens, old, A, logp, lse,
                                    ref_logp=ref, kl_coef=0.1)
    assert (back - grad).abs().max() <= 4e-5 * A.abs().max() * 4


@pytest.mark.parametrize("V,dtype", [(4099, "f32"), (151936, "bf16")])
def test_in_place_and_what_lies_around(V, dtype):
    z, tokens, g = rows_of(9, V, dtype, 8, pad=5, offset=3)
    old, A, ref = _around(z, tokens, 1.0, g)
    loss, logp, lse, grad = df2.policy_loss(z, tokens, old, A, grad=True)
    up = torch.ones(9, device="cuda")
    for alone in (False, True):
        y = place(z.float(), dtype, pad=5, offset=3)
        around = y._base.clone()
        if alone:
            df2.policy_loss_backward(up, y, tokens, old, A, logp, lse, grad=y)
            assert torch.equal(y, df2.policy_loss_backward(up, z, tokens, old, A, logp, lse))
        else:
            df2.policy_loss(y, tokens, old, A, grad=y)
            assert torch.equal(y, grad)
        now = y._base.clone()
        view = around[3:3 + 9 * (V + 5)].view(9, V + 5)
        assert torch.isnan(now[:3]).all() and torch.isnan(now[3 + 9 * (V + 5):]).all()
        assert torch.isnan(now[3:3 + 9 * (V + 5)].view(9, V + 5)[:, V:]).all()
        assert torch.isnan(view[:, V:]).all()


def test_the_same_rows_give_the_same_bits():
    """In a batch of the same number of rows that start alike, whatever the others are; and
    every time."""
    z, tokens, g = rows_of(64, 20008, "bf16", 10)
    old, A, ref = _around(z, tokens, 1.0, g)
    kw = dict(ref_logp=ref, kl_coef=0.1, grad=True)
    a = df2.policy_loss(z, tokens, old, A, **kw)
    b = df2.policy_loss(z, tokens, old, A, **kw)
    assert all(equal_bits(x, y) for x, y in zip(a, b))
    perm = torch.randperm(64, generator=g).cuda()
    c = df2.policy_loss(z[perm].contiguous(), tokens[perm], old[perm], A[perm],
                        ref_logp=ref[perm], kl_coef=0.1, grad=True)
    assert all(equal_bits(x[perm], y) for x, y in zip(a, c))


def test_another_stream_and_a_captured_graph():
    z, tokens, g = rows_of(20, 9001, "bf16", 11)
    old, A, ref = _around(z, tokens, 1.0, g)
    want = df2.policy_loss(z, tokens, old, A, ref_logp=ref, kl_coef=0.1, grad=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = df2.policy_loss(z, tokens, old, A, ref_logp=ref, kl_coef=0.1, grad=True)
    torch.cuda.current_stream().wait_stream(side)
    assert all(equal_bits(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    y, t = z.clone(), tokens.clone()
    with torch.cuda.graph(graph):
        out = df2.policy_loss(y, t, old, A, ref_logp=ref, kl_coef=0.1, grad=True)
        back = df2.policy_loss_backward(torch.ones_like(old), y, t, old, A, out[1], out[2],
                                        ref_logp=ref, kl_coef=0.1)
    for k in range(3):
        y.copy_(z.roll(k, 0))
        t.copy_(tokens.roll(k, 0))
        graph.replay()
        want = df2.policy_loss(y, t, old, A, ref_logp=ref, kl_coef=0.1, grad=True)
        assert all(equal_bits(a, b) for a, b in zip(want, out))
        assert equal_bits(back, df2.policy_loss_backward(
            torch.ones_like(old), y, t, old, A, want[1], want[2], ref_logp=ref, kl_coef=0.1))


def test_leading_dimensions_and_given_outputs():
    z, tokens, g = rows_of(12, 600, "f32", 12)
    old, A, ref = _around(z, tokens, 1.0, g)
    want = df2.policy_loss(z, tokens, old, A, grad=True)
    out = [torch.full((3, 4), NAN, device="cuda") for _ in range(3)]
    grad = torch.full((3, 4, 600), NAN, device="cuda")
    got = df2.policy_loss(z.view(3, 4, 600), tokens.view(3, 4), old.view(3, 4), A.view(3, 4),
                          grad=grad, loss=out[0], logp=out[1], lse=out[2])
    assert got[3] is grad and all(a is b for a, b in zip(got, out))
    assert all(equal_bits(a, b.view(a.shape)) for a, b in zip(got, want))


def test_a_single_row_without_leading_dimensions_and_spaced_views():
    z, tokens, g = rows_of(12, 600, "bf16", 14, pad=8)
    old, A, ref = _around(z, tokens, 1.0, g)
    want = df2.policy_loss(z[:1], tokens[:1], old[:1], A[:1], grad=True)
    one = df2.policy_loss(z[0], tokens[0], old[0], A[0], grad=True)
    assert one[0].shape == () and one[3].shape == (600,)
    assert all(equal_bits(a.view(b.shape), b) for a, b in zip(one, want))
    # every third row, and a view of three dimensions, of a padded buffer
    for view, t in ((z[::3], slice(None, None, 3)), (z.unflatten(0, (3, 4)), slice(None))):
        shape = view.shape[:-1]
        tt, oo, aa = (v[t].contiguous().view(shape) for v in (tokens, old, A))
        got = df2.policy_loss(view, tt, oo, aa, grad=True)
        flat = df2.policy_loss(view.reshape(-1, 600).contiguous(), tt.view(-1), oo.view(-1),
                               aa.view(-1), grad=True)
        assert all(equal_bits(a.reshape(b.shape), b) for a, b in zip(got, flat))


def test_beside_autograd():
    g = torch.Generator().manual_seed(1)
    h = torch.randn((6, 8), generator=g).cuda()
    w = torch.randn((500, 8), generator=g).cuda().requires_grad_()
    z = h @ w.t()
    tokens = torch.arange(6, dtype=torch.int32, device="cuda")
    old = logp64(z.detach(), tokens, 1.0)[0].float()
    A = linspace(-1, 1, 6)
    loss, logp, lse, grad = df2.policy_loss(z, tokens, old, A, grad=True)
    assert not loss.requires_grad and not grad.requires_grad
    later = (z * z).sum()
    z.backward(grad, retain_graph=True)
    assert torch.allclose(w.grad, grad.t() @ h, rtol=1e-5, atol=1e-6)
    before = z._version
    df2.policy_loss(z, tokens, old, A, grad=z)
    df2.policy_loss_backward(A, z, tokens, old, A, logp, lse, grad=z)
    assert z._version == before + 2
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        later.backward()


def test_refusals():
    z, tokens, g = rows_of(4, 50, "f32", 13)
    f = torch.zeros(4, device="cuda")
    ok = (z, tokens, f, f)
    for bad in [(z.half(), tokens, f, f), (z, tokens.long(), f, f), (z, tokens, f.double(), f),
                (z, tokens[:3], f, f), (z, tokens, f, f[:2]), (z, tokens.cpu(), f, f),
                (z.t(), tokens, f, f)]:
        with pytest.raises((TypeError, ValueError)):
            df2.policy_loss(*bad)
    for kw in [dict(kl_coef=0.1), dict(temperature=0.0), dict(clip_low=-0.1), dict(clip_high=NAN),
               dict(kl_coef=INF, ref_logp=f), dict(loss=f), dict(weight=f, lse=f)]:
        with pytest.raises(df2.Dflash2Error):
            df2.policy_loss(*ok, **kw)
    for kw in [dict(grad=torch.empty(4, 50, device="cuda", dtype=torch.bfloat16)),
               dict(grad=torch.empty(4, 49, device="cuda")), dict(weight=f[:1])]:
        with pytest.raises((TypeError, ValueError)):
            df2.policy_loss(*ok, **kw)
