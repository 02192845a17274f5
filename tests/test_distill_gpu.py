"""The distillation loss and its gradient against their formulas in 64 bits.

Bounds (with T the temperature, z and y the two logits, all over T, in fp32):
  lse: z * c - b is one rounded fused multiply-add with c = log2(e) / T rounded, 2^x is
    good to 2^-22 and the sum of positive terms adds at most 2^-24 a step of a tree of
    depth < 80: 8e-6 in the sum; c's rounding scales lse: 2^-22 * |lse|.
  loss: q and log q are good to 8 * 2^-23 * (1 + |y|), z's and lse's common scale
    cancels but for 2^-22 * |z - lse|, and the sum's 8e-6 stays.
  gradient: an absolute 1e-5 (the sum's 8e-6 and 2^-21 of s * log s, |s log s| < 0.37) and
    q's 8 * 2^-23 * (1 + |y|), times weight / T; in bf16 its unit roundoff, 2^-8, of the value more.
"""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()
    assert df2.take_device_faults() == 0


def _place(x, dtype, pad=0, offset=0):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows, V = x.shape
    buf = torch.full((rows * (V + pad) + offset + 64,), NAN, dtype=dt, device="cuda")
    v = buf[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, :V]
    v.copy_(x.to(dt))
    return v


def _inputs(rows, V, K, dtype, seed, pad=0, offset=0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    z = _place(torch.randn((rows, V), generator=g) * std, dtype, pad, offset)
    y = torch.randn((rows, V), generator=g) * std + z.float().cpu() * 0.5
    val, ids = torch.topk(y, K, dim=1)
    return z, ids.to(torch.int32).cuda(), val.float().cuda()


def _formula(z, ids, y, T, w, up=None):
    """loss, lse and gradient of one row, in 64 bits (numpy)."""
    z, y = z.double().cpu().numpy(), y.double().cpu().numpy()
    ids = ids.cpu().numpy()
    V = len(z)
    if w == 0:
        return 0.0, 0.0, np.zeros(V)
    zt = z / T
    m = zt.max()
    e = np.exp(zt - m) if m > -np.inf else np.zeros(V)
    lse = m + np.log(e.sum()) if m > -np.inf else -np.inf
    s = e / e.sum() if m > -np.inf else e
    use = (ids >= 0) & (ids < V)
    yt = np.where(use, y / T, -np.inf)
    if not (yt > -np.inf).any():
        return 0.0, lse, np.zeros(V)
    lq = yt - yt.max() - np.log(np.exp(yt - yt.max()).sum())
    q = np.exp(lq)
    has = q > 0
    loss = (q[has] * (lq[has] - (zt[ids[has]] - m - np.log(e.sum())))).sum() if m > -np.inf else \
        np.inf
    g = s.copy()
    np.subtract.at(g, ids[use], q[use])
    return w * loss, lse, g * (w if up is None else w * up) / T


def _bounds(z, y, T, lse):
    zt = np.abs(z.double().cpu().numpy()) / T
    yt = np.abs(y.double().cpu().numpy()) / T
    zm, ym = zt[np.isfinite(zt)].max(initial=0), yt[np.isfinite(yt)].max(initial=0)
    q = 8 * 2.0 ** -23 * (1 + ym)
    lse_b = 8e-6 + 2.0 ** -22 * abs(lse) if np.isfinite(lse) else 0
    loss_b = 8e-6 + 2.0 ** -22 * (zm + (abs(lse) if np.isfinite(lse) else 0)) + q * (2 + ym + zm)
    return lse_b, loss_b, 1e-5 + q


def _same(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(got[~fine], ref[~fine], err_msg=str(what))
    err = np.abs(got[fine] - ref[fine])
    lim = np.broadcast_to(bound, ref.shape)[fine]
    assert (err <= lim).all(), (what, float((err - lim).max()), float(err.max()))


def _check(z, ids, y, T=1.0, w=None, up=None, grad_ld=None):
    rows, V = z.shape
    bf = z.dtype == torch.bfloat16
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse, none = df2.distill(z, ids, y, temperature=T, weight=w, err_flag=flag)
    assert none is None
    loss2, lse2, grad = df2.distill(z, ids, y, temperature=T, weight=w, grad=True)
    assert torch.equal(loss.view(torch.int32), loss2.view(torch.int32))
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    ups = torch.linspace(0.5, 2, rows, device="cuda") if up is None else up
    back = df2.distill_backward(ups, z, ids, y, lse, temperature=T, weight=w)
    for r in range(rows):
        wr = 1.0 if w is None else w[r].item()
        ur = ups[r].item()
        rl, rs, rg = _formula(z[r], ids[r], y[r], T, wr)
        lb, ob, gb = _bounds(z[r], y[r], T, rs)
        _same(lse[r].item(), rs, lb, ("lse", r))
        _same(loss[r].item(), rl, abs(wr) * ob + 2.0 ** -23 * abs(rl), ("loss", r))
        rnd = 2.0 ** -8 * np.abs(rg) if bf else 0
        _same(grad[r].double().cpu().numpy(), rg, abs(wr) / T * gb + rnd, ("grad", r))
        # backward takes the rounded lse: its error is the share's, 2^-23 of |lse| more
        gb += 2.0 ** -23 * (abs(rs) if np.isfinite(rs) else 0)
        _same(back[r].double().cpu().numpy(), rg * ur, abs(wr * ur) / T * gb + rnd * abs(ur),
              ("backward", r))
    return loss, lse, grad, int(flag.item())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 2), (7, 3), (33, 33), (257, 16), (1000, 4),
                                 (4099, 64), (20011, 200), (151936, 16), (151936, 1024)])
def test_formula(V, K, dtype):
    for i, T in enumerate((1.0, 0.5, 2.0)):
        z, ids, y = _inputs(3, V, K, dtype, V + i, pad=i, offset=(0, 1, 3)[i])
        _check(z, ids, y, T=T, w=None if i == 0 else torch.tensor([0.3, 0.0, -2.0]).cuda())


@pytest.mark.parametrize("rows", [1, 2, 77, 600])
def test_row_counts(rows):
    z, ids, y = _inputs(rows, 3000, 8, "bf16", rows)
    _check(z, ids, y, w=0.9 ** (torch.arange(rows) % 16).float().cuda())


@pytest.mark.parametrize("V,dtype", [(500_001, "f32"), (1_000_003, "bf16")])
def test_rows_too_wide_for_shared_memory(V, dtype):
    z, ids, y = _inputs(2, V, 40, dtype, 9, pad=1)
    loss, lse, grad, _ = _check(z, ids, y)
    inplace = df2.distill(z, ids, y, grad=z)[2]
    assert inplace is z and torch.equal(z, grad)


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_gradient_against_differences(T):
    """Central differences of the loss, h = 2^-6: the remainder is at most h^2/6 of the third
    derivative (below 0.25/T^3), and twice the loss' bound of 1.3e-5 over 2h."""
    V, K, h = 19, 5, 2.0 ** -6
    z, ids, y = _inputs(1, V, K, "f32", 4)
    grad = df2.distill(z, ids, y, temperature=T, grad=True)[2][0]
    step = torch.eye(V, device="cuda") * h
    up = df2.distill((z + step).contiguous(), ids.expand(V, K).contiguous(),
                     y.expand(V, K).contiguous(), temperature=T)[0]
    down = df2.distill((z - step).contiguous(), ids.expand(V, K).contiguous(),
                       y.expand(V, K).contiguous(), temperature=T)[0]
    diff = (up.double() - down.double()) / (2 * h)
    bound = h * h / 6 * 0.25 / T ** 3 + 1.3e-5 / h
    assert (diff - grad.double()).abs().max().item() <= bound
    assert grad.abs().max().item() > 20 * bound
    assert abs(grad.double().sum().item()) < 1e-5  # shifting all logits changes nothing


def test_tokens_that_stand_in_several_slots():
    z, ids, y = _inputs(3, 500, 40, "f32", 1)
    ids[0, ::3] = ids[0, 0]
    ids[1, :] = 7
    ids[2, 30:] = ids[2, :10]
    _check(z, ids, y)


def test_empty_slots_and_bad_tokens():
    z, ids, y = _inputs(6, 301, 12, "bf16", 2, pad=1)
    ids[0, 5:] = -1
    y[0, 5:] = NAN                 # as topk() pads a row
    ids[1] = -1                    # no teacher at all
    y[2] = -INF                    # nor a share
    y[3, 0] = -INF                 # one slot without a share
    ids[4, 2] = -7
    assert _check(z, ids, y)[3] == 0
    ids[5, 3] = 301                # outside: an empty slot, and flagged
    loss, lse, grad, flag = _check(z, ids, y)
    assert flag == 1
    assert loss[1] == 0 and loss[2] == 0 and not grad[1:3].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_logits(dtype):
    z, ids, y = _inputs(4, 700, 9, dtype, 3, pad=1)
    keep = ids[0].long().cpu()
    mask = torch.ones(700, dtype=torch.bool)
    mask[keep] = False
    z[0, mask.cuda()] = -INF                       # only the teacher's tokens are left
    z[1, ids[1, 4].long()] = -INF                  # one of the teacher's tokens is masked away
    z[2] = -INF                                    # nothing left
    z[3] = torch.finfo(torch.bfloat16).min         # the type's lowest value everywhere
    loss, lse, grad, _ = _check(z, ids, y)
    assert torch.isfinite(loss[0]) and loss[1] == INF and loss[2] == INF and lse[2] == -INF
    q = torch.softmax(y[3].double(), 0)            # against a student that is 1/700 everywhere
    assert abs(loss[3].item() - ((q * q.log()).sum() + np.log(700)).item()) < 1e-5
    assert torch.isfinite(grad).all()


def test_nan_stays_in_its_row_and_weight_zero_hides_it():
    z, ids, y = _inputs(6, 900, 5, "f32", 5)
    z[0, 800] = NAN
    z[1, 3] = INF
    y[2, 4] = NAN
    y[3, 0] = INF
    z[4, :] = NAN
    w = torch.ones(6, device="cuda")
    w[4] = 0
    loss, lse, grad = df2.distill(z, ids, y, weight=w, grad=True)
    assert torch.isnan(loss[:4]).all() and loss[4] == 0 and lse[4] == 0
    assert torch.isnan(grad[0]).all() and not grad[4].any()
    assert torch.isnan(grad[2, ids[2].long()]).all()
    rl, rs, rg = _formula(z[5], ids[5], y[5], 1.0, 1.0)
    assert abs(loss[5].item() - rl) < 1e-4
    up = torch.ones(6, device="cuda")
    up[4] = 0
    back = df2.distill_backward(up, z, ids, y, lse)
    assert not back[4].any() and torch.isfinite(back[5]).all() and torch.isnan(back[0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad,offset", [(1000, 0, 0), (1003, 2, 1), (151936, 0, 0)])
def test_in_place_and_other_spacing(V, pad, offset, dtype):
    z, ids, y = _inputs(3, V, 6, dtype, 7, pad, offset)
    w = torch.tensor([1.0, 0.0, 0.5]).cuda()
    want = df2.distill(z, ids, y, weight=w, grad=True)[2]
    assert want.stride() == z.stride()
    # a gradient whose rows lie elsewhere modulo 16 bytes
    other = _place(torch.zeros((3, V)), dtype, pad + 1, offset + 1)
    assert df2.distill(z, ids, y, weight=w, grad=other)[2] is other
    assert torch.equal(other, want)
    assert torch.isnan(other._base[:offset + 1].float()).all()        # nothing written outside
    gap = other._base[offset + 1:offset + 1 + 3 * (V + pad + 1)].view(3, -1)[:, V:]
    assert torch.isnan(gap.float()).all()
    up = torch.ones(3, device="cuda")
    lse = df2.distill(z, ids, y)[1]
    b1 = df2.distill_backward(up, z, ids, y, lse, weight=w)
    b2 = df2.distill_backward(up, z, ids, y, lse, weight=w, grad=other)
    assert torch.equal(b1, b2)
    z2 = z.clone()
    assert torch.equal(df2.distill_backward(up, z2, ids, y, lse, weight=w, grad=z2), b1)
    df2.distill(z, ids, y, weight=w, grad=z)
    assert torch.equal(z, want)


def test_offsets_beyond_32_bits():
    V, ld = 3000, (1 << 30) + 8
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    z, g = (torch.as_strided(b, (3, V), (ld, 1)) for b in (buf, out))
    y, ids, t = _inputs(3, V, 6, "bf16", 7)
    z.copy_(y)
    a, b = df2.distill(z, ids, t, grad=g), df2.distill(y, ids, t, grad=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_runs_give_the_same_bits_in_any_batch():
    z, ids, y = _inputs(1, 151936, 32, "bf16", 12)
    one = df2.distill(z, ids, y, grad=True)
    again = df2.distill(z, ids, y, grad=True)
    assert all(torch.equal(p, q) for p, q in zip(one, again))


def test_other_stream_leading_dimensions_and_graph():
    z, ids, y = _inputs(6, 2048, 4, "bf16", 1)
    z = z.contiguous().view(2, 3, 2048)
    ids, y = ids.view(2, 3, 4), y.view(2, 3, 4)
    want = df2.distill(z, ids, y, grad=True)
    assert want[0].shape == want[1].shape == (2, 3) and want[2].shape == z.shape
    side, z2 = torch.cuda.Stream(), torch.zeros_like(z)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        z2.copy_(z)
        got = df2.distill(z2, ids, y, grad=True)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    loss, lse, grad = (torch.zeros_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df2.distill(z, ids, y, grad=grad, loss=loss, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, (loss, lse, grad)))


def test_with_the_framework_s_own_top_k():
    z, _, _ = _inputs(5, 4096, 4, "f32", 1)
    t = torch.randn((5, 4096), generator=torch.Generator().manual_seed(2)).cuda()
    t[1, 3:] = NAN                                  # three entries only: topk pads with -1 and NaN
    ids, val = df2.topk(t, 16)
    _check(z, ids, val)


def test_no_rows():
    e = torch.empty((0, 50), device="cuda")
    ids, y = torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda")
    loss, lse, grad = df2.distill(e, ids, y, grad=True)
    assert loss.shape == (0,) and grad.shape == (0, 50)
    assert df2.distill_backward(loss, e, ids, y, lse).shape == (0, 50)


def test_refusals():
    z, ids, y = _inputs(4, 100, 3, "f32", 1)
    z = z.contiguous()
    one = torch.ones(4, device="cuda")
    lse = df2.distill(z, ids, y)[1]
    bad = [dict(logits=z.half()), dict(logits=z.cpu()), dict(logits=z[:, ::2]),
           dict(logits=z[:1].expand(4, 100)), dict(teacher_ids=ids.long()),
           dict(teacher_ids=ids[:3]), dict(teacher_ids=ids[:, :2]), dict(teacher_logits=y.half()),
           dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=INF),
           dict(temperature=NAN), dict(weight=one[:3]), dict(weight=one.double()),
           dict(grad=z.bfloat16()), dict(grad=z[:3]), dict(grad=z.view(-1)[:396].view(4, 99)),
           dict(teacher_ids=ids[:, :0], teacher_logits=y[:, :0])]
    for b in bad:
        args = {"logits": z, "teacher_ids": ids, "teacher_logits": y} | b
        with pytest.raises((ValueError, TypeError, df2.Dflash2Error)):
            df2.distill(**args)
        with pytest.raises((ValueError, TypeError, df2.Dflash2Error)):
            df2.distill_backward(grad_loss=one, lse=lse, **args)
    with pytest.raises((ValueError, TypeError, df2.Dflash2Error)):
        df2.distill_backward(one[:2], z, ids, y, lse)
    with pytest.raises((ValueError, TypeError, df2.Dflash2Error)):
        df2.distill_backward(one, z, ids, y, lse.double())
    shifted = z.view(-1)[4:].view(-1)[:300].view(3, 100)      # overlaps, but is not in place
    with pytest.raises(df2.Dflash2Error):
        df2.distill(z[:3], ids[:3].contiguous(), y[:3].contiguous(), grad=shifted)
