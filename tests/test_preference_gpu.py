"""The preference loss of pairs of sequences, its gradient in the same call and the gradient
alone, against the formulas in 64 bits.  The bounds of logp and of the gradient's shares
are derived in loss_rows.py; on top of them:
  S: the sum of the rows' bounds, and one rounding (2^-24 of the result); a mean: over the number
  margin m, in the loss: beta times both sequences' bounds, and 2^-23 of m; in the gradient also the
    roundings of S and of both differences to fp32: 2^-23 of |S| and of |ref| in each sequence
  loss: m's error (its slope is below 1), and 2^-20 of it
  slope: beta / 4 times m's error, and 2^-20 of it
"""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from loss_rows import (INF, NAN, by_numbers, equal_bits, gradient64, gradient_bound, linspace,
                       logp64, logp_bound, lse_bound, place, rows_of, same)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()
    assert df2.take_device_faults() == 0


def _offsets(lengths, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lengths)]), dtype=torch.int32,
                        device="cuda")


def _formula(z, tokens, offsets, ref, w, beta, e, margin, average, up=None):
    P = offsets.numel() // 2
    logp, lse, share = logp64(z, tokens, 1.0)
    used = (tokens >= 0) & (tokens < z.shape[1])
    logp, lse = torch.where(used, logp, 0.0), torch.where(used, lse, 0.0)
    at = offsets.tolist()
    S, Sb, n = [], [], []
    for a, b in zip(at, at[1:]):
        k = max(1, int(used[a:b].sum())) if average else 1
        S.append(logp[a:b].sum() / k)
        Sb.append((logp_bound(logp[a:b]) * used[a:b]).sum() / k)
        n.append(k)
    S, Sb = torch.stack(S), torch.stack(Sb) if Sb else None
    fin = torch.nan_to_num(S, 0, 0, 0).abs()
    r = torch.zeros_like(S) if ref is None else ref.double()
    d = S - r
    m = beta * (d[:P] - d[P:]) - margin
    fm = torch.nan_to_num(m, 0, 0, 0).abs()
    w = torch.ones_like(m) if w is None else w.double()
    soft = torch.nn.functional.softplus
    loss = (1 - e) * soft(-m) + (e * soft(m) if e else 0.0)
    loss = torch.where(w == 0, 0.0, w * loss)
    mb = beta * (Sb[:P] + Sb[P:]) + 2.0 ** -23 * fm + 2.0 ** -23 * abs(margin)
    lb = w.abs() * mb + 2.0 ** -20 * torch.nan_to_num(loss, 0, 0, 0).abs()
    slope = -beta * w * ((1 - e) * torch.sigmoid(-m) - (e * torch.sigmoid(m) if e else 0.0))
    slope = torch.where(w == 0, 0.0, slope)
    rounding = 2.0 ** -23 * (fin + r.abs())
    gmb = mb + beta * 2 * (rounding[:P] + rounding[P:])
    sb = beta * w.abs() / 4 * gmb + 2.0 ** -20 * beta * w.abs()
    if up is not None:
        slope, sb = slope * up.double(), sb * up.double().abs()
    g, gb = torch.zeros_like(logp), torch.zeros_like(logp)
    for s, (a, b) in enumerate(zip(at, at[1:])):
        i, sign = (s, 1) if s < P else (s - P, -1)
        g[a:b] = torch.where(used[a:b], sign * slope[i] / n[s], 0.0)
        gb[a:b] = sb[i] / n[s]
    return dict(loss=loss, seq=S, logp=logp, lse=lse, grad=gradient64(share, tokens, g, 1.0), g=g,
                loss_bound=lb, seq_bound=Sb + 2.0 ** -24 * fin, g_bound=gb)


def _check(z, tokens, offsets, ref=None, w=None, beta=0.1, e=0.0, margin=0.0, average=False):
    bf = z.dtype == torch.bfloat16
    kw = dict(ref_logp=ref, beta=beta, label_smoothing=e, margin=margin, average=average, weight=w)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, seq, logp, lse, none = df2.preference_loss(z, tokens, offsets, err_flag=flag, **kw)
    assert none is None
    *again, grad = df2.preference_loss(z, tokens, offsets, grad=True, **kw)
    assert all(equal_bits(a, b) for a, b in zip(again, (loss, seq, logp, lse)))
    f = _formula(z, tokens, offsets, ref, w, beta, e, margin, average)
    same(logp, f["logp"], logp_bound(f["logp"]), "logp")
    same(lse, f["lse"], lse_bound(f["lse"]), "lse")
    same(seq, f["seq"], f["seq_bound"], "seq_logp")
    same(loss, f["loss"], f["loss_bound"], "loss")
    far = 2.0 ** -23 * torch.nan_to_num(f["lse"], 0, 0, 0).abs()  # a share by the rounded lse
    same(grad, f["grad"], gradient_bound(f["grad"], f["g"], f["g_bound"] + far * f["g"].abs(), 1.0,
                                         bf), "grad")
    up = linspace(0.5, 2, loss.numel())
    back = df2.preference_loss_backward(up, z, tokens, offsets, seq, lse, **kw)
    b = _formula(z, tokens, offsets, ref, w, beta, e, margin, average, up)
    same(back, b["grad"], gradient_bound(b["grad"], b["g"], b["g_bound"] + far * b["g"].abs(), 1.0,
                                         bf), "backward")
    return loss, seq, logp, lse, grad, int(flag)


def _ref(z, tokens, offsets, average, g, spread=3.0):
    logp = torch.where(tokens >= 0, logp64(z, tokens, 1.0)[0], 0.0)
    at = offsets.tolist()
    S = [logp[a:b].sum() / (max(1, int((tokens[a:b] >= 0).sum())) if average else 1)
         for a, b in zip(at, at[1:])]
    return (torch.stack(S).float() + torch.randn(len(S), generator=g).cuda() * spread)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 33, 1000, 4099, 20011, 151936])
def test_formula(V, dtype):
    lengths = [3, 1, 4, 2, 5, 2]
    for i, average in enumerate((False, True)):
        z, tokens, g = rows_of(18, V, dtype, V + i, pad=i, offset=(0, 3)[i])
        offsets = _offsets(lengths)
        tokens[[0, 4, 9]] = -1
        ref = _ref(z, tokens, offsets, average, g)
        w = None if i == 0 else by_numbers([0.5, 0.0, -2.0])[0]
        _check(z, tokens, offsets, ref, w, beta=(0.1, 2.0)[i], e=(0.0, 0.1)[i],
               margin=(0.0, 0.5)[i], average=average)


@pytest.mark.parametrize("lengths", [[1, 1], [0, 1], [0, 0], [700, 3], [2, 700], [0, 5, 0, 0, 3, 9],
                                     [1] * 66, [257, 256, 1, 255]])
def test_lengths(lengths):
    rows = sum(lengths)
    z, tokens, g = rows_of(max(rows, 1), 515, "f32", rows)
    z, tokens = z[:rows], tokens[:rows]
    tokens[::3] = -1
    offsets = _offsets(lengths)
    for average in (False, True):
        _check(z, tokens, offsets, _ref(z, tokens, offsets, average, g), average=average)


def test_many_pairs():
    """More offsets than one and than two turns of the search look at."""
    rng = np.random.default_rng(0)
    lengths = rng.integers(0, 3, 2 * 1100)
    z, tokens, g = rows_of(int(lengths.sum()), 65, "bf16", 1)
    offsets = _offsets(lengths)
    _check(z, tokens, offsets, _ref(z, tokens, offsets, False, g), beta=0.7)


@pytest.mark.parametrize("V,dtype", [(500_001, "f32"), (1_000_003, "bf16")])
def test_rows_too_wide_for_shared_memory(V, dtype):
    z, tokens, g = rows_of(3, V, dtype, 9, pad=1)
    offsets = _offsets([1, 2])
    grad = _check(z, tokens, offsets, None, beta=0.5)[4]
    df2.preference_loss(z, tokens, offsets, beta=0.5, grad=z)
    assert torch.equal(z, grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_outside_all_sequences(dtype):
    z, tokens, g = rows_of(12, 300, dtype, 2, pad=1)
    offsets = _offsets([2, 3, 1, 2], first=2)   # rows 0, 1, 10 and 11 are in none
    z[11] = NAN
    tokens[1] = tokens[11] = -1
    loss, seq, logp, lse, grad, flag = _check(z, tokens, offsets, _ref(z[:10], tokens[:10], offsets,
                                                                       False, g))
    assert flag == 0 and logp[0] != 0 and logp[11] == 0
    assert not grad[[0, 1, 10, 11]].any()
    tokens[3], tokens[4] = 300, 2 ** 31 - 1     # not in the vocabulary
    *_, grad, flag = _check(z, tokens, offsets)
    assert flag == 1 and not grad[[3, 4]].any()


@pytest.mark.parametrize("at", [[0, 3, 2, 5, 6], [-1, 2, 3, 5, 6], [0, 2, 3, 5, 7],
                                [6, 5, 3, 2, 0], [2 ** 31 - 1, -2 ** 31, 0, 2 ** 31 - 1, 3]])
def test_bad_offsets_are_flagged_and_touch_nothing_else(at):
    z, tokens, _ = rows_of(6, 200, "f32", 3, pad=2, offset=1)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    around = torch.isnan(z._base)               # everything but the rows
    _, seq, _, lse, _ = df2.preference_loss(z, tokens, offsets, grad=True, err_flag=flag)
    assert int(flag) == 1
    df2.preference_loss_backward(torch.ones(2, device="cuda"), z, tokens, offsets, seq, lse, grad=z)
    assert torch.isnan(z._base[around]).all()


@pytest.mark.parametrize("average", [False, True])
def test_gradient_against_differences(average):
    """Central differences of the loss, h = 2^-6: the remainder is at most h^2/6 of the third
    derivative (below 2 for beta = 1: that of log(1 + exp) is 0.1, of logp 0.25, products
    with three of logp's slopes 1), and twice the loss' bound over 2h.  With 11 logits a row's logp is
    off by 2^-22 for the powers, 8 roundings of 2^-24 for their sum and 2^-22 of |logp| < 6 beside:
    2.2e-6; there are 4 rows, and the sums' and the loss' own rounding, 2^-22 of 10 each."""
    V, h = 11, 2.0 ** -6
    z, tokens, _ = rows_of(5, V, "f32", 4, std=1.5)
    tokens[1] = -1
    offsets = _offsets([3, 2])
    grad = df2.preference_loss(z, tokens, offsets, beta=1.0, average=average, label_smoothing=0.1,
                               grad=True)[4]

    def loss(x):
        return df2.preference_loss(x, tokens, offsets, beta=1.0, average=average,
                                   label_smoothing=0.1)[0].double().item()

    bound = h * h / 6 * 2 + (4 * 2.2e-6 + 3 * 2.4e-6) / h
    for r in range(5):
        for j in range(V):
            up, down = z.clone(), z.clone()
            up[r, j] += h
            down[r, j] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - grad[r, j].item()) <= bound, (r, j)
    assert not grad[1].any() and grad.abs().max().item() > 10 * bound


def test_infinite_margins():
    """A masked token makes its sequence's sum -inf: the loss of a chosen one is infinite, of a
    rejected one 0, and the gradients stay finite."""
    z, tokens, _ = rows_of(4, 100, "f32", 5)
    z[0, tokens[0].long()] = -INF
    z[3, tokens[3].long()] = -INF
    offsets = _offsets([1, 1, 1, 1])  # pairs (0, 2) and (1, 3)
    loss, seq, logp, lse, grad, _ = _check(z, tokens, offsets)
    assert loss[0] == INF and loss[1] == 0 and seq[0] == -INF and seq[3] == -INF
    assert torch.isfinite(grad).all() and grad[0].any() and not grad[[1, 3]].any()
    assert df2.preference_loss(z, tokens, offsets, label_smoothing=0.1)[0][1] == INF
    loss = df2.preference_loss(z, tokens, offsets, label_smoothing=1.0)[0]
    assert loss[0] == 0 and loss[1] == INF


@pytest.mark.parametrize("shift", [300.0, -1e4, 1e6])
def test_logits_far_from_zero(shift):
    z, tokens, g = rows_of(6, 5000, "bf16" if shift == 300.0 else "f32", 7, std=2.0)
    z.copy_(((z.float() + shift) / 2).round() * 2)
    offsets = _offsets([2, 1, 1, 2])
    _check(z, tokens, offsets, _ref(z, tokens, offsets, False, g), beta=0.3)
    z[2] = torch.finfo(torch.bfloat16).min
    _check(z, tokens, offsets, _ref(z, tokens, offsets, False, g), beta=0.3)


@pytest.mark.parametrize("V,dtype", [(4099, "f32"), (151936, "bf16")])
def test_in_place(V, dtype):
    z, tokens, g = rows_of(9, V, dtype, 8, pad=5, offset=3)
    tokens[4] = -1
    offsets = _offsets([2, 2, 1, 3])
    loss, seq, logp, lse, grad = df2.preference_loss(z, tokens, offsets, grad=True)
    for alone in (False, True):
        y = place(z.float(), dtype, pad=5, offset=3)
        if alone:
            df2.preference_loss_backward(torch.ones(2, device="cuda"), y, tokens, offsets, seq, lse,
                                         grad=y)
        else:
            df2.preference_loss(y, tokens, offsets, grad=y)
        assert torch.equal(y, grad)
        now = y._base
        assert torch.isnan(now[:3]).all() and torch.isnan(now[3 + 9 * (V + 5):]).all()
        assert torch.isnan(now[3:3 + 9 * (V + 5)].view(9, V + 5)[:, V:]).all()


def test_the_same_pair_gives_the_same_sums():
    """A sequence's sum depends on its rows alone, and comes out the same every time."""
    z, tokens, g = rows_of(40, 2000, "bf16", 10)
    a = df2.preference_loss(z, tokens, _offsets([10, 10, 10, 10]), grad=True)
    b = df2.preference_loss(z, tokens, _offsets([10, 10, 10, 10]), grad=True)
    assert all(equal_bits(x, y) for x, y in zip(a, b))
    c = df2.preference_loss(z, tokens, _offsets([10, 20, 0, 10]))
    assert a[1][0] == c[1][0] and a[1][3] == c[1][3]


def test_another_stream_and_a_captured_graph():
    z, tokens, g = rows_of(20, 9001, "bf16", 11)
    offsets = _offsets([5, 4, 6, 5])
    want = df2.preference_loss(z, tokens, offsets, grad=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = df2.preference_loss(z, tokens, offsets, grad=True)
    torch.cuda.current_stream().wait_stream(side)
    assert all(equal_bits(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    y, t, at = z.clone(), tokens.clone(), offsets.clone()
    up = torch.ones(2, device="cuda")
    with torch.cuda.graph(graph):
        out = df2.preference_loss(y, t, at, grad=True)
        back = df2.preference_loss_backward(up, y, t, at, out[1], out[3])
    for k in range(3):
        y.copy_(z.roll(k, 0))
        t.copy_(tokens.roll(k, 0))
        at.copy_(_offsets([5 - k, 4 + k, 6, 5]))
        graph.replay()
        want = df2.preference_loss(y, t, at, grad=True)
        assert all(equal_bits(a, b) for a, b in zip(want, out))
        assert equal_bits(back, want[4])


def test_leading_dimensions_given_outputs_and_autograd():
    z, tokens, g = rows_of(12, 600, "f32", 12)
    offsets = _offsets([3, 3, 3, 3])
    want = df2.preference_loss(z, tokens, offsets, grad=True)
    out = dict(loss=torch.full((2,), NAN, device="cuda"),
               seq_logp=torch.full((4,), NAN, device="cuda"),
               logp=torch.full((3, 4), NAN, device="cuda"),
               lse=torch.full((3, 4), NAN, device="cuda"))
    grad = torch.full((3, 4, 600), NAN, device="cuda")
    version = grad._version
    got = df2.preference_loss(z.view(3, 4, 600), tokens.view(3, 4), offsets, grad=grad, **out)
    assert got[4] is grad and all(a is b for a, b in zip(got, out.values()))
    assert grad._version == version + 1
    assert all(equal_bits(a, b.view(a.shape)) for a, b in zip(got, want))


def test_refusals():
    z, tokens, _ = rows_of(4, 50, "f32", 13)
    offsets, f = _offsets([2, 2]), torch.zeros(4, device="cuda")
    for bad in [(z, tokens, offsets[:2]), (z, tokens, offsets.long()), (z, tokens, offsets.cpu()),
                (z, tokens.long(), offsets), (z.half(), tokens, offsets),
                (z, tokens, offsets.view(1, 3))]:
        with pytest.raises((TypeError, ValueError)):
            df2.preference_loss(*bad)
    for kw in [dict(ref_logp=f), dict(weight=f), dict(grad=z[:2]), dict(loss=f)]:
        with pytest.raises((TypeError, ValueError)):
            df2.preference_loss(z, tokens, offsets, **kw)
    for kw in [dict(beta=INF), dict(margin=NAN), dict(label_smoothing=-0.1),
               dict(label_smoothing=1.5), dict(loss=f[:1], seq_logp=f[:2]), dict(logp=f, lse=f)]:
        with pytest.raises(df2.Dflash2Error):
            df2.preference_loss(z, tokens, offsets, **kw)
    none = torch.empty((0, 50), device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    loss, seq, *_ = df2.preference_loss(none, t, _offsets([0, 0]), margin=1.0)
    assert abs(loss.item() - torch.nn.functional.softplus(torch.tensor(1.0)).item()) < 1e-6
    assert not seq.any()
    loss, *_ , grad = df2.preference_loss(z, tokens, _offsets([]), grad=True)
    assert loss.shape == (0,) and not grad.any()
