"""Sampling by temperature, top-k, top-p and min-p against plain implementations.

Two comparisons.  (1) The rule in whole numbers, written with numpy integers from
the weights W = round(2^40 * 2^((x - max) * (log2(e) / T))), whose fp32 power of two is
torch's: tokens must be equal, probabilities equal to fp32 rounding.  (2) The rule
in 64 bits with exp((x - max) / T): the token must be kept, and u must lie in its
interval of the running sum, up to TOL.

TOL: the fp32 depth d = (x - max) * c has three roundings, so at most 3 * 2^-24 * |d|
with |d| <= 41; times ln 2 that is 5.1e-6 in w, and 2^x is good to 2^-22, so a weight is
off by less than 5.4e-6 of itself, a share by less than twice that, and each of the V
weights by 2^-41 more from rounding to a whole number (V <= 2^21: 1e-6 in all).
"""
import math

import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2

pytestmark = pytest.mark.gpu

TOL = 1.2e-5
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()
    assert df2.take_device_faults() == 0


def _rows(rows, V, dtype, seed, std=2.0, peak=12.0, pad=0, offset=0):
    """[rows, V] logits on the GPU (some entries stand out), rows V + pad apart, from
    element `offset` of their buffer."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, V), generator=g) * std
    at = torch.randint(0, V, (rows, min(V, 9)), generator=g)
    x.scatter_(1, at, peak * torch.rand((rows, min(V, 9)), generator=g))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return _place(x, dt, pad, offset)


def _place(x, dt, pad=0, offset=0):
    rows, V = x.shape
    buf = torch.full((rows * (V + pad) + offset + 64,), NAN, dtype=dt, device="cuda")
    v = buf[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, :V]
    v.copy_(x.to(dt))
    return v


def _one_of(v, r):
    return v[r].item() if isinstance(v, torch.Tensor) else v


def _weights(x32, T):
    """W of one row (int64 numpy), by torch's fp32 power of two on the GPU."""
    m = torch.where(torch.isnan(x32), -INF, x32).max()
    c = torch.tensor(1.4426950408889634, dtype=torch.float32, device=x32.device) / \
        torch.tensor(T if T > 0 else 1.0, dtype=torch.float32, device=x32.device)
    w = torch.exp2(torch.where(x32 == m, torch.zeros_like(x32), (x32 - m) * c))
    w = torch.where(x32 > -INF, w, torch.zeros_like(w))
    return w.cpu().numpy(), torch.round(w * 2.0 ** 40).long().cpu().numpy()


def _order(x):
    """Indices by falling value, ties by index; NaN last (numpy, fp64 values)."""
    v = np.where(np.isnan(x), -np.inf, x) + 0.0
    return np.lexsort((np.arange(len(v)), -v))


def _rule(x32, u, T, k, p, mp):
    x = x32.double().cpu().numpy()
    live = np.where(np.isnan(x), -np.inf, x)
    if not (live > -np.inf).any():
        return -1, 0.0
    w, W = _weights(x32, T)
    V = len(x)
    if not T > 0:
        k = 1
    if k <= 0 or k > V:
        k = V
    order = _order(x)
    sW, sw = W[order].copy(), w[order]
    sW[k:] = 0
    before = np.cumsum(sW) - sW
    keep = np.arange(V) < k
    if p < 1:
        keep &= before.astype(np.float64) < float(np.float32(p)) * float(sW.sum())
    if mp > 0:
        keep &= sw >= np.float32(mp)
    keep[0] = True
    kept = np.zeros(V, np.int64)
    kept[order[keep]] = W[order[keep]]
    cum = np.cumsum(kept)
    t = min(int(float(np.float32(u)) * float(cum[-1])), int(cum[-1]) - 1)
    tok = int(np.searchsorted(cum, t, side="right"))
    return tok, float(kept[tok]) / float(cum[-1])


def _in_64_bits(x32, u, T, k, p, mp, token, prob):
    """Whether the token stands by the rule in 64 bits; None where a cut is too near."""
    x = x32.double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, x)
    V = len(x)
    order = _order(x)
    if not T > 0 or k == 1:
        return token == order[0] and abs(prob - 1) < TOL
    w = np.exp((x - x.max()) / T)[order]
    n = V if k <= 0 or k > V else k
    w[n:] = 0
    cum = np.cumsum(w)
    keep = np.arange(V) < n
    if p < 1:
        before = (cum - w) / cum[-1]
        if np.abs(before - p)[:n].min() < TOL:
            return None
        keep &= before < p
    if mp > 0:
        if np.abs(w / mp - 1)[:n].min() < TOL:
            return None
        keep &= w >= mp
    keep[0] = True
    share = np.zeros(V)
    share[order[keep]] = w[keep]
    share /= share.sum()
    hi = np.cumsum(share)
    return share[token] > 0 and hi[token] - share[token] - TOL <= u <= hi[token] + TOL and \
        abs(prob - share[token]) <= 2 * TOL * share[token] + 1e-12


def _check(x, u, T=1.0, k=0, p=1.0, mp=0.0, near_ok=True):
    tok, prob = df2.sample(x, u, temperature=T, top_k=k, top_p=p, min_p=mp)
    assert tok.shape == prob.shape == x.shape[:-1]
    flat = x.reshape(-1, x.shape[-1]).float()
    tok, prob = tok.reshape(-1).cpu().numpy(), prob.reshape(-1).cpu().numpy()
    sure = 0
    for r in range(flat.shape[0]):
        s = [_one_of(v.reshape(-1) if isinstance(v, torch.Tensor) else v, r) for v in (T, k, p, mp)]
        ur = u.reshape(-1)[r].item()
        rt, rp = _rule(flat[r], ur, *s)
        assert tok[r] == rt, (r, s, ur, tok[r], rt)
        assert abs(prob[r] - rp) <= 2.0 ** -23 * rp, (r, s, prob[r], rp)
        if rt >= 0 and not (flat[r] == INF).any():
            ok = _in_64_bits(flat[r], ur, *s, tok[r], prob[r])
            assert ok is None or ok, (r, s, ur, tok[r], prob[r])
            sure += ok is not None
    return tok, prob


def _u(n, seed=0):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed + 17)).cuda()


SETTINGS = [dict(), dict(T=0.0), dict(T=0.7), dict(T=3.0), dict(k=1), dict(k=2), dict(k=20),
            dict(p=0.95), dict(p=0.5, T=1.5), dict(p=0.999, T=4.0), dict(mp=0.05),
            dict(mp=0.3, T=2.0), dict(k=20, p=0.95), dict(k=50, p=0.3, mp=0.01),
            dict(k=500, p=0.9, T=5.0), dict(k=3, mp=0.9)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 257, 1000, 4099, 20011])
def test_every_setting(V, dtype):
    for i, s in enumerate(SETTINGS):
        x = _rows(3, V, dtype, V + i, pad=i % 4, offset=i % 3)
        _check(x, _u(3, i), **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("s", SETTINGS[::3] + [dict(k=128), dict(k=3000), dict(p=0.9, T=1.0)])
def test_vocabulary_rows(dtype, s):
    x = _rows(4, 151936, dtype, 5)
    x[0] = torch.randn(151936, generator=torch.Generator().manual_seed(3)).to(x.dtype).cuda()  # flat
    x[1].mul_(4)
    _check(x, _u(4), **s)


@pytest.mark.parametrize("V,dtype", [(1 << 21, "bf16"), (600_001, "f32")])
def test_rows_too_wide_for_shared_memory(V, dtype):
    x = _rows(2, V, dtype, 8, pad=1)
    for s in (dict(), dict(k=20, p=0.9), dict(p=0.6, T=2.0), dict(T=0.0), dict(mp=0.1)):
        _check(x, _u(2), **s)


def test_settings_of_every_row():
    rows, V = 41, 5003
    x = _rows(rows, V, "bf16", 2, pad=3)
    g = torch.Generator().manual_seed(4)

    def pick(vals, dt):
        return torch.tensor(vals, dtype=dt)[torch.randint(0, len(vals), (rows,), generator=g)].cuda()

    _check(x, _u(rows), T=pick([0.0, 0.5, 1.0, 2.0, -1.0, NAN], torch.float32),
           k=pick([-3, 0, 1, 5, 60, 1000, 10000], torch.int32),
           p=pick([-1.0, 0.0, 0.2, 0.9, 1.0, 2.0], torch.float32),
           mp=pick([-1.0, 0.0, 0.02, 0.5, 2.0], torch.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_are_kept_by_index(dtype):
    V = 3001
    rows = [np.zeros(V), np.where(np.arange(V) % 3 == 0, 1.0, 0.0), np.round(np.sin(np.arange(V)) * 2),
            np.where(np.arange(V) % 2 == 0, 0.0, -0.0), -np.ones(V) * 7]
    x = _place(torch.tensor(np.stack(rows)), torch.bfloat16 if dtype == "bf16" else torch.float32)
    u = torch.tensor([0.0, 0.3, 0.6, 0.999, 0.5]).cuda()
    for s in (dict(), dict(k=1), dict(k=17), dict(k=1500), dict(p=0.5), dict(k=1200, p=0.31),
              dict(T=0.0), dict(mp=0.5), dict(k=1100, p=0.9, T=0.2)):
        _check(x, u, **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("levels,copies,span", [(60, 700, 8.0), (200, 220, 3.0), (24, 1500, 6.0)])
def test_cuts_among_levels(levels, copies, span, dtype):
    """Few values, each many times: within the bins of a cut by weight the values are not
    spread evenly, so that what the bins' middles tell of the cut is often wrong."""
    rows, V = 24, levels * copies
    g = torch.Generator().manual_seed(levels)
    lev = torch.rand((rows, levels), generator=g) * -span
    at = torch.stack([torch.randperm(V, generator=g) for _ in range(rows)])
    x = torch.empty((rows, V)).scatter_(1, at, lev.repeat_interleave(copies, dim=1))
    x = _place(x, torch.bfloat16 if dtype == "bf16" else torch.float32)
    for i, p in enumerate((0.3, 0.7, 0.95)):
        _check(x, _u(rows, 40 + i), p=p)
        _check(x, _u(rows, 50 + i), p=p, k=V // 3, mp=0.01)


def test_values_that_crowd_round_zero():
    """fp32 values of every exponent: the bin with the cut spans most of the keys."""
    V = 9001
    g = np.random.default_rng(0)
    x = np.sign(g.standard_normal(V)) * 10.0 ** g.uniform(-37, 0, V)
    x[::50] = 0.0
    rows = np.stack([x, x * 1e-30, np.abs(x) * 1e-38 * 1e-6, -np.abs(x)])
    t = _place(torch.tensor(rows, dtype=torch.float32), torch.float32, pad=1)
    for s in (dict(k=1), dict(k=5), dict(k=4000), dict(p=0.4), dict(k=4500, p=0.7), dict(p=0.99)):
        _check(t, _u(4), **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_and_non_finite_entries(dtype):
    V = 2050
    g = torch.Generator().manual_seed(6)
    x = torch.randn((8, V), generator=g) * 3
    low = torch.finfo(torch.bfloat16).min
    x[0] = -INF                                   # nothing left
    x[1] = -INF
    x[1, 77] = -3.0                               # one left
    x[2, ::2] = NAN
    x[3] = NAN                                    # only NaN
    x[4, 5] = x[4, 900] = INF
    x[5] = low                                    # masked by the type's lowest value, all of it
    x[6] = low
    x[6, 13] = 1.0
    x[7, :] = -INF
    x[7, -1] = x[7, 0] = 2.0                      # the two ends
    t = _place(x, torch.bfloat16 if dtype == "bf16" else torch.float32, pad=1)
    for s in (dict(), dict(T=0.0), dict(k=3), dict(p=0.9), dict(mp=0.2), dict(k=100, p=0.5, T=2.0)):
        tok, prob = _check(t, _u(8, 3), **s)
        assert tok[0] == -1 and tok[3] == -1 and prob[0] == 0 and prob[3] == 0
        assert tok[1] == 77 and prob[1] == 1 and tok[6] == 13 and tok[4] in (5, 900)


def test_what_lies_between_the_rows_is_not_read():
    x = _rows(3, 1003, "bf16", 1, pad=5, offset=1)     # the padding is NaN
    y = _rows(3, 1003, "bf16", 1)
    x.copy_(y)
    x._base[:1] = INF
    a = df2.sample(x, _u(3), top_p=0.9)
    b = df2.sample(y, _u(3), top_p=0.9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_uniform_outside_its_range():
    x = _rows(4, 300, "f32", 1)
    x[1:] = x[0]
    u = torch.tensor([-1.0, NAN, 1.0, 5.0]).cuda()
    tok, _ = df2.sample(x, u, top_k=30)
    kept = torch.topk(x[0], 30)[1].sort()[0]
    assert tok.tolist() == [kept[0], kept[0], kept[-1], kept[-1]]


def test_a_row_gives_the_same_token_in_any_batch():
    """How a row is split depends on the number of rows; its token does not."""
    V = 151936
    x = _rows(1, V, "bf16", 11, peak=4.0)
    for s in (dict(), dict(top_p=0.9), dict(top_k=40, top_p=0.8)):
        u = _u(64, 5)
        many = df2.sample(x.expand(64, V).contiguous(), u, **s)
        lots = df2.sample(x.expand(640, V).contiguous(), u.repeat(10), **s)
        for r in range(0, 64, 9):
            one = df2.sample(x, u[r:r + 1], **s)
            assert one[0].item() == many[0][r].item() == lots[0][r].item() == lots[0][576 + r].item()
            assert one[1].item() == many[1][r].item()


def test_frequencies_follow_the_shares():
    """8192 stratified numbers on one row: every token's count is within 2 of 8192 times its
    share (the numbers are (i + 0.5) / 8192, and a kept token's interval is contiguous)."""
    n, V = 8192, 64
    x = _rows(1, V, "f32", 21, peak=3.0)
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    tok, _ = df2.sample(x.expand(n, V).contiguous(), u, temperature=0.9, top_p=0.9)
    w = torch.softmax(x[0].double() / np.float64(np.float32(0.9)), 0)
    order = torch.argsort(w, descending=True)
    before = torch.cumsum(w[order], 0) - w[order]
    w[order[before >= 0.9]] = 0
    w /= w.sum()
    count = torch.bincount(tok.long(), minlength=V)
    assert (count - n * w).abs().max() <= 2


def test_offsets_beyond_32_bits():
    V, ld = 5000, (1 << 30) + 8                         # row 2 starts past 2^31 elements
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, V), (ld, 1))
    y = _rows(3, V, "bf16", 3)
    x.copy_(y)
    for s in (dict(), dict(top_k=9), dict(top_p=0.8)):
        a, b = df2.sample(x, _u(3), **s), df2.sample(y, _u(3), **s)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_on_another_stream_and_with_given_outputs():
    x = _rows(5, 4096, "f32", 4)
    u = _u(5)
    want = df2.sample(x, u, top_p=0.7)
    side = torch.cuda.Stream()
    y = torch.zeros_like(x)
    tok = torch.empty(5, dtype=torch.int32, device="cuda")
    prob = torch.empty(5, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        y.copy_(x)
        got = df2.sample(y, u, top_p=0.7, tokens=tok, probs=prob)
    side.synchronize()
    assert got[0] is tok and got[1] is prob
    assert torch.equal(tok, want[0]) and torch.equal(prob, want[1])


def test_leading_dimensions_and_graph_capture():
    x = _rows(12, 1500, "bf16", 6).contiguous().view(3, 4, 1500)
    u = _u(12).view(3, 4)
    _check(x, u, k=10, p=0.9)
    one = df2.sample(x[0, 0], u[0, 0])
    assert one[0].shape == ()
    want = df2.sample(x, u, top_p=0.9)
    tok, prob = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df2.sample(x, u, top_p=0.9, tokens=tok, probs=prob)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, want[0]) and torch.equal(prob, want[1])


def test_no_rows():
    tok, prob = df2.sample(torch.empty((0, 100), device="cuda"), torch.empty(0, device="cuda"))
    assert tok.shape == prob.shape == (0,)


def test_refusals():
    x, u = _rows(4, 100, "f32", 1), _u(4)
    ok = torch.zeros(4, device="cuda")
    bad = [dict(uniform=u[:3]), dict(uniform=u.double()), dict(uniform=u.cpu()),
           dict(logits=x.half()), dict(logits=x.cpu()), dict(logits=x.t()),
           dict(logits=x[:, ::2]), dict(logits=x[:1].expand(4, 100)),
           dict(temperature=ok.double()), dict(temperature=ok[:2]), dict(temperature=-1.0),
           dict(temperature=NAN), dict(top_k=ok), dict(top_p=NAN), dict(min_p=NAN),
           dict(tokens=ok), dict(probs=ok.int()), dict(probs=u),
           dict(logits=torch.empty((4, 0), device="cuda")),
           dict(logits=torch.zeros((1, (1 << 21) + 1), device="cuda"), uniform=u[:1])]
    for b in bad:
        args = {"logits": x, "uniform": u} | b
        with pytest.raises((ValueError, TypeError, df2.Dflash2Error)):
            df2.sample(**args)
