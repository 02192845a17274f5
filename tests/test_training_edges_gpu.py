"""The operators of training at calls that their documentation allows and that are easily missed:
rows and pairs without weight beside an upstream gradient that is not finite, steps that are left
out, given outputs and autograd, lists that do not match, the bits of weights that are rounded by
chance, and the loops of the example that tunes a head."""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from dflash2_draft_head_gb300 import tune_draft
from dflash2_draft_head_gb300.train_draft import AdamW
from loss_rows import INF, NAN, by_numbers, equal_bits, logp64, rows_of
from test_adamw_gpu import HYPER, Case, _chance, _expect, _one

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()
    assert df2.take_device_faults() == 0


# ------------------------------------------------------------------ no weight, no gradient


@pytest.mark.parametrize("odd", [NAN, INF, -INF])
@pytest.mark.parametrize("V,dtype", [(1000, "f32"), (151936, "bf16")])
def test_a_policy_row_without_weight_or_upstream_gradient(V, dtype, odd):
    """Either factor 0 makes the gradient 0 and leaves the row unread, whatever the other one is;
    other rows do not notice."""
    z, tokens, _ = rows_of(6, V, dtype, 21, pad=1)
    old = logp64(z, tokens, 1.0)[0].float() - 0.05
    A, ref = by_numbers([1.0, -1.0, 0.5, 2.0, 1.0, -0.5], [-1.0] * 6)
    kw = dict(ref_logp=ref, kl_coef=0.1)
    _, logp, lse, _ = df2.policy_loss(z, tokens, old, A, **kw)
    w, up = by_numbers([1.0, 0.0, 2.0, -0.0, odd, 0.5], [1.0, odd, 0.5, odd, 0.0, 2.0])
    silent = [1, 3, 4]
    plain_w, plain_up = w.clone(), up.clone()
    plain_w[silent] = plain_up[silent] = 0.0
    want = df2.policy_loss_backward(plain_up, z, tokens, old, A, logp, lse, weight=plain_w, **kw)
    z[silent] = NAN
    grad = df2.policy_loss_backward(up, z, tokens, old, A, logp, lse, weight=w, **kw)
    assert not grad[silent].any() and want[[0, 2, 5]].any(1).all()
    assert equal_bits(grad, want)


@pytest.mark.parametrize("odd", [NAN, INF, -INF])
@pytest.mark.parametrize("average", [False, True])
def test_a_pair_without_weight_or_upstream_gradient(average, odd):
    for V, dtype in ((1000, "f32"), (151936, "bf16")):
        z, tokens, _ = rows_of(9, V, dtype, 22, pad=1)
        offsets = torch.tensor([0, 1, 3, 5, 6, 8, 9], dtype=torch.int32, device="cuda")
        _, seq, _, lse, _ = df2.preference_loss(z, tokens, offsets, average=average)
        w, up = by_numbers([0.0, 2.0, odd], [odd, 0.5, 0.0])
        plain_w, plain_up = by_numbers([0.0, 2.0, 0.0], [0.0, 0.5, 0.0])
        kw = dict(average=average)
        want = df2.preference_loss_backward(plain_up, z, tokens, offsets, seq, lse, weight=plain_w,
                                            **kw)
        grad = df2.preference_loss_backward(up, z, tokens, offsets, seq, lse, weight=w, **kw)
        assert not grad[[0, 3, 4, 5, 8]].any() and grad[[1, 2, 6, 7]].any(1).all()
        assert equal_bits(grad, want)


# ------------------------------------------------------------------ steps that are left out


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_that_is_left_out_does_not_count(bits):
    """Bad gradients at the first step and at a later one: as if they had not been."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    start = torch.randn(5000, device="cuda", generator=g)
    grads = [torch.randn(5000, device="cuda", generator=g) for _ in range(4)]
    bad = grads[0].clone()
    bad[17] = NAN
    with_bad, plain = (AdamW([start.clone()], 1e-2, bits, seed=5) for _ in range(2))
    for k, x in enumerate(grads):
        if k in (0, 2):
            assert torch.isnan(with_bad.step([bad]))
        a, b = with_bad.step([x]), plain.step([x])
        assert equal_bits(a, b) and equal_bits(with_bad.params[0], plain.params[0])
        assert torch.equal(with_bad.exp_avg[0], plain.exp_avg[0])
        assert torch.equal(with_bad.exp_avg_sq[0], plain.exp_avg_sq[0])


@pytest.mark.parametrize("setting", [dict(step=0), dict(step=-3), dict(lr=NAN), dict(lr=INF),
                                     dict(lr=-INF)])
def test_a_setting_on_the_device_that_a_host_call_refuses_leaves_everything_as_it_was(setting):
    for small in (False, True):
        case = Case([3000, 17], "bf16", "bf16", small=small, master=True, offset=1)
        before = case.copy()
        args, more = case.args()
        kind = dict(step=torch.int32, lr=torch.float32)
        kw = HYPER | dict(step=1) | {k: torch.tensor([v], dtype=kind[k], device="cuda")
                                     for k, v in setting.items()}
        df2.adamw(*args, seed=3, **kw, **more)
        for name, ts in case.lists.items():
            for t, old in zip(ts, before[name]):
                assert torch.equal(torch.nan_to_num(t._base.float()), torch.nan_to_num(old.float()))


def test_clipping_where_the_scaled_norm_leaves_fp32():
    """norm * |grad_scale| above 3.4e38, the norm itself below: the gradient is clipped, not lost.
    The factor max_norm / norm is a normal number; norm, factor, g' and m are rounded once each and
    the norm's sum to 2^-21: 2^-19 is a bound on m's error."""
    n = 40
    x = torch.full((n,), 2.0 ** 120, device="cuda")
    norm = df2.grad_norm([x])
    assert torch.isfinite(norm) and norm.item() * 2.0 ** 10 > 3.5e38
    p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    df2.adamw([p], [x], [m], [v], step=1, lr=1e-2, norm=norm, max_norm=1.0, grad_scale=2.0 ** 10)
    want = 0.1 / n ** 0.5
    assert (m.double() - want).abs().max().item() <= 2.0 ** -19 * want
    # the first step of Adam moves by lr against the gradient; eps is 1e-8 of 0.16 beside it
    assert (p.double() + 1e-2).abs().max().item() <= 1e-2 * 2.0 ** -17


# ------------------------------------------------------------------ given outputs


def _small_rows():
    z, tokens, _ = rows_of(4, 100, "f32", 23)
    return z.contiguous().clone(), tokens, torch.full((4,), -3.0, device="cuda")


def _writers():
    """(name, outputs, call that writes them) of every entry point that takes outputs."""
    z, tokens, f = _small_rows()
    A = torch.ones(4, device="cuda")
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    up = torch.ones(1, device="cuda")

    def new(*s, dtype=torch.float32):
        return torch.full(s, 3, dtype=dtype, device="cuda")

    _, logp, lse, _ = df2.policy_loss(z, tokens, f, A)
    _, seq, _, plse, _ = df2.preference_loss(z, tokens, offsets)
    codes, scale = df2.state_encode(torch.ones(70, device="cuda"))
    return [
        ("policy", dict(loss=new(4), logp=new(4), lse=new(4), grad=new(4, 100)),
         lambda o: df2.policy_loss(z, tokens, f, A, **o)),
        ("policy_back", dict(grad=new(4, 100)),
         lambda o: df2.policy_loss_backward(A, z, tokens, f, A, logp, lse, **o)),
        ("preference", dict(loss=new(1), seq_logp=new(2), logp=new(4), lse=new(4), grad=new(4, 100)),
         lambda o: df2.preference_loss(z, tokens, offsets, **o)),
        ("preference_back", dict(grad=new(4, 100)),
         lambda o: df2.preference_loss_backward(up, z, tokens, offsets, seq, plse, **o)),
        ("norm", dict(out=new(1)), lambda o: df2.grad_norm([z], **o)),
        ("decode", dict(out=new(70)), lambda o: df2.state_decode(codes, scale, **o)),
        ("encode", dict(codes=new(70, dtype=torch.uint8), scale=new(3, dtype=torch.uint8)),
         lambda o: df2.state_encode(torch.ones(70, device="cuda"), **o)),
    ]


WRITERS = ["policy", "policy_back", "preference", "preference_back", "norm", "decode", "encode"]


@pytest.mark.parametrize("k", range(len(WRITERS)), ids=WRITERS)
def test_what_is_written_raises_its_version(k):
    name, outs, call = _writers()[k]
    assert name == WRITERS[k]
    before = {n: t._version for n, t in outs.items()}
    call(outs)
    for n, t in outs.items():
        assert t._version == before[n] + 1, n
    for n, t in outs.items():
        if not t.is_floating_point():
            continue
        x = torch.ones_like(t).requires_grad_()
        later = (x * t).sum()                   # saves t
        call(outs)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            later.backward()


@pytest.mark.parametrize("k", range(len(WRITERS)), ids=WRITERS)
def test_outputs_made_in_inference_mode(k):
    """They have no version, and autograd does not save them: taken, in that mode and outside."""
    _, outs, call = _writers()[k]
    with torch.inference_mode():
        inside, outside = ({n: t.clone() for n, t in outs.items()} for _ in range(2))
        call(inside)
    call(outside)
    call(outs)
    for n, t in outs.items():
        assert torch.equal(inside[n], t) and torch.equal(outside[n], t), n


# ------------------------------------------------------------------ lists


def test_scales_that_are_in_the_wrong_list():
    """As many scales as there have to be, but one of exp_avg_sq's among exp_avg's."""
    def small(n):
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def lists():
        return [[torch.zeros(40, device="cuda") for _ in range(2)] for _ in range(2)] + \
            [[small(40) for _ in range(2)] for _ in range(2)]

    for a, b in ((3, 1), (1, 3), (4, 0)):
        with pytest.raises(ValueError, match="must have 2 tensors"):
            df2.adamw(*lists(), step=1, lr=1e-3, exp_avg_scale=[small(2) for _ in range(a)],
                      exp_avg_sq_scale=[small(2) for _ in range(b)])
    df2.adamw(*lists(), step=1, lr=1e-3, exp_avg_scale=[small(2) for _ in range(2)],
              exp_avg_sq_scale=[small(2) for _ in range(2)])


@pytest.mark.parametrize("name,dtype", [("master", torch.float32), ("exp_avg_scale", torch.uint8),
                                        ("exp_avg_sq_scale", torch.uint8)])
def test_no_parameters_beside_other_lists(name, dtype):
    with pytest.raises(ValueError):
        df2.adamw([], [], [], [], step=1, lr=1e-3,
                  **{name: [torch.zeros(2, dtype=dtype, device="cuda")]})


def test_a_limit_of_the_norm_that_fp32_does_not_hold():
    """It would count as 0, which is no limit."""
    one = torch.ones(1, device="cuda")
    with pytest.raises(df2.Dflash2Error, match="max_norm"):
        df2.adamw(**_one(norm=one, max_norm=1e-60))
    df2.adamw(**_one(norm=one, max_norm=1e-40))


# ------------------------------------------------------------------ weights rounded by chance


def _by_chance(w, bits):
    """fp32's upper half after 16 bits of chance are added, from a value in 64 bits: towards 0 in
    steps of bf16."""
    ulp = 2.0 ** (np.frexp(np.where(w == 0, 1.0, np.abs(w)))[1] - 8.0)
    return np.sign(w) * np.floor(np.abs(w) / ulp + bits / 65536.0) * ulp


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1])
def test_weights_rounded_by_chance_bit_by_bit(small, g, offset):
    """bf16 weights are where the element's own bits put them.  Where the bound of the step's error
    in fp32 reaches over the place at which they decide, the neighbour is right too: twice the bound
    over a bf16 step of them, 2^-13 where the weight's own rounding makes up the bound."""
    for sizes in ([1, 33, 4097, 20011], [7] * 390):       # the second goes in two launches
        for step, seed in ((1, 5), (1000, 2 ** 40 + 12345)):
            case = Case(sizes, "bf16", g, small, offset=offset, seed=step)
            args, more = case.args()
            values = case.values()
            df2.adamw(*args, step=step, seed=seed, **HYPER, **more)
            clear, total = 0, 0
            for k, (_, _, (w, wb), _, _) in enumerate(_expect(values, step, 1.0, **HYPER)):
                bits = _chance(sizes[k], seed, step, k)[2].astype(np.float64)
                inner = np.where(np.abs(w) > wb, w - np.sign(w) * wb, 0.0)
                a, b = _by_chance(inner, bits), _by_chance(w + np.sign(w) * wb, bits)
                got = case.lists["params"][k].double().cpu().numpy()
                assert ((got >= np.minimum(a, b)) & (got <= np.maximum(a, b))).all(), (k, step)
                clear, total = clear + (a == b).sum(), total + len(a)
            assert clear >= 0.98 * total


# ------------------------------------------------------------------ the loops of the example


@pytest.mark.parametrize("method", ["policy", "preference"])
def test_the_tuning_loop_follows_its_formula(method, monkeypatch):
    """What the loop hands on: old and reference log-probabilities of the drawn tokens, a higher
    worth for tokens that are the target's, chosen drafts that hit more, the formula's gradient by
    the weight, and a step against it."""
    seen = dict(states=[], sampled=[], steps=[])
    real = {n: getattr(tune_draft.df2, n) for n in ("sample", "policy_loss", "preference_loss")}
    randn = torch.randn

    def states(*a, **k):
        t = randn(*a, **k)
        seen["states"].append(t)
        return t

    def sample(z, *a, **k):
        out = real["sample"](z, *a, **k)
        seen["sampled"].append(out[0].clone())
        return out

    def loss(name):
        def call(z, *a, **k):
            if k.get("grad") is not None:
                seen["loss"] = (z.clone(), a, {n: t for n, t in k.items() if n != "grad"})
            return real[name](z, *a, **k)
        return call

    class Recorded(AdamW):
        def step(self, grads):
            before = self.params[0].clone()
            out = super().step(grads)
            seen["steps"].append((grads[0], before, self.params[0].clone()))
            return out

    monkeypatch.setattr(torch, "randn", states)
    monkeypatch.setattr(tune_draft.df2, "sample", sample)
    for name in ("policy_loss", "preference_loss"):
        monkeypatch.setattr(tune_draft.df2, name, loss(name))
    monkeypatch.setattr(tune_draft, "AdamW", Recorded)
    n = 16
    tune_draft.tune(steps=1, blocks=8, n=n, V=512, method=method)
    # accepted() samples once before and once after the step
    want, drawn = seen["sampled"][1], seen["sampled"][2:-1]
    h = seen["states"][-1].double()
    z, args, kw = seen["loss"]
    slope, before, after = seen["steps"][0]
    x = z.double().requires_grad_()
    tokens = args[0].long()
    logp = torch.log_softmax(x, 1).gather(1, tokens[:, None]).squeeze(1)
    if method == "policy":
        old, A = args[1], args[2]
        assert torch.equal(args[0], drawn[0])
        hit = args[0] == want
        assert hit.any() and not hit.all() and (A[hit] > 0).all() and (A[~hit] < 0).all()
        assert (old.double() - logp.detach()).abs().max() <= 1e-4
        # the reference is the head itself at the first step
        assert (kw["ref_logp"].double() - logp.detach()).abs().max() <= 1e-4
        rho, d = torch.exp(logp - old.double()), kw["ref_logp"].double() - logp
        each = kw["kl_coef"] * (torch.exp(d) - d - 1) - torch.minimum(rho * A, rho.clamp(0.8, 1.2) * A)
        (each * kw["weight"]).sum().backward()
    else:
        h = h.repeat(2, 1)
        pairs = (args[1].numel() - 1) // 2
        assert args[1].tolist() == list(range(0, 2 * pairs * n + 1, n))
        target = want.view(pairs, n)
        chosen, rejected = args[0].view(2, pairs, n)
        better, worse = ((t == target).sum(1) for t in (chosen, rejected))
        assert (better >= worse).all() and (better > worse).any()
        assert torch.equal(kw["weight"] > 0, better > worse)
        S = logp.view(2 * pairs, n).sum(1)
        assert (kw["ref_logp"].double() - S.detach()).abs().max() <= n * 1e-4
        r = S - kw["ref_logp"].double()
        m = kw["beta"] * (r[:pairs] - r[pairs:])
        (kw["weight"].double() * torch.nn.functional.softplus(-m)).sum().backward()
    # the logits' gradient is rounded to bf16 (2^-8 of the value), its shares are good to 1e-5, and
    # so is the product with the states to 2^-23 * rows of the sum of its terms' magnitudes
    size = x.grad.abs().t() @ h.abs()
    bound = size * (2.0 ** -8 + 2.0 ** -23 * h.shape[0]) + 1e-4 * x.grad.abs().amax() * h.abs().sum(0)
    assert ((slope.double() - x.grad.t() @ h).abs() <= bound).all()
    assert slope.any() and ((after - before).double() * slope.double()).sum() < 0
    moved = after != before
    assert (((after - before).sign() == -slope.sign()) | (slope.abs() < 1e-6) | ~moved).all()
