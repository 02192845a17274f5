"""AdamW over lists of tensors, with states in fp32 and in 8 bits, against the formula in 64 bits.

Bounds, from the fp32 operations of the step (g' one product, m two products and a sum, v three and
a sum, constants rounded once):
  m: 2^-22 of beta1 |m| + (1 - beta1) |g'|;  v: 2^-21 of beta2 v + (1 - beta2) g'^2
  p: its own rounding and that of the decay, 2^-23 |p|; the step's: 2^-20 of it, and m's error times
    lr / (1 - beta1^t) over the divisor (v's relative error counts half); bf16 to the nearest 2^-8 of
    the value more, by chance 2^-7
8-bit codes are compared one by one with the rounding of m and v that numpy's fp32 gives for the
same operations, which are all rounded to the nearest once each.
"""
import threading

import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from loss_rows import INF, NAN

pytestmark = pytest.mark.gpu

KIND = {"f32": torch.float32, "bf16": torch.bfloat16}
U32 = np.uint32


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()


def _tensor(n, dtype, offset, fill):
    """A tensor of n elements that starts `offset` elements into a guarded buffer."""
    buf = torch.full((n + offset + 40,), fill, dtype=dtype, device="cuda")
    return buf[offset:offset + n]


class Case:
    """Lists of tensors with their guards, in the given types."""

    def __init__(self, sizes, p="f32", g="f32", small=False, master=False, offset=0, seed=0,
                 scale=1e-2):
        rng = np.random.default_rng(seed)
        self.sizes, self.small, self.master = sizes, small, master
        self.lists = {k: [] for k in ("params", "grads", "exp_avg", "exp_avg_sq", "master",
                                      "exp_avg_scale", "exp_avg_sq_scale")}
        for k, n in enumerate(sizes):
            o = offset * (k % 3 + 1)

            def put(name, x, dtype, off=o):
                t = _tensor(len(x), dtype, off, 77 if dtype == torch.uint8 else NAN)
                t.copy_(torch.from_numpy(np.ascontiguousarray(x)).to(dtype))
                self.lists[name].append(t)
                return t

            w = rng.standard_normal(n).astype(np.float32)
            spread = 2.0 ** rng.normal(0, 3, n)
            put("grads", (rng.standard_normal(n) * scale * spread).astype(np.float32), KIND[g])
            t = put("params", w, KIND[p])
            if master:
                put("master", w, torch.float32)
            m = torch.from_numpy((rng.standard_normal(n) * scale * spread / 3).astype(np.float32))
            v = torch.from_numpy((rng.random(n) * scale * spread).astype(np.float32) ** 2)
            if small:
                for name, x, sq in (("exp_avg", m, False), ("exp_avg_sq", v, True)):
                    c, s = df2.state_encode(x.cuda(), squares=sq)
                    put(name, c.cpu().numpy(), torch.uint8)
                    put(name + "_scale", s.cpu().numpy(), torch.uint8)
            else:
                put("exp_avg", m.numpy(), torch.float32)
                put("exp_avg_sq", v.numpy(), torch.float32)
            assert t.numel() == n

    def args(self):
        g = self.lists
        kw = dict(master=g["master"]) if self.master else {}
        if self.small:
            kw |= dict(exp_avg_scale=g["exp_avg_scale"], exp_avg_sq_scale=g["exp_avg_sq_scale"])
        return (g["params"], g["grads"], g["exp_avg"], g["exp_avg_sq"]), kw

    def copy(self):
        """Host copies of all buffers, guards too."""
        return {k: [t._base.clone() for t in v] for k, v in self.lists.items()}

    def values(self):
        """(w, g, m, v) of every tensor in fp32 on the host."""
        out = []
        for k in range(len(self.sizes)):
            w = self.lists["master" if self.master else "params"][k].float().cpu().numpy()
            g = self.lists["grads"][k].float().cpu().numpy()
            if self.small:
                m, v = (df2.state_decode(self.lists[n][k], self.lists[n + "_scale"][k],
                                         squares=n.endswith("sq")).cpu().numpy()
                        for n in ("exp_avg", "exp_avg_sq"))
            else:
                m, v = (self.lists[n][k].cpu().numpy() for n in ("exp_avg", "exp_avg_sq"))
            out.append((w, g, m, v))
        return out

    def guards_hold(self, before):
        for name, ts in self.lists.items():
            for t, old in zip(ts, before[name]):
                start = t.storage_offset()
                for a, b in ((t._base[:start], old[:start]),
                             (t._base[start + t.numel():], old[start + t.numel():])):
                    assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
        for t, old in zip(self.lists["grads"], before["grads"]):
            assert torch.equal(torch.nan_to_num(t._base.float()), torch.nan_to_num(old.float()))


def _mix(x):
    x = U32(x)
    x = (x ^ x >> U32(16)) * U32(0x927aa3cd)
    x = (x ^ x >> U32(15)) * U32(0x93e1aa55)
    return x ^ x >> U32(16)


def _chance(n, seed, step, tensor):
    with np.errstate(over="ignore"):
        key = _mix(U32(seed & 0xffffffff) ^ _mix(U32(seed >> 32) ^ _mix(U32(step))))
        x = (np.arange(n, dtype=U32) ^ key) * U32(0x927aa3cd)
        x = ((x ^ x >> U32(16)) + _mix(key + U32(tensor) + U32(1))) * U32(0x93e1aa55)
        x = x ^ x >> U32(15)
        return x & U32(0xffff), x >> U32(16), (x * U32(0x927aa3cd)) >> U32(16)


def _codes(x, squares, bits):
    """Codes and scales of fp32 values: block by block, by the definition of the format."""
    n = len(x)
    codes, scales = np.zeros(n, np.uint8), np.zeros(-(-n // 32), np.uint8)
    lowest, top = (-14, 15) if squares else (-6, 7)
    for b in range(len(scales)):
        at = slice(32 * b, min(n, 32 * b + 32))
        y = np.abs(x[at].astype(np.float64))
        if not np.isfinite(y).all():
            scales[b] = 255
            continue
        e = np.frexp(y.max())[1] - 1 if y.max() >= 2.0 ** -126 else -127
        scales[b] = max(e - top + 127, 1)
        y = y * 2.0 ** (127 - int(scales[b]))
        power = np.maximum(np.frexp(np.maximum(y, 2.0 ** -40))[1] - 1, lowest)
        q = y / 2.0 ** (power - 3.0)             # 8 to 16, or below 8 at the smallest power
        # Where q is below 8 the value is first taken as a subnormal fp32 number, i.e. to the
        # nearest multiple of 2^-20 of a code's distance (from 8 on q has no bits below that): a
        # value nearer than 2^-21 to the middle of two codes is a tie there.
        q = np.round(q * 2.0 ** 20) / 2.0 ** 20
        if bits is None:
            whole = np.round(q)                  # ties to even
        else:
            whole = np.floor(q + (bits[at].astype(np.float64) * 16 + 8) / 2.0 ** 20)
        code = (whole + (power - lowest) * 8).astype(np.int64)
        if squares:
            code = np.where((x[at] > 0) & (code == 0), 1, code)
        else:
            code = code | np.where(np.signbit(x[at]), 128, 0)
        codes[at] = code
    return codes, scales


HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _expect(values, step, coef, lr, beta1, beta2, eps, weight_decay):
    """Per tensor: m, v in fp32 by the kernel's operations; w, m, v in 64 bits, and their bounds."""
    f = np.float32
    for w, g, m, v in values:
        with np.errstate(all="ignore"):
            gs = g * f(coef)
            m32 = m * f(beta1) + gs * f(1 - beta1)
            v32 = v * f(beta2) + (gs * gs) * f(1 - beta2)
            w, g, m, v = (x.astype(np.float64) for x in (w, g, m, v))
            g = g * float(f(coef))
            m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
            mb = 2.0 ** -22 * (beta1 * np.abs(m) + (1 - beta1) * np.abs(g))
            vb = 2.0 ** -21 * v1
            rate = lr / (1 - beta1 ** step)
            under = np.sqrt(v1 / (1 - beta2 ** step)) + eps
            w1 = w - lr * weight_decay * w - rate * m1 / under
            wb = 2.0 ** -23 * np.abs(w) + 2.0 ** -24 * np.abs(w1) + \
                abs(rate) * (2.0 ** -20 * np.abs(m1) + mb) / under
        yield m32, v32, (w1, wb), (m1, mb), (v1, vb)


def _within(got, ref, bound, what):
    err = np.abs(got.astype(np.float64) - ref)
    assert (err <= bound).all(), (what, float((err - bound).max()), float(err.max()))


def _check(case, step=7, coef=1.0, hyper=HYPER, seed=None, **kw):
    args, more = case.args()
    values, before = case.values(), case.copy()
    df2.adamw(*args, step=step, seed=seed, **hyper, **more, **kw)
    torch.cuda.synchronize()
    case.guards_hold(before)
    bf = case.lists["params"][0].dtype == torch.bfloat16
    for k, (m32, v32, w, m, v) in enumerate(_expect(values, step, coef, **hyper)):
        r = [None] * 3 if seed is None else _chance(case.sizes[k], seed, step, k)
        if case.small:
            for name, x, sq, bits in (("exp_avg", m32, False, r[0]), ("exp_avg_sq", v32, True, r[1])):
                codes, scales = _codes(x, sq, bits)
                np.testing.assert_array_equal(case.lists[name + "_scale"][k].cpu().numpy(), scales)
                np.testing.assert_array_equal(case.lists[name][k].cpu().numpy(), codes)
        else:
            _within(case.lists["exp_avg"][k].cpu().numpy(), *m, ("m", k))
            _within(case.lists["exp_avg_sq"][k].cpu().numpy(), *v, ("v", k))
        got = case.lists["params"][k].float().cpu().numpy()
        if case.master:
            copy = case.lists["master"][k]
            _within(copy.cpu().numpy(), *w, ("master", k))
            assert torch.equal(case.lists["params"][k], copy.bfloat16())
        else:
            rounding = 0 if not bf else 2.0 ** -8 if seed is None else 2.0 ** -7
            _within(got, w[0], w[1] + rounding * np.abs(w[0]), ("p", k))
    return case


KINDS = [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
         ("bf16", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", True)]
SIZES = [1, 31, 32, 33, 0, 4095, 4096, 4097, 8, 20011]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("p,g,master", KINDS)
def test_formula(p, g, master, small, offset):
    for seed in (None, 2 ** 40 + 12345):
        for step in (1, 1000):
            _check(Case(SIZES, p, g, small, master, offset, seed=step), step, seed=seed)


@pytest.mark.parametrize("count", [1, 16, 17, 384, 385, 800])
def test_numbers_of_tensors(count):
    """As many as fit one launch's parameters and more: the place in the list counts through."""
    rng = np.random.default_rng(count)
    sizes = [int(n) for n in rng.integers(0, 200, count)]
    _check(Case(sizes, "bf16", "bf16", small=True, seed=count), seed=99)
    _check(Case([0] * (count - 1) + [5000]))


@pytest.mark.parametrize("hyper", [dict(beta1=0.0), dict(beta2=0.0), dict(weight_decay=0.0),
                                   dict(lr=0.0), dict(eps=1.0), dict(lr=-1e-3), dict(beta2=0.9999),
                                   dict(eps=1e-12), dict(eps=1e-30)])
def test_settings(hyper):
    _check(Case([1000, 77]), hyper=HYPER | hyper)
    _check(Case([1000, 77], "bf16", "f32", small=True), hyper=HYPER | hyper, seed=1)


def test_empty_states():
    """A first step from states of zeros, also where gradients are 0: nothing but the decay."""
    for small in (False, True):
        case = Case([500, 64], small=small)
        for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            for t in case.lists[name]:
                t.zero_()
        case.lists["grads"][1].zero_()
        before = case.lists["params"][1].clone()
        _check(case, step=1)
        assert torch.allclose(case.lists["params"][1], before * (1 - 3e-4), rtol=1e-6, atol=0)


@pytest.mark.parametrize("small", [False, True])
def test_gradients_over_many_powers_of_two(small):
    """From below fp32's normal numbers to where squares nearly overflow."""
    case = Case([4096] * 4, small=small)
    for t, s in zip(case.lists["grads"], (2.0 ** -100, 2.0 ** -66, 2.0 ** 40, 2.0 ** 55)):
        t.mul_(s)
    for t in case.lists["exp_avg_scale" if small else "exp_avg"][:2]:
        t.zero_()
    for t in case.lists["exp_avg_sq_scale" if small else "exp_avg_sq"][:2]:
        t.zero_()
    args, more = case.args()
    values = case.values()
    df2.adamw(*args, step=3, seed=5 if small else None, **HYPER, **more)
    for k, (m32, v32, w, m, v) in enumerate(_expect(values, 3, 1.0, **HYPER)):
        if small:
            for name, x, sq, bits in zip(("exp_avg", "exp_avg_sq"), (m32, v32), (False, True),
                                         _chance(4096, 5, 3, k)):
                codes, scales = _codes(x, sq, bits)
                np.testing.assert_array_equal(case.lists[name + "_scale"][k].cpu().numpy(), scales)
                # below fp32's normal numbers the code's own arithmetic rounds once more
                far = np.abs(case.lists[name][k].cpu().numpy().astype(int) - codes.astype(int))
                assert far.max() <= (1 if k < 2 else 0)
        # v's rounding to multiples of 2^-149 weighs on the divisor, which eps dominates there
        _within(case.lists["params"][k].cpu().numpy(), w[0],
                w[1] + 3e-3 * 2.0 ** -74 * np.abs(m[0]) / HYPER["eps"] ** 2 * 50, ("p", k))


@pytest.mark.parametrize("norm,max_norm,scale", [(5.0, 1.0, 1.0), (0.5, 1.0, 1.0), (0.0, 1.0, 1.0),
                                                 (5.0, None, 0.25), (5.0, 1.0, 0.5), (5.0, 1.0, -2.0),
                                                 (5.0, 0.0, 1.0), (5.0, 1.0, 0.0)])
def test_clipping(norm, max_norm, scale):
    f = np.float32
    coef = f(scale)
    if max_norm and norm * abs(scale) > max_norm:
        coef = coef * (f(max_norm) / (f(norm) * f(abs(scale))))
    for small in (False, True):
        _check(Case([3000, 17], "bf16", "bf16", small=small, master=True), coef=coef,
               norm=torch.tensor([norm], device="cuda"), max_norm=max_norm, grad_scale=scale, seed=3)


@pytest.mark.parametrize("norm", [INF, NAN, -INF])
def test_a_norm_that_is_not_finite_leaves_everything_as_it_was(norm):
    for small in (False, True):
        case = Case([3000, 17], "bf16", "bf16", small=small, master=True, offset=1)
        before = case.copy()
        args, more = case.args()
        value = torch.tensor([norm], device="cuda")
        for max_norm in (None, 1.0):
            df2.adamw(*args, step=1, norm=value, max_norm=max_norm, **HYPER, **more)
        for name, ts in case.lists.items():
            for t, old in zip(ts, before[name]):
                assert torch.equal(torch.nan_to_num(t._base.float()), torch.nan_to_num(old.float()))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_bad_gradients_stay_visible(bad):
    """A NaN or an infinity without a norm: in fp32 states the element's own, in 8 bits its
    block's; everything else goes on."""
    for small in (False, True):
        case = Case([100, 100], small=small)
        case.lists["grads"][0][40] = bad
        args, more = case.args()
        values = case.values()
        df2.adamw(*args, step=2, **HYPER, **more)
        hit = np.zeros(100, bool)
        hit[40] = True
        for k, (_, _, w, m, _) in enumerate(_expect(values, 2, 1.0, **HYPER)):
            got = case.lists["params"][k].cpu().numpy()
            assert (np.isnan(got) == (hit & (k == 0))).all()
            _within(np.where(np.isnan(got), 0, got), np.where(np.isnan(got), 0, w[0]),
                    np.nan_to_num(w[1], nan=1, posinf=1), k)
        after = case.values()
        block = np.zeros(100, bool)
        block[32:64] = True
        wrong = ~np.isfinite(after[0][2])
        assert (wrong == (block if small else hit)).all()
        if small:
            assert case.lists["exp_avg_scale"][0][1] == 255 and np.isnan(after[0][2][block]).all()
            assert case.lists["exp_avg_sq_scale"][0][1] == 255 and np.isnan(after[0][3][block]).all()
        assert np.isfinite(after[1][2]).all()


def test_step_and_rate_on_the_device():
    """expm1 of step * log(beta): a relative 2^-21 in each correction, half of it under the root;
    lr * weight_decay in fp32."""
    for step in (1, 10, 100000):
        case, plain = Case([5000, 3]), Case([5000, 3])
        args, more = case.args()
        df2.adamw(*args, **(HYPER | dict(lr=torch.tensor([3e-3], device="cuda"))), **more,
                  step=torch.tensor([step], dtype=torch.int32, device="cuda"))
        args, more = plain.args()
        df2.adamw(*args, step=step, **HYPER, **more)
        for a, b, old in zip(case.lists["params"], plain.lists["params"], Case([5000, 3]).lists["params"]):
            moved = (b - old).abs()
            assert ((a - b).abs() <= 2.0 ** -20 * moved + 2.0 ** -23 * old.abs()).all()
        for name in ("exp_avg", "exp_avg_sq"):
            assert all(torch.equal(a, b) for a, b in zip(case.lists[name], plain.lists[name]))


@pytest.mark.parametrize("which", ["step", "lr"])
def test_one_setting_on_the_device(which):
    both, one = Case([5000, 3], small=True), Case([5000, 3], small=True)
    step = torch.tensor([9], dtype=torch.int32, device="cuda")
    lr = torch.tensor([3e-3], device="cuda")
    args, more = both.args()
    df2.adamw(*args, **more, **(HYPER | dict(lr=lr)), step=step, seed=6)
    args, more = one.args()
    df2.adamw(*args, **more, **(HYPER | (dict(lr=lr) if which == "lr" else {})),
              step=step if which == "step" else 9, seed=6)
    for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        assert all(torch.equal(a, b) for a, b in zip(both.lists[name], one.lists[name]))
    for a, b, old in zip(both.lists["params"], one.lists["params"], Case([5000, 3]).lists["params"]):
        assert ((a - b).abs() <= 2.0 ** -20 * (b - old).abs() + 2.0 ** -23 * old.abs()).all()


def test_a_captured_step_that_is_replayed():
    """Step number, rate, norm and chance follow the device's values from replay to replay, two
    graphs of different lists beside one another."""
    def lists():
        return Case([3000, 70], "bf16", "bf16", small=True, seed=1)

    step = torch.ones(1, dtype=torch.int32, device="cuda")
    lr = torch.full((1,), 1e-2, device="cuda")
    cases, graphs = [lists(), lists()], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        args, more = c.args()
        df2.grad_norm(args[1])
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            norm = df2.grad_norm(args[1])
            df2.adamw(*args, step=step, norm=norm, max_norm=0.1, seed=4, **(HYPER | dict(lr=lr)), **more)
        graphs.append(graph)
    want = lists()
    args, more = want.args()
    for k in range(1, 5):
        for graph in graphs:
            graph.replay()
        norm = df2.grad_norm(args[1])
        df2.adamw(*args, step=step, norm=norm, max_norm=0.1, seed=4, **(HYPER | dict(lr=lr)), **more)
        for name, ts in want.lists.items():
            for c in cases:
                assert all(torch.equal(a, b) for a, b in zip(ts, c.lists[name])), (name, k)
        step += 1
        lr *= 0.5


def test_chance_is_fair():
    """The mean over 4096 steps of one rounding each: the odds are multiples of 2^-16, the spread of
    a mean of n is at most half a code's distance over sqrt(n), and 6 of these are never passed."""
    n, times = 64, 4096
    rng = np.random.default_rng(0)
    g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    p0 = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda().bfloat16()
    total = {k: torch.zeros(n, dtype=torch.float64, device="cuda") for k in ("p", "m", "v")}
    for k in range(times):
        p = p0.clone()
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        ms, vs = (torch.zeros(2, dtype=torch.uint8, device="cuda") for _ in range(2))
        df2.adamw([p], [g], [m], [v], step=1, lr=1e-3, weight_decay=0.0, seed=k,
                  exp_avg_scale=[ms], exp_avg_sq_scale=[vs])
        total["p"] += p.double()
        total["m"] += df2.state_decode(m, ms).double()
        total["v"] += df2.state_decode(v, vs, squares=True).double()
    g = g.double()
    for name, want, part in (("m", 0.1 * g, 8), ("v", 0.001 * g * g, 8),
                             ("p", p0.double() - 1e-3 * g / (g.abs() + 1e-8), 128)):
        off = (total[name] / times - want).abs()
        step = want.abs() / part                 # a code's distance, at most
        low = want.abs().view(-1, 32).amax(1).repeat_interleave(32) * 2.0 ** -15 if part == 8 else 0
        assert (off <= (step + low) * (6 * 0.5 / times ** 0.5 + 2.0 ** -16) + 1e-6 * want.abs()).all(), name


def test_states_in_8_bits_follow():
    """3000 steps with gradients of variance 1: the mean over 32768 elements of v stays with that of
    a state in fp32 (an element's own spread is about a fifth of it: 5 of 0.21 / sqrt(32768) are
    0.6 percent)."""
    n = 32768
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    p, q = (torch.zeros(n, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, device="cuda") for _ in range(2))
    mc, vc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(n // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    for step in range(1, 3001):
        x = torch.randn(n, device="cuda", generator=g)
        df2.adamw([p], [x], [m], [v], step=step, lr=1e-3)
        df2.adamw([q], [x], [mc], [vc], step=step, lr=1e-3, exp_avg_scale=[ms],
                  exp_avg_sq_scale=[vs], seed=8)
    small = df2.state_decode(vc, vs, squares=True).double().mean().item()
    assert abs(small / v.double().mean().item() - 1) <= 0.006


def test_codes_to_values_and_back():
    """Every code decodes to its definition's value, exactly in bf16 too, and comes back."""
    code = torch.arange(256, dtype=torch.uint8, device="cuda")
    c = np.arange(256)
    for squares in (False, True):
        mag = c if squares else c & 127
        e, f = mag >> 3, (mag & 7) / 8
        low = -14.0 if squares else -6.0
        want = np.where(e > 0, (1 + f) * 2.0 ** (e + low - 1), f * 2.0 ** low)
        want = np.where((c >= 128) & (not squares), -want, want)
        for scale in (1, 60, 127, 200, 230):
            s = torch.full((8,), scale, dtype=torch.uint8, device="cuda")
            for dtype in KIND.values():
                got = df2.state_decode(code, s, squares=squares, dtype=dtype)
                expect = want * 2.0 ** (scale - 127.0)
                keep = np.abs(expect) >= 2.0 ** -126   # a subnormal bf16 has fewer bits
                np.testing.assert_array_equal(got.double().cpu().numpy()[keep], expect[keep])
            back, s2 = df2.state_encode(df2.state_decode(code, s, squares=squares), squares=squares)
            again = df2.state_decode(back, s2, squares=squares)
            np.testing.assert_array_equal(again.cpu().numpy(),
                                          df2.state_decode(code, s, squares=squares).cpu().numpy())


@pytest.mark.parametrize("n", [0, 1, 31, 33, 5000, 2 ** 20 + 7])
@pytest.mark.parametrize("squares", [False, True])
def test_encode(n, squares):
    rng = np.random.default_rng(n)
    x = (rng.standard_normal(n) * 2.0 ** rng.normal(0, 6, n)).astype(np.float32)
    x = np.abs(x) if squares else x
    for offset in (0, 1):
        for dtype in KIND.values():
            t = _tensor(n, dtype, offset, NAN)
            t.copy_(torch.from_numpy(x))
            c = _tensor(n, torch.uint8, offset, 9)
            s = _tensor(-(-n // 32), torch.uint8, offset, 9)
            df2.state_encode(t, squares=squares, codes=c, scale=s)
            if n <= 5000:
                want, scales = _codes(t.float().cpu().numpy(), squares, None)
                np.testing.assert_array_equal(c.cpu().numpy(), want)
                np.testing.assert_array_equal(s.cpu().numpy(), scales)
            for y in (c, s):
                keep = torch.ones(y._base.numel(), dtype=torch.bool, device="cuda")
                keep[offset:offset + y.numel()] = False
                assert (y._base[keep] == 9).all()
            out = _tensor(n, dtype, offset, NAN)
            df2.state_decode(c, s, squares=squares, out=out)
            top = np.abs(t.float().cpu().numpy())
            top = np.pad(top, (0, -n % 32)).reshape(-1, 32).max(1).repeat(32)[:n]
            got = out.float().cpu().numpy()
            ref = t.float().cpu().numpy()
            assert (np.abs(got - ref) <= np.abs(ref) / 16 + top * 2.0 ** -16 *
                    (1 if not squares else 2.0 ** -13)).all()


def test_encode_what_is_not_a_number():
    for bad, squares in ((NAN, False), (INF, False), (-INF, False), (NAN, True), (INF, True),
                         (-1.0, True)):
        x = torch.ones(96, device="cuda")
        x[40] = bad
        c, s = df2.state_encode(x, squares=squares)
        y = df2.state_decode(c, s, squares=squares)
        assert torch.isnan(y[32:64]).all() and (y[:32] == 1).all() and (y[64:] == 1).all()


def test_another_stream():
    case, plain = Case([100000, 3]), Case([100000, 3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        args, more = case.args()
        df2.adamw(*args, step=1, **HYPER, **more)
    torch.cuda.current_stream().wait_stream(side)
    args, more = plain.args()
    df2.adamw(*args, step=1, **HYPER, **more)
    for name in case.lists:
        assert all(torch.equal(a, b) for a, b in zip(case.lists[name], plain.lists[name]))


def test_two_threads_on_streams_of_their_own():
    """Calls do not hold Python's lock while they check and launch."""
    cases, plain = [Case([5000] * 40, seed=k) for k in range(2)], [Case([5000] * 40, seed=k) for k in range(2)]
    torch.cuda.synchronize()
    errors = []

    def work(case):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                args, more = case.args()
                for step in range(1, 31):
                    norm = df2.grad_norm(args[1])
                    df2.adamw(*args, step=step, norm=norm, max_norm=1.0, **HYPER, **more)
            stream.synchronize()
        except Exception as e:  # told by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c in plain:
        work(c)
    torch.cuda.synchronize()
    for a, b in zip(cases, plain):
        for name in a.lists:
            assert all(torch.equal(x, y) for x, y in zip(a.lists[name], b.lists[name]))


def test_parameters_of_a_module():
    """Leaves that require gradients; autograd learns that they moved."""
    lin = torch.nn.Linear(40, 30, device="cuda")
    x = torch.randn(5, 40, device="cuda")
    params = list(lin.parameters())
    lin(x).square().sum().backward()
    kept = (lin.weight * lin.weight).sum()
    state = [[torch.zeros_like(p) for p in params] for _ in range(2)]
    before = [p.detach().clone() for p in params]
    version = params[0]._version
    df2.adamw(params, [p.grad for p in params], *state, step=1, lr=0.1, weight_decay=0.0)
    assert params[0]._version > version and params[0].requires_grad
    for p, b in zip(params, before):
        # the first step of Adam moves every weight by lr, against its gradient's sign
        assert torch.allclose(p, b - 0.1 * p.grad.sign() * (p.grad != 0), atol=1e-5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()


def _one(n=40, **kw):
    t = dict(params=[torch.zeros(n, device="cuda")], grads=[torch.zeros(n, device="cuda")],
             exp_avg=[torch.zeros(n, device="cuda")], exp_avg_sq=[torch.zeros(n, device="cuda")],
             step=1, lr=1e-3)
    return t | kw


def test_refusals():
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    for kw in [dict(grads=[]), dict(exp_avg=[]), dict(params=[z(40), z(40)]), dict(grads=[z(41)]),
               dict(grads=[z(40).half()]), dict(params=[z(40).half()]), dict(exp_avg=[z(40).bfloat16()]),
               dict(grads=[z(80)[::2]]), dict(params=[z(4, 10).t()], grads=[z(10, 4)],
                                              exp_avg=[z(10, 4)], exp_avg_sq=[z(10, 4)]),
               dict(grads=[torch.zeros(40)]), dict(params=[torch.zeros(40)]), dict(grads=[None]),
               dict(exp_avg=[z(40, dtype=torch.uint8)]), dict(exp_avg_scale=[z(2, dtype=torch.uint8)]),
               dict(master=[z(41)]), dict(master=[z(40).bfloat16()]), dict(norm=z(2)),
               dict(norm=torch.zeros(1)), dict(step=z(1)), dict(lr=z(1).double()), dict(step=0),
               dict(step=2 ** 31)]:
        with pytest.raises((TypeError, ValueError)):
            df2.adamw(**_one(**kw))
    p = z(40)
    for kw in [dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(eps=1e-60), dict(lr=NAN),
               dict(weight_decay=INF), dict(max_norm=1.0), dict(max_norm=-1.0, norm=z(1)),
               dict(grad_scale=NAN), dict(master=[z(40)]), dict(params=[p], grads=[p]),
               dict(params=[p], exp_avg=[p]), dict(norm=p[:1], params=[p])]:
        with pytest.raises(df2.Dflash2Error):
            df2.adamw(**_one(**kw))
    twice = {k: v * 2 for k, v in _one().items() if isinstance(v, list)}
    with pytest.raises(df2.Dflash2Error, match="overlaps"):
        df2.adamw(**twice, step=1, lr=1e-3)
    both = z(100)
    with pytest.raises(df2.Dflash2Error, match="overlaps"):
        df2.adamw(**_one(params=[both[:40]], exp_avg=[both[39:79]]))
    shared = z(40)                      # two gradients may share memory
    two = {k: [v[0], v[0].clone()] for k, v in _one().items() if isinstance(v, list)}
    df2.adamw(**(two | dict(grads=[shared, shared])), step=1, lr=1e-3)
    df2.adamw([], [], [], [], step=1, lr=1e-3)
    with pytest.raises(ValueError):
        df2.adamw([], [p], [], [], step=1, lr=1e-3)
    for bad in [(p, z(2, dtype=torch.uint8)), (z(40, dtype=torch.uint8), z(3, dtype=torch.uint8))]:
        with pytest.raises((TypeError, ValueError)):
            df2.state_decode(*bad)
    with pytest.raises((TypeError, ValueError)):
        df2.state_encode(z(40).half())
