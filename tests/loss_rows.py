"""Inputs, formulas in 64 bits and error bounds of the losses of a token's log-probability.

Bounds, for logits z over T in fp32 (c = log2(e) / T rounded):
  logp: z * c - base is one rounded fused multiply-add, 2^x is good to 2^-22, the sum of
    positive terms adds at most 2^-24 a step of a tree of depth < 80: 8e-6 in log's
    argument; c, the multiply-add, log2 and the product with ln 2 are good to 2^-22 of depth
    and log together, which make up logp and have the same sign: 2^-21 * |logp|.
  lse: the same 8e-6, and 2^-22 * |lse| for c.
  exp(logp - old): the exponent is off by logp's bound and a rounding, the power by 2^-21.
  exp(d) - d - 1: (exp(d) - 1) times d's error, and 2^-21 of exp(d), d and 1.
  gradient: g's error, and 1e-5 of g for the share (8e-6 and 2^-21 of s * log s); over T; in bf16
    its unit roundoff, 2^-8 of the value, more.
"""
import numpy as np
import torch

NAN, INF = float("nan"), float("inf")
F32 = torch.float32


def place(x, dtype, pad=0, offset=0):
    """x in a buffer with NaN around its rows, which start at any element."""
    dt = torch.bfloat16 if dtype == "bf16" else F32
    rows, V = x.shape
    buf = torch.full((rows * (V + pad) + offset + 64,), NAN, dtype=dt, device="cuda")
    v = buf[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, :V]
    v.copy_(x.to(dt))
    return v


def rows_of(rows, V, dtype, seed, pad=0, offset=0, std=3.0):
    """Logits and a token of every row, on the whole a likely one."""
    g = torch.Generator().manual_seed(seed)
    z = place(torch.randn((rows, V), generator=g) * std, dtype, pad, offset)
    pick = z.float().cpu() + torch.randn((rows, V), generator=g) * 2
    return z, pick.argmax(1).to(torch.int32).cuda(), g


def logp64(z, tokens, T):
    """(logp, lse, shares) in 64 bits; a row with nothing above -inf has no shares."""
    x = z.double() / T
    m = x.amax(1, keepdim=True)
    e = torch.where(m > -INF, torch.exp(x - torch.where(m > -INF, m, 0.0)), 0.0)
    s = e.sum(1, keepdim=True)
    lse = torch.where(m > -INF, m + torch.log(s), -INF).squeeze(1)
    at = x.gather(1, tokens.long().clamp(0, z.shape[1] - 1)[:, None])
    # the maximum first: beside -3e38 the logarithm of the sum is lost in 64 bits too
    logp = torch.where(lse > -INF, ((at - m) - torch.log(s)).squeeze(1),
                       torch.where(torch.isnan(lse), NAN, -INF))
    return logp, lse, e / torch.where(s == 0, 1.0, s)


def logp_bound(logp):
    return 8e-6 + 2.0 ** -21 * torch.where(torch.isfinite(logp), logp, 0.0).abs()


def lse_bound(lse):
    return 8e-6 + 2.0 ** -22 * torch.where(torch.isfinite(lse), lse, 0.0).abs()


def gradient64(share, tokens, g, T):
    d = -share
    at = tokens.long().clamp(0, share.shape[1] - 1)[:, None]
    d = d.scatter_add(1, at, torch.ones_like(at, dtype=torch.float64))
    return torch.where(g[:, None] == 0, 0.0, d * (g / T)[:, None])


def gradient_bound(grad, g, g_bound, T, bf16):
    b = ((g_bound + 1e-5 * g.abs()) / T)[:, None]
    return b + (2.0 ** -8 * grad.abs() if bf16 else 2.0 ** -22 * grad.abs())


def same(got, ref, bound, what):
    """Within the bound where the reference is finite, the same elsewhere."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), (what, "NaN")
    odd = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[odd], ref[odd]), (what, "infinite")
    err = torch.where(fine, got - ref, 0.0).abs()
    bound = torch.as_tensor(bound, dtype=torch.float64, device=err.device).expand(err.shape)
    over = torch.where(fine, err - bound, -1.0)
    assert not (over > 0).any(), (what, over.max().item(), err.max().item())


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def equal_bits(a, b):
    return torch.equal(bits(a), bits(b))


def policy64(z, tokens, old, A, ref, w, T, lo, hi, kl, up=None, edge=None):
    """(loss, logp, lse, grad, g, bounds of loss and g, rows at an edge) of all rows.  At an edge of
    the clamp, where fp32's error in the ratio reaches over it, both one-sided slopes are right:
    `edge` (a truth value for every row) says whether the ratio counts as inside there."""
    lp, lse, share = logp64(z, tokens, T)
    used = (tokens >= 0) & (tokens < z.shape[1]) & (w != 0)
    logp = lp
    A, w = A.double(), w.double()
    old = old.double()
    rho = torch.exp(logp - old)
    inside = torch.where(A > 0, ~(rho > 1 + hi), ~(rho < 1 - lo))
    e1 = logp_bound(logp) + 2.0 ** -23 * (torch.nan_to_num(logp, 0, 0, 0).abs() + old.abs())
    limit = torch.where(A > 0, 1.0 + hi, 1.0 - lo)
    at_edge = (rho - limit).abs() <= rho * (e1 + 2.0 ** -21) + 2.0 ** -24 * limit
    if edge is not None:
        inside = torch.where(at_edge, edge, inside)
    gain = torch.where(A == 0, 0.0, torch.where(inside, rho, torch.where(A > 0, 1.0 + hi, 1.0 - lo)) * A)
    g = torch.where((A != 0) & inside, -A * rho, 0.0)
    off = torch.where((A != 0) & inside, A.abs() * rho, 0.0) * (e1 + 2.0 ** -21)
    loss, g_off = -gain, off
    if kl:
        d = ref.double() - logp
        up_d = torch.exp(d)
        e2 = logp_bound(logp) + 2.0 ** -23 * (torch.nan_to_num(logp, 0, 0, 0).abs() + ref.double().abs())
        loss = loss + kl * torch.where(up_d == INF, INF, torch.expm1(d) - d)
        g = g + kl * (1 - up_d)
        rest = 2.0 ** -21 * (up_d + torch.nan_to_num(d, 0, 0, 0).abs() + 1)
        off = off + abs(kl) * ((up_d - 1).abs() * e2 + rest)
        g_off = g_off + abs(kl) * (up_d * e2 + rest)
    g, g_off = g * w, g_off * w.abs()
    if up is not None:
        g, g_off = g * up.double(), g_off * up.double().abs()
    zero = torch.zeros_like(loss)
    g, g_off = torch.where(used, g, zero), torch.where(used, g_off, zero)
    loss = torch.where(used, w * loss, zero)
    grad = gradient64(share, tokens, g, T)
    return (loss, torch.where(used, logp, zero), torch.where(used, lse, zero), grad, g,
            w.abs() * off + 2.0 ** -21 * torch.nan_to_num(loss, 0, 0, 0).abs(), g_off,
            at_edge & used & (A != 0))


def policy64_like(got, z, *args):
    """policy64 with the rows at an edge on the side that `got`, the gradient, is nearer to."""
    a = policy64(z, *args)
    if not a[7].any():
        return a[:7]
    sides = [policy64(z, *args, edge=torch.full((z.shape[0],), e, device=z.device))
             for e in (True, False)]
    far = [torch.nan_to_num(got.double() - s[3], 0, 0, 0).abs().sum(1) for s in sides]
    return policy64(z, *args, edge=far[0] <= far[1])[:7]


def by_numbers(*values):
    return [torch.tensor(v, dtype=F32, device="cuda") for v in values]


def linspace(lo, hi, n):
    return torch.from_numpy(np.linspace(lo, hi, n).astype(np.float32)).cuda()
