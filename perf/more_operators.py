"""Measured cases of the operators that train a draft head on rewards and move its weights.

policy / policy_backward: the clipped policy loss with a KL term on whole vocabulary
    rows, with its gradient in the same call (a training step), and the gradient alone.
preference / preference_forward / preference_backward: the loss of pairs of sequences by
    their log ratios, with its gradient, the loss alone, the gradient alone.
norm: the 2-norm of the gradients of many tensors.
adamw: one AdamW step over many tensors, where `clip` is set behind their norm, with states
    in 32 bits or in 8.

Sizes of tensors are a text of numbers.  The tensors of an optimizer case are parts of one
buffer, as programs keep them that gather their weights, so that a case returns a buffer
instead of each of its tensors; what lies between two tensors stays zero.
"""
import math

import torch

own = False

HEAD_TINY = "1024,8192,4096,16000,16000"             # base, taps' projection, projection, codebooks
HEAD = "20480,819200,655360,19447808,19447808"
HEAD_WIDE = "21504,903168,1376256,67108864,67108864"
C1, C2, MASK = 0x927aa3cd, 0x93e1aa55, 0xffffffff    # of the rounding's pseudo-random bits
BLOCK = 32                                           # elements that share an exponent


def listed():
    """The cases that are always measured, small to large."""
    return [
        # the smallest step on rewards: one draft block of the tiny fp32 configuration
        _policy("policy_tiny_8x1000_f32", "policy", "f32", 8, 1000, kl_coef=0.04),
        # the gradient behind a loss that was mixed with others: ragged rows of an odd width in
        # a padded buffer, drafts sampled at a temperature, positions that count less
        _policy("policy_grad_333x50021", "policy_backward", "bf16", 333, 50021, pad=3,
                kl_coef=0.02, temperature=0.7, weighted=True),
        # a training step over the batched regime's positions
        _policy("policy_train_4096x151936", "policy", "bf16", 4096, 151936, kl_coef=0.04,
                weighted=True),
        # the smallest preference step: two pairs of short drafts
        _preference("preference_tiny_26x1000_f32", "preference", "f32", 26, 1000, pairs=2),
        # the evaluation loss of wide fp32 rows, mean log ratios
        _preference("preference_eval_512x262144_f32", "preference_forward", "f32", 512, 262144,
                    pairs=4, average=True),
        # a training step: eight pairs of about 128 positions, a quarter of each a prompt
        _preference("preference_train_2048x151936", "preference", "bf16", 2048, 151936, pairs=8,
                    smoothing=0.1),
        # the gradients' norm of the tiny configuration's head, and of the batched one's
        _norm("norm_tiny_f32", "f32", HEAD_TINY),
        _norm("norm_head_bf16", "bf16", HEAD),
        # a step of the tiny head, clipped: latency counts
        _adamw("adamw_tiny_f32", HEAD_TINY, clip=0.5),
        # sixty tensors of odd sizes, bf16 with fp32 copies
        _adamw("adamw_ragged_60", _sizes(7, 60, 1, 400000), p="bf16", g="bf16", master=True),
        # the batched configuration's head with states in 8 bits, clipped, rounded by chance
        _adamw("adamw_head_8bit", HEAD, p="bf16", g="bf16", state=8, clip=1.0, chance=True),
        # the wide configuration's head, everything in fp32
        _adamw("adamw_wide_f32", HEAD_WIDE),
    ]


def _policy(name, op, dtype, rows, V, pad=0, kl_coef=0.0, temperature=1.0, weighted=False):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "V": V, "pad": pad,
            "kl_coef": kl_coef, "temperature": temperature, "weighted": weighted}


def _preference(name, op, dtype, rows, V, pad=0, pairs=1, average=False, smoothing=0.0,
                margin=0.0, weighted=False):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "V": V, "pad": pad,
            "pairs": pairs, "average": average, "smoothing": smoothing, "margin": margin,
            "weighted": weighted}


def _norm(name, dtype, sizes):
    return {"name": name, "op": "norm", "g": dtype, "sizes": sizes}


def _adamw(name, sizes, p="f32", g="f32", state=32, master=False, clip=0.0, chance=False):
    return {"name": name, "op": "adamw", "sizes": sizes, "p": p, "g": g, "state": state,
            "master": master, "clip": clip, "chance": chance}


def _sizes(seed, count, lo, hi):
    """`count` sizes spread over the logarithm of [lo, hi], the same for the same seed."""
    got, x = [], seed * 2654435761 + 12345
    for _ in range(count):
        x = (x * 1103515245 + 12345) % (1 << 31)
        got.append(int(round(lo * (hi / lo) ** (x / (1 << 31)))))
    return ",".join(str(n) for n in got)


def draw(rng):
    """One more case: 1 to 4096 rows of 512 to 262144 entries, both types, any settings; 1 to 60
    tensors of 1 to 60 million elements, all types."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["policy", "policy_backward", "preference", "preference_forward",
                     "preference_backward", "norm", "adamw", "adamw"])
    if op in ("norm", "adamw"):
        count = spread(1, 60)
        most = spread(300, 60000000)
        most = min(most, 120000000 // count)
        sizes = _sizes(rng.randrange(1 << 20), count, max(1, most // spread(1, 10000)), most)
        g = rng.choice(["f32", "bf16"])
        if op == "norm":
            c = _norm("", g, sizes)
        else:
            p = rng.choice(["f32", "bf16"])
            c = _adamw("", sizes, p, g, rng.choice([32, 8]), p == "bf16" and rng.random() < 0.5,
                       rng.choice([0.0, 0.5, 100.0]), rng.random() < 0.5)
        del c["name"]
        return c
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = spread(512, 262144)
    V = V // 64 * 64 if rng.random() < 0.5 else V
    es = 4 if dtype == "f32" else 2
    rows = min(spread(1, 4096), 4096 * 151936 * 2 // (V * es))
    pad = rng.choice([0, 0, 1, 7, 64])
    if op.startswith("policy"):
        c = _policy("", op, dtype, rows, V, pad, rng.choice([0.0, 0.04, 0.2]),
                    rng.choice([1.0, 1.0, 0.6, 1.5]), rng.random() < 0.5)
    else:
        rows = max(2, rows * 2 // 3)
        c = _preference("", op, dtype, rows, V, pad, spread(1, max(1, rows // 4)),
                        rng.random() < 0.3, rng.choice([0.0, 0.0, 0.1]),
                        rng.choice([0.0, 0.0, 0.5]), rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def _logits(case, g):
    """Logit rows: a normal bulk and, in every row, 64 tokens that stand out by an
    amount that falls off with their rank; 0 (a flat row) to 18 (a sure one) at the top.
    In the case's type, in a buffer whose rows are V + pad elements apart."""
    rows, V, dev = case["rows"], case["V"], "cuda"
    x = torch.randn((rows, V), device=dev, generator=g) * 2.0
    top = torch.rand((rows, 1), device=dev, generator=g) * 18.0
    fall = torch.exp(-torch.arange(64, device=dev, dtype=torch.float32) / 6.0)
    ids = torch.sort(torch.randint(0, V, (rows, 64), device=dev, generator=g), dim=1)[0]
    fresh = torch.ones_like(ids, dtype=torch.bool)
    fresh[:, 1:] = ids[:, 1:] != ids[:, :-1]  # an id drawn twice counts once
    order = torch.argsort(torch.rand((rows, 64), device=dev, generator=g), dim=1)
    x.scatter_add_(1, ids, top * fall[order] * fresh)
    buf = torch.zeros((rows, V + case["pad"]), device=dev,
                      dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
    buf[:, :V] = x
    return buf[:, :V], x


def _drawn_tokens(x, T, g):
    """A token of every row with its share at temperature T, and the rows' lse there."""
    lse = torch.logsumexp(x / T, dim=1)
    # share / an exponential variable each: the largest falls on j with its share
    e = torch.empty_like(x).exponential_(generator=g)
    tokens = torch.argmax(x / T - torch.log(e), dim=1)
    return tokens, lse


def _lengths(case):
    """Rows of every sequence: about equal parts, some shorter, some longer, one in a hundred
    of the rows left over behind the last."""
    n, rows = 2 * case["pairs"], case["rows"]
    rows -= rows // 100
    cuts = [rows * k // n + ((k * 7919) % 5 - 2) * (rows // n // 8) for k in range(n)]
    cuts[0] = 0
    return [b - a for a, b in zip(cuts, cuts[1:] + [rows])]


def _prompt(length):
    return length // 4


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] in ("norm", "adamw"):
        return _prepare_tensors(case, g, s)
    rows, dev = case["rows"], "cuda"
    s["logits"], x = _logits(case, g)
    x.copy_(s["logits"])
    T = case.get("temperature", 1.0)
    tokens, lse = _drawn_tokens(x, T, g)
    logp = x.gather(1, tokens[:, None]).squeeze(1) / T - lse
    s["tokens"], s["lse"], s["logp"] = tokens.to(torch.int32), lse, logp

    def noise(scale):
        return torch.randn((rows,), device=dev, generator=g) * scale

    s["weight"] = None
    if case["op"].startswith("policy"):
        # the drafts come from a slightly older head, the reference is further away
        s["old"], s["ref"] = logp + noise(0.15), logp + noise(0.4)
        s["advantage"] = noise(1.0)
        if case["weighted"]:  # blocks of 16 positions, later ones count less, two are padding
            at = torch.arange(rows, device=dev) % 16
            s["weight"] = torch.where(at < 14, 0.95 ** at.float(), 0.0) / rows
        s["grad_loss"] = (0.5 + torch.rand((rows,), device=dev, generator=g)) / rows
        return s
    lengths = _lengths(case)
    ends = [sum(lengths[:k]) for k in range(len(lengths) + 1)]
    for start, n in zip(ends, lengths):
        s["tokens"][start:start + _prompt(n)] = -1
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=dev)
    s["tokens"][ends[-1]:] = -1
    s["pairs"] = pairs = case["pairs"]
    counted = (s["tokens"] >= 0).float() * logp
    total, count = _by_sequence(counted, s), _by_sequence((s["tokens"] >= 0).float(), s)
    s["seq_logp"] = total / count.clamp(min=1) if case["average"] else total
    s["ref"] = s["seq_logp"] + torch.randn((2 * pairs,), device=dev, generator=g) * (
        1.0 if case["average"] else 6.0)
    if case["weighted"]:
        s["weight"] = 0.25 + torch.rand((pairs,), device=dev, generator=g)
        s["weight"][0] = 0.0
    s["grad_loss"] = (0.5 + torch.rand((pairs,), device=dev, generator=g)) / pairs
    return s


def _by_sequence(v, s):
    """Sums of a value of every row over the sequences, in 64 bits."""
    run = torch.zeros(v.numel() + 1, dtype=torch.float64, device=v.device)
    run[1:] = v.double().cumsum(0)
    at = s["offsets"].long()
    return (run[at[1:]] - run[at[:-1]]).float()


def _numbers(case):
    return [int(n) for n in case["sizes"].split(",")]


def _place(sizes):
    """Where each tensor starts in the buffer, and the buffer's size."""
    at, ends = 0, []
    for n in sizes:
        ends.append(at)
        at += -(-n // 64) * 64
    return ends, at


def _views(flat, sizes, per=1):
    starts = _place(sizes)[0]
    return [flat[a // per:a // per + -(-n // per)] for a, n in zip(starts, sizes)]


def _prepare_tensors(case, g, s):
    sizes, dev = _numbers(case), "cuda"
    _, total = _place(sizes)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    held = torch.zeros(total, dtype=torch.bool, device=dev)
    for v in _views(held, sizes):
        v.fill_(True)

    def values(dtype, scale):
        x = torch.randn(total, device=dev, generator=g) * held
        # neighbours differ by orders of magnitude, as rows of rare tokens do
        x *= torch.exp2(torch.randn(-(-total // 16), device=dev, generator=g) * 2.0
                        ).repeat_interleave(16)[:total] * scale
        return x.to(dtype)

    s["grad"] = values(kind[case["g"]], 1e-3)
    s["grads"] = _views(s["grad"], sizes)
    if case["op"] == "norm":
        return s
    p = torch.randn(total, device=dev, generator=g).mul_(0.02).mul_(held)
    s["param"] = p.to(kind[case["p"]])
    s["params"] = _views(s["param"], sizes)
    s["copy"] = s["copies"] = None
    if case["master"]:
        s["copy"] = p
        s["copies"] = _views(p, sizes)
    m, v = values(torch.float32, 4e-4), values(torch.float32, 1e-3).square_()
    if case["state"] == 8:
        m, s["m_scale"] = _encode(m, True, None)
        v, s["v_scale"] = _encode(v, False, None)
        s["m_scales"] = _views(s["m_scale"], sizes, BLOCK)
        s["v_scales"] = _views(s["v_scale"], sizes, BLOCK)
    s["m"], s["v"] = m, v
    s["ms"], s["vs"] = _views(m, sizes), _views(v, sizes)
    s["step"], s["seed"] = 1000, 20260 + int(torch.randint(0, 1 << 30, (1,), generator=g,
                                                            device=dev)) if case["chance"] else None
    return s


LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.01


# ------------------------------------------------------------------ one pass


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    if c["op"].startswith("policy"):
        return _plain_policy(s, c)
    if c["op"].startswith("preference"):
        return _plain_preference(s, c)
    if c["op"] == "norm":
        return {"norm": _plain_norm(s["grads"])}
    return _plain_adamw(s, c)


def _own(s, c):
    import dflash2_draft_head_gb300 as df2
    op = c["op"]
    if op == "policy":
        loss, logp, lse, grad = df2.policy_loss(
            s["logits"], s["tokens"], s["old"], s["advantage"], ref_logp=s["ref"],
            temperature=c["temperature"], kl_coef=c["kl_coef"], weight=s["weight"], grad=True)
        return {"loss": loss, "logp": logp, "lse": lse, "grad": grad}
    if op == "policy_backward":
        return {"grad": df2.policy_loss_backward(
            s["grad_loss"], s["logits"], s["tokens"], s["old"], s["advantage"], s["logp"],
            s["lse"], ref_logp=s["ref"], temperature=c["temperature"], kl_coef=c["kl_coef"],
            weight=s["weight"])}
    if op in ("preference", "preference_forward"):
        loss, seq_logp, logp, lse, grad = df2.preference_loss(
            s["logits"], s["tokens"], s["offsets"], ref_logp=s["ref"],
            label_smoothing=c["smoothing"], margin=c["margin"], average=c["average"],
            weight=s["weight"], grad=op == "preference")
        out = {"loss": loss, "seq_logp": seq_logp, "logp": logp, "lse": lse}
        return out | ({"grad": grad} if op == "preference" else {})
    if op == "preference_backward":
        return {"grad": df2.preference_loss_backward(
            s["grad_loss"], s["logits"], s["tokens"], s["offsets"], s["seq_logp"], s["lse"],
            ref_logp=s["ref"], label_smoothing=c["smoothing"], margin=c["margin"],
            average=c["average"], weight=s["weight"])}
    if op == "norm":
        return {"norm": df2.grad_norm(s["grads"])}
    norm = df2.grad_norm(s["grads"]) if c["clip"] else None
    small = c["state"] == 8
    df2.adamw(s["params"], s["grads"], s["ms"], s["vs"], step=s["step"], lr=LR, beta1=BETA1,
              beta2=BETA2, eps=EPS, weight_decay=DECAY, master=s["copies"],
              exp_avg_scale=s["m_scales"] if small else None,
              exp_avg_sq_scale=s["v_scales"] if small else None, norm=norm,
              max_norm=c["clip"] if c["clip"] else None, seed=s["seed"])
    out = {"param": s["param"], "m": s["m"], "v": s["v"]}
    if small:
        out["m"] = df2.state_decode(s["m"], s["m_scale"], dtype=torch.bfloat16)
        out["v"] = df2.state_decode(s["v"], s["v_scale"], squares=True, dtype=torch.bfloat16)
    if c["master"]:
        out["copy"] = s["copy"]
    if norm is not None:
        out["norm"] = norm
    return out


def _share_and_gradient(s, lse, g, inv):
    """g[r] * (1 at the row's token - softmax) / T, in the logits' type."""
    z = s["logits"].float() * inv
    token = s["tokens"].long()
    grad = torch.exp(z - lse[:, None]) * (-g * inv)[:, None]
    # a row without a token has g = 0
    grad.scatter_add_(1, token.clamp(min=0)[:, None], (g * inv)[:, None])
    return grad.to(s["logits"].dtype)


def _logp(s, inv):
    z = s["logits"].float() * inv
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    token = s["tokens"].long()
    return z.gather(1, token.clamp(min=0)[:, None]).squeeze(1) - lse, lse


def _plain_policy(s, c):
    inv, kl, A, low, high = 1.0 / c["temperature"], c["kl_coef"], s["advantage"], 0.8, 1.2
    weight = 1.0 if s["weight"] is None else s["weight"]
    if c["op"] == "policy":
        logp, lse = _logp(s, inv)
    else:
        logp, lse = s["logp"], s["lse"]
    ratio = torch.exp(logp - s["old"])
    back = torch.exp(s["ref"] - logp)
    inside = torch.where(A > 0, ratio <= high, ratio >= low)
    g = weight * (kl * (1.0 - back) - torch.where(inside, A * ratio, 0.0))
    if c["op"] == "policy_backward":
        g = g * s["grad_loss"]
        return {"grad": _share_and_gradient(s, lse, g, inv)}
    gain = torch.minimum(ratio * A, ratio.clamp(low, high) * A)
    loss = weight * (kl * (back - (s["ref"] - logp) - 1.0) - gain)
    grad = _share_and_gradient(s, lse, g, inv)
    if s["weight"] is not None:
        logp, lse = (torch.where(weight != 0, v, 0.0) for v in (logp, lse))
    return {"loss": loss, "logp": logp, "lse": lse, "grad": grad}


def _plain_preference(s, c):
    P, beta, smooth = c["pairs"], 0.1, c["smoothing"]
    weight = 1.0 if s["weight"] is None else s["weight"]
    used = s["tokens"] >= 0
    count = _by_sequence(used.float(), s).clamp(min=1)
    if c["op"] == "preference_backward":
        seq, lse = s["seq_logp"], s["lse"]
    else:
        logp, lse = _logp(s, 1.0)
        logp, lse = (torch.where(used, v, 0.0) for v in (logp, lse))
        seq = _by_sequence(logp, s)
        seq = seq / count if c["average"] else seq
    d = seq - s["ref"]
    m = beta * (d[:P] - d[P:]) - c["margin"]
    # log(1 + e^x) without overflow
    minus, plus = (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())) for x in (-m, m))
    out = {}
    if c["op"] != "preference_backward":
        out = {"loss": weight * ((1 - smooth) * minus + smooth * plus), "seq_logp": seq,
               "logp": logp, "lse": lse}
        if c["op"] == "preference_forward":
            return out
    up = s["grad_loss"] if c["op"] == "preference_backward" else 1.0
    by_margin = ((1 - smooth) / (1 + torch.exp(m)) - smooth / (1 + torch.exp(-m))) * (
        beta * weight * up)
    by_seq = torch.cat([-by_margin, by_margin])
    by_seq = by_seq / count if c["average"] else by_seq
    rows = torch.arange(used.numel(), device=used.device)
    of = torch.bucketize(rows, s["offsets"].long(), right=True) - 1
    g = torch.where(used & (of < 2 * P), by_seq[of.clamp(max=2 * P - 1)], 0.0)
    return out | {"grad": _share_and_gradient(s, lse, g, 1.0)}


def _plain_norm(grads):
    return torch.sqrt(torch.stack([g.float().square().sum(dtype=torch.float64)
                                   for g in grads]).sum()).float().reshape(1)


def _decode(codes, scale, signed):
    """Values of 8-bit codes: the bits of a short float (sign and 4 exponent bits, or 5 and no
    sign; 3 of mantissa) times 2^(scale - 127), the scale shared by 32."""
    n = codes.numel()
    code = codes.to(torch.int32)
    x = ((code & 127 if signed else code) << 20).view(torch.float32)
    x = x * (2.0 ** 120 if signed else 2.0 ** 112)
    x = x * (scale.to(torch.int32) << 23).view(torch.float32).repeat_interleave(BLOCK)[:n]
    return torch.where(code >= 128, -x, x) if signed else x


def _encode(x, signed, bits):
    """(codes, scales) of fp32 values: to the nearest where `bits` is None, else up or down by
    16 of them.  A value above 0 in a state without sign has a code above 0."""
    n = x.numel()
    wide = torch.zeros(-(-n // BLOCK) * BLOCK, device=x.device)
    wide[:n] = x
    field = (wide.view(-1, BLOCK).abs().amax(1).view(torch.int32) >> 23)
    scale = (field - (7 if signed else 15)).clamp(min=1)
    y = x.abs() * ((254 - scale) << 23).view(torch.float32).repeat_interleave(BLOCK)[:n]
    w = (y * (2.0 ** -120 if signed else 2.0 ** -112)).view(torch.int32)
    if bits is None:
        code = (w + 0x7ffff + ((w >> 20) & 1)) >> 20
    else:
        code = (w + (bits << 4 | 8)) >> 20
    if signed:
        code = code | torch.where(x < 0, 128, 0)
    else:
        code = torch.where(x > 0, code.clamp(min=1), code)
    return code.to(torch.uint8), scale.to(torch.uint8)


def _mix(x):
    for shift, mul in ((16, C1), (15, C2), (16, 1)):
        x = (x ^ x >> shift) * mul & MASK
    return x


def _keys(seed, step, tensor):
    k1 = _mix((seed & MASK) ^ _mix((seed >> 32 & MASK) ^ _mix(step)))
    return k1, _mix(k1 + tensor + 1 & MASK)


def _chance(n, keys, dev):
    """Three 16-bit numbers for every element: of the first state, the second, the weight."""
    x = (torch.arange(n, device=dev) ^ keys[0]) * C1 & MASK
    x = ((x ^ x >> 16) + keys[1] & MASK) * C2 & MASK
    x = x ^ x >> 15
    return [v.to(torch.int32) for v in (x & 0xffff, x >> 16, (x * C1 & MASK) >> 16)]


def _plain_adamw(s, c):
    norm = None
    if c["clip"]:
        norm = _plain_norm(s["grads"])
        by = torch.clamp(c["clip"] / norm, max=1.0)
    left1, left2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    small = c["state"] == 8
    for k, (p, g, m, v) in enumerate(zip(s["params"], s["grads"], s["ms"], s["vs"])):
        w = s["copies"][k] if c["master"] else p.float()
        m32 = _decode(m, s["m_scales"][k], True) if small else m
        v32 = _decode(v, s["v_scales"][k], False) if small else v
        g = g.float()
        if norm is not None:
            g = g * by
        m32 = m32 * BETA1 + g * (1 - BETA1)
        v32 = v32 * BETA2 + g * g * (1 - BETA2)
        w = w * (1 - LR * DECAY) - (LR / left1) * m32 / (torch.sqrt(v32) / math.sqrt(left2) + EPS)
        r = [None] * 3
        if s["seed"] is not None and (small or c["p"] == "bf16" and not c["master"]):
            r = _chance(p.numel(), _keys(s["seed"], s["step"], k), p.device)
        if small:
            m32, s["m_scales"][k][:] = _encode(m32, True, r[0])
            v32, s["v_scales"][k][:] = _encode(v32, False, r[1])
        m.copy_(m32)
        v.copy_(v32)
        if c["master"]:
            s["copies"][k].copy_(w)
        elif r[2] is not None and c["p"] == "bf16":
            w = ((w.view(torch.int32) + r[2]) & -65536).view(torch.float32)
        p.copy_(w)
    out = {"param": s["param"], "m": s["m"], "v": s["v"]}
    if small:
        out["m"] = _decode(s["m"], s["m_scale"], True).bfloat16()
        out["v"] = _decode(s["v"], s["v_scale"], False).bfloat16()
    if c["master"]:
        out["copy"] = s["copy"]
    if norm is not None:
        out["norm"] = norm
    return out


# ------------------------------------------------------------------ what a pass needs


def work(case):
    if case["op"] in ("norm", "adamw"):
        n = sum(_numbers(case))
        eg = 4 if case["g"] == "f32" else 2
        if case["op"] == "norm":
            return {"bytes": n * eg, "flops": 2 * n}
        ep = 4 if case["p"] == "f32" else 2
        state = 8 if case["state"] == 32 else 2 + 2 / BLOCK
        once = (ep + 8 if case["master"] else 2 * ep) + eg + 2 * state
        return {"bytes": n * once, "flops": 14 * n}
    rows, V = case["rows"], case["V"]
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("policy"):
        live = sum(1 for r in range(rows) if r % 16 < 14) if case["weighted"] else rows
        flops = (7 if case["op"] == "policy" else 4) * live * V
        return {"bytes": (live + rows) * V * es + rows * 32, "flops": flops}
    live = sum(n - _prompt(n) for n in _lengths(case))
    if case["op"] == "preference_forward":
        return {"bytes": live * V * es + rows * 12, "flops": 4 * live * V}
    flops = (8 if case["op"] == "preference" else 4) * live * V
    return {"bytes": (live + rows) * V * es + rows * 12, "flops": flops}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The same outputs in 64 bits; logit rows block by block."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        return {"norm": torch.linalg.vector_norm(s["grad"].double()).reshape(1)}
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    rows, V = case["rows"], case["V"]
    T = case.get("temperature", 1.0)
    tokens = s["tokens"].long()
    used = tokens >= 0
    step = max(1, (1 << 26) // V)
    blocks = [(lo, min(rows, lo + step)) for lo in range(0, rows, step)]

    def log_shares(lo, hi, lse=None):
        z = s["logits"][lo:hi].double() / T
        return z - (torch.logsumexp(z, dim=1) if lse is None else lse).unsqueeze(1)

    alone = case["op"].endswith("backward")
    lse = s["lse"].double()
    if not alone:
        lse = torch.cat([torch.logsumexp(s["logits"][lo:hi].double() / T, dim=1)
                         for lo, hi in blocks])
    at_token = s["logits"].gather(1, tokens.clamp(min=0)[:, None]).squeeze(1).double() / T
    if case["op"].startswith("policy"):
        out, g = _exact_policy(case, s, s["logp"].double() if alone else at_token - lse, lse, alone)
    else:
        out, g = _exact_preference(case, s, torch.where(used, at_token - lse, 0.0),
                                   torch.where(used, lse, 0.0), used, alone)
    if not case["op"].endswith("forward"):
        parts = []
        for lo, hi in blocks:
            d = -torch.exp(log_shares(lo, hi, lse[lo:hi]))
            here = torch.arange(hi - lo, device=d.device)[used[lo:hi]]
            d[here, tokens[lo:hi][used[lo:hi]]] += 1
            parts.append((d * (g[lo:hi] / T).unsqueeze(1)).to(torch.float32)
                         if rows * V > 1 << 28 else d * (g[lo:hi] / T).unsqueeze(1))
        out["grad"] = torch.cat(parts)
    return out


def _exact_policy(case, s, logp, lse, alone):
    A, k = s["advantage"].double(), case["kl_coef"]
    w = torch.ones_like(logp) if s["weight"] is None else s["weight"].double()
    rho, behind = torch.exp(logp - s["old"].double()), s["ref"].double() - logp
    lowest = torch.where(A >= 0, torch.full_like(A, -math.inf), torch.full_like(A, 0.8))
    highest = torch.where(A >= 0, torch.full_like(A, 1.2), torch.full_like(A, math.inf))
    # where A > 0 only the upper limit can lower the product, where A < 0 only the lower one
    held = torch.maximum(torch.minimum(rho, highest), lowest)
    loss = w * (k * (torch.exp(behind) - behind - 1) - held * A)
    g = w * (k * (1 - torch.exp(behind)) - A * rho * (held == rho))
    if alone:
        return {}, g * s["grad_loss"].double()
    return {"loss": loss, "logp": torch.where(w != 0, logp, 0.0),
            "lse": torch.where(w != 0, lse, 0.0)}, g


def _exact_preference(case, s, logp, lse, used, alone):
    P, ends = case["pairs"], [int(v) for v in s["offsets"]]
    logits_of, g = [], torch.zeros_like(logp)
    counts = [max(1, int(used[a:b].sum())) for a, b in zip(ends, ends[1:])]
    for n, a, b in zip(counts, ends, ends[1:]):
        logits_of.append(logp[a:b].sum() / (n if case["average"] else 1))
    seq = s["seq_logp"].double() if alone else torch.stack(logits_of)
    ratio = seq - s["ref"].double()
    m = 0.1 * (ratio[:P] - ratio[P:]) - case["margin"]
    w = torch.ones_like(m) if s["weight"] is None else s["weight"].double()
    e = case["smoothing"]
    loss = -w * ((1 - e) * torch.nn.functional.logsigmoid(m)
                 + e * torch.nn.functional.logsigmoid(-m))
    slope = -w * ((1 - e) * torch.sigmoid(-m) - e * torch.sigmoid(m))
    if alone:
        slope = slope * s["grad_loss"].double()
    for k, (n, a, b) in enumerate(zip(counts, ends, ends[1:])):
        by = 0.1 * slope[k % P] / (n if case["average"] else 1)
        g[a:b] = torch.where(used[a:b], by if k < P else -by, 0.0)
    return ({} if alone else {"loss": loss, "seq_logp": seq, "logp": logp, "lse": lse}), g


def _exact_value(codes, scale, signed):
    c = codes.double()
    minus = torch.where(c >= 128, -1.0, 1.0) if signed else torch.ones_like(c)
    c = torch.where(c >= 128, c - 128, c) if signed else c
    e, f = torch.floor(c / 8), c % 8
    x = torch.where(e > 0, (8 + f) * 2.0 ** (e - 1), f)  # in units of the smallest step
    lowest = -9.0 if signed else -17.0
    return minus * x * 2.0 ** (scale.double().repeat_interleave(BLOCK)[:c.numel()] - 127 + lowest)


def _exact_code_value(x, signed, bits):
    """x rounded to its block's grid."""
    n = x.numel()
    wide = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    wide[:n] = x.abs()
    top = wide.view(-1, BLOCK).amax(1)
    power = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    # at the border of two powers the storage type decides
    power = torch.where(top.float().double() >= 2.0 ** (power + 1), power + 1, power)
    unit = 2.0 ** (torch.where(top > 0, power - (7 if signed else 15), -126.0).clamp(min=-126.0))
    unit = unit.repeat_interleave(BLOCK)[:n]
    y = x.abs() / unit
    first = -6.0 if signed else -14.0
    e = torch.floor(torch.log2(torch.where(y > 0, y, 1.0))).clamp(min=first)
    e = torch.where(y > 0, e, first)
    grid = 2.0 ** (e - 3)
    if bits is None:
        q = torch.round(y / grid) * grid
    else:
        q = torch.floor(y / grid + (bits.double() * 16 + 8) / 2.0 ** 20) * grid
    if not signed:
        q = torch.where((x > 0) & (q == 0), 2.0 ** -17, q)
    return torch.sign(x) * q * unit


def _exact_adamw(case, s):
    sizes = _numbers(case)
    norm = torch.linalg.vector_norm(s["grad"].double())
    by = min(1.0, case["clip"] / float(norm)) if case["clip"] else 1.0
    t, small = s["step"], case["state"] == 8
    p = (s["copy"] if case["master"] else s["param"]).double()
    m = _exact_value(s["m"], s["m_scale"], True) if small else s["m"].double()
    v = _exact_value(s["v"], s["v_scale"], False) if small else s["v"].double()
    g = s["grad"].double() * by
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** t)) / (
        torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out = {"param": p, "m": m, "v": v}
    by_chance = s["seed"] is not None
    if small or by_chance and case["p"] == "bf16" and not case["master"]:
        total = p.numel()
        r = None
        if by_chance:
            r = [torch.zeros(total, dtype=torch.int32, device=p.device) for _ in range(3)]
            for k, parts in enumerate(zip(*(_views(x, sizes) for x in r))):
                got = _chance(sizes[k], _keys(s["seed"], t, k), p.device)
                for x, y in zip(parts, got):
                    x.copy_(y)
        if small:
            out["m"] = _exact_code_value(m, True, r[0] if by_chance else None)
            out["v"] = _exact_code_value(v, False, r[1] if by_chance else None)
        if by_chance and case["p"] == "bf16" and not case["master"]:
            e = torch.floor(torch.log2(torch.where(p != 0, p.abs(), 1.0)))
            ulp = 2.0 ** (e - 7)
            q = torch.floor(p.abs() / ulp + r[2].double() / 65536) * ulp
            out["param"] = torch.sign(p) * q
    if case["master"]:
        out["copy"] = p
    if case["clip"]:
        out["norm"] = norm.reshape(1)
    return out
