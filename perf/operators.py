"""Measured cases of the operators on whole vocabulary rows: sampling and distillation.

sample: one token of every logit row, from a given uniform number, after
    temperature, top-k, top-p and min-p.
distill / distill_forward / distill_backward: the Kullback-Leibler loss of the
    student's rows against a teacher's top-K logits, and its gradient: both in
    one call (what a training step makes), the loss alone (evaluation), and the
    gradient alone from a given upstream gradient.

Every case names the operator, the input type, the rows, the vocabulary width V
and the padding of a row (`pad` more elements between the starts of two rows).
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634
SCALE = float(1 << 40)  # the sampling weights are whole multiples of 2^-40


def listed():
    """The cases that are always measured, small to large."""
    return [
        # one decode step of one request, fp32 logits, nucleus sampling: latency counts
        _sample("sample_token_1x151936_f32", "f32", 1, 151936, top_p=0.95),
        # the positions of one draft block, with the settings that the draft head's
        # own end-to-end runs use (temperature 1, top-k 20, top-p 0.95)
        _sample("sample_block_16x151936", "bf16", 16, 151936, top_k=20, top_p=0.95),
        # a serving batch: every request has its own settings, rows of an odd width in a
        # padded buffer, some vocabulary entries masked away by a grammar
        _sample("sample_serving_256x151935", "bf16", 256, 151935, pad=1, mixed=True, masked=True),
        # long nucleus sampling over the widest vocabulary, fp32
        _sample("sample_nucleus_512x262144_f32", "f32", 512, 262144, top_p=0.95, min_p=0.0001),
        # every position of the batched verification regime, plain temperature sampling
        _sample("sample_verify_4096x151936", "bf16", 4096, 151936, temperature=0.8),
        # the smallest training step: the tiny fp32 configuration
        _distill("distill_tiny_8x1000_f32", "distill", "f32", 8, 1000, K=4),
        # the evaluation loss of one draft block
        _distill("distill_eval_16x151936", "distill_forward", "bf16", 16, 151936, K=16),
        # the evaluation loss of a set of wide fp32 rows
        _distill("distill_eval_512x262144_f32", "distill_forward", "f32", 512, 262144, K=64),
        # a training step on ragged rows: odd width, padded buffer, masked positions
        _distill("distill_ragged_333x50021", "distill", "bf16", 333, 50021, pad=3, K=33,
                 weighted=True, temperature=2.0),
        # the gradient alone on fp32 rows of an odd width
        _distill("distill_grad_128x4099_f32", "distill_backward", "f32", 128, 4099, K=16),
        # the gradient alone, an ordinary micro-batch
        _distill("distill_grad_1024x151936", "distill_backward", "bf16", 1024, 151936, K=16,
                 weighted=True),
        # a training step over the batched regime's positions, position weights
        _distill("distill_train_4096x151936", "distill", "bf16", 4096, 151936, K=64,
                 weighted=True),
    ]


def _sample(name, dtype, rows, V, pad=0, mixed=False, masked=False, temperature=1.0, top_k=0,
            top_p=1.0, min_p=0.0):
    return {"name": name, "op": "sample", "dtype": dtype, "rows": rows, "V": V, "pad": pad,
            "mixed": mixed, "masked": masked, "temperature": temperature, "top_k": top_k,
            "top_p": top_p, "min_p": min_p}


def _distill(name, op, dtype, rows, V, pad=0, K=16, weighted=False, temperature=1.0):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "V": V, "pad": pad, "K": K,
            "weighted": weighted, "temperature": temperature}


def draw(rng):
    """One more case: 1 to 4096 rows, 512 to 262144 entries, both types, any settings."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["sample", "sample", "distill", "distill_forward", "distill_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = spread(512, 262144)
    V = V // 64 * 64 if rng.random() < 0.5 else V
    rows = min(spread(1, 4096), 4096 * 151936 * 2 // (V * (4 if dtype == "f32" else 2)))
    pad = rng.choice([0, 0, 1, 7, 64])
    if op == "sample":
        c = _sample("", dtype, rows, V, pad, mixed=rng.random() < 0.4, masked=rng.random() < 0.3,
                    temperature=rng.choice([0.0, 0.6, 0.8, 1.0, 1.0, 1.3]),
                    top_k=rng.choice([0, 0, 1, 20, 50, spread(2, 2000)]),
                    top_p=rng.choice([1.0, 1.0, 0.95, 0.9, round(rng.uniform(0.1, 0.99), 3)]),
                    min_p=rng.choice([0.0, 0.0, 0.05, round(rng.uniform(0.001, 0.3), 4)]))
    else:
        c = _distill("", op, dtype, rows, V, pad, K=min(V, spread(1, 256)),
                     weighted=rng.random() < 0.5, temperature=rng.choice([1.0, 1.0, 0.5, 2.0]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def _rows(case, g):
    """Logit rows: a normal bulk and, in every row, 64 tokens that stand out by an
    amount that falls off with their rank; 0 (a flat row) to 18 (a sure one) at the top."""
    rows, V, dev = case["rows"], case["V"], "cuda"
    x = torch.randn((rows, V), device=dev, generator=g) * 2.0
    top = torch.rand((rows, 1), device=dev, generator=g) * 18.0
    fall = torch.exp(-torch.arange(64, device=dev, dtype=torch.float32) / 6.0)
    ids = torch.randint(0, V, (rows, 64), device=dev, generator=g)
    # an id drawn twice counts once, so that the sum below has one order
    ids = torch.sort(ids, dim=1)[0]
    fresh = torch.ones_like(ids, dtype=torch.bool)
    fresh[:, 1:] = ids[:, 1:] != ids[:, :-1]
    order = torch.argsort(torch.rand((rows, 64), device=dev, generator=g), dim=1)
    x.scatter_add_(1, ids, top * fall[order] * fresh)
    return x


def _stored(x, case):
    """x in the case's type, in a buffer whose rows are V + pad elements apart."""
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    buf = torch.zeros((case["rows"], case["V"] + case["pad"]), dtype=dt, device=x.device)
    buf[:, :case["V"]] = x
    return buf[:, :case["V"]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows, V, dev = case["rows"], case["V"], "cuda"
    x = _rows(case, g)
    s = {"case": dict(case)}
    if case["op"] == "sample":
        if case["masked"]:  # every fourth row allows one entry in 16, the last row none at all
            gone = torch.rand((rows, V), device=dev, generator=g) >= 1.0 / 16
            gone &= (torch.arange(rows, device=dev) % 4 == 1)[:, None]
            if rows > 1:
                gone[-1] = True
            x.masked_fill_(gone, float("-inf"))
        s["logits"] = _stored(x, case)
        s["u"] = torch.rand((rows,), device=dev, generator=g)

        def pick(values, dtype):
            at = torch.randint(0, len(values), (rows,), device=dev, generator=g)
            return torch.tensor(values, dtype=dtype, device=dev)[at]

        if case["mixed"]:
            s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3], torch.float32)
            s["top_k"] = pick([0, 0, 1, 20, 50, 200], torch.int32)
            s["top_p"] = pick([1.0, 0.95, 0.9, 0.5], torch.float32)
            s["min_p"] = pick([0.0, 0.0, 0.05, 0.1], torch.float32)
        else:
            for k in ("temperature", "top_k", "top_p", "min_p"):
                s[k] = case[k]
        return s
    s["logits"] = _stored(x, case)
    # the teacher agrees with the student in part; its K largest entries, largest first
    y = x.mul_(0.8).add_(torch.randn((rows, V), device=dev, generator=g), alpha=1.5)
    val, ids = torch.topk(y, case["K"], dim=1)
    s["ids"], s["teacher"] = ids.to(torch.int32).contiguous(), val.contiguous()
    s["weight"] = None
    if case["weighted"]:  # blocks of 16 positions, later ones count less, the last two are padding
        at = torch.arange(rows, device=dev) % 16
        s["weight"] = torch.where(at < 14, 0.9 ** at.float(), 0.0)
    if case["op"] == "distill_backward":
        s["grad_loss"] = (0.5 + torch.rand((rows,), device=dev, generator=g)) / rows
        z = s["logits"].float() * (1.0 / case["temperature"])
        m = z.amax(1, keepdim=True)
        s["lse"] = (m + torch.log(torch.exp(z - m).sum(1, keepdim=True))).squeeze(1)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    c = s["case"]
    if own:
        import dflash2_draft_head_gb300 as df2
        if c["op"] == "sample":
            tokens, probs = df2.sample(s["logits"], s["u"], temperature=s["temperature"],
                                       top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
            return {"tokens": tokens, "probs": probs}
        if c["op"] == "distill_backward":
            return {"grad": df2.distill_backward(s["grad_loss"], s["logits"], s["ids"],
                                                 s["teacher"], s["lse"],
                                                 temperature=c["temperature"],
                                                 weight=s["weight"])}
        loss, lse, grad = df2.distill(s["logits"], s["ids"], s["teacher"],
                                      temperature=c["temperature"], weight=s["weight"],
                                      grad=c["op"] == "distill")
        return {"loss": loss, "lse": lse} | ({"grad": grad} if c["op"] == "distill" else {})
    if c["op"] == "sample":
        return _plain_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"],
                             s["min_p"])
    return _plain_distill(s, c)


def _per_row(v, rows, dtype, dev):
    if isinstance(v, torch.Tensor):
        return v[:, None]
    return torch.full((rows, 1), v, dtype=dtype, device=dev)


def _plain_sample(logits, u, temperature, top_k, top_p, min_p):
    """The sampling rule in torch operations.

    Weights: w = 2^((x - max) * (log2(e) / T)) in fp32, taken as the whole number
    W = round(w * 2^40), so that every sum below is exact whatever its order.  A
    temperature of 0 keeps the largest entry alone.  In order of falling logit (ties:
    lowest index first) an entry is kept while fewer than top_k stand before it,
    the weights before it are below top_p of the top_k entries' sum, and w >= min_p.
    The token is the first one, in order of index, at which the running sum of the
    kept weights passes u times their sum."""
    rows, V = logits.shape
    dev = logits.device
    T = _per_row(temperature, rows, torch.float32, dev)
    k = _per_row(top_k, rows, torch.int32, dev).long()
    p = _per_row(top_p, rows, torch.float32, dev)
    mp = _per_row(min_p, rows, torch.float32, dev)
    k = torch.where(T > 0, torch.where(k <= 0, V, k), 1)
    c = torch.full_like(T, LOG2E) / torch.where(T > 0, T, 1.0)
    x = logits.float()
    m = x.amax(1, keepdim=True)
    w = torch.exp2(torch.where(x == m, 0.0, (x - m) * c))
    W = torch.where(x > float("-inf"), torch.round(w * SCALE), 0.0).long()
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    sw, sW = w.gather(1, order), W.gather(1, order)
    rank = torch.arange(V, device=dev)[None, :]
    keep = rank < k
    sW = sW * keep
    total = sW.sum(1, keepdim=True)
    before = torch.cumsum(sW, 1) - sW
    keep &= ((before.double() < p.double() * total.double()) | (p >= 1) | (rank == 0))
    keep &= (sw >= mp) | (rank == 0)
    kept = torch.zeros_like(W).scatter_(1, order, sW * keep)
    cum = torch.cumsum(kept, 1)
    total = cum[:, -1:]
    t = torch.minimum((u[:, None].double() * total.double()).long(), total - 1)
    at = (cum <= t).sum(1, keepdim=True)
    some = total > 0
    prob = kept.gather(1, torch.where(some, at, 0)).double() / total.clamp(min=1).double()
    return {"tokens": torch.where(some, at, -1).squeeze(1).to(torch.int32),
            "probs": torch.where(some, prob, 0.0).squeeze(1).float()}


def _plain_distill(s, c):
    """loss[r] = weight[r] * sum_k q_k * (log q_k - (z_k / T - lse)), q the softmax of the
    teacher's K logits over T; d loss[r] / d z_j = weight[r] * (softmax(z/T)_j - q_j) / T."""
    ids, inv = s["ids"].long(), 1.0 / c["temperature"]
    z = s["logits"].float() * inv
    y = s["teacher"] * inv
    e = torch.exp(y - y.amax(1, keepdim=True))
    q = e / e.sum(1, keepdim=True)
    weight = 1.0 if s["weight"] is None else s["weight"]
    out = {}
    if c["op"] == "distill_backward":
        lse, scale = s["lse"], s["grad_loss"] * weight * inv
    else:
        m = z.amax(1)
        lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
        out["loss"] = weight * (q * (torch.log(q) - z.gather(1, ids) + lse[:, None])).sum(1)
        out["lse"] = lse if s["weight"] is None else torch.where(weight != 0, lse, 0.0)
        if c["op"] == "distill_forward":
            return out
        scale = torch.full_like(lse, inv) * weight
    g = torch.exp(z - lse[:, None])
    g.scatter_add_(1, ids, -q)
    out["grad"] = (g * scale[:, None]).to(s["logits"].dtype)
    return out


# ------------------------------------------------------------------ what a pass needs


def work(case):
    rows, V = case["rows"], case["V"]
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "sample":  # the rows, u and the settings in; a token and its share out
        return {"bytes": rows * V * es + rows * (4 + 8 + (16 if case["mixed"] else 0)),
                "flops": 5 * rows * V}
    live = sum(1 for r in range(rows) if r % 16 < 14) if case["weighted"] else rows
    small = rows * (case["K"] * 8 + 8 + (4 if case["weighted"] else 0))
    if case["op"] == "distill_forward":
        return {"bytes": live * V * es + small, "flops": 4 * live * V}
    flops = (7 if case["op"] == "distill" else 4) * live * V
    return {"bytes": (live + rows) * V * es + small, "flops": flops}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The same outputs in 64 bits, row block by row block.  A token has no such value; its
    share is that of the token that the rule picks in 64 bits."""
    s = prepare(case, seed)
    rows, V = case["rows"], case["V"]
    step = max(1, (1 << 26) // V)
    parts = []
    for lo in range(0, rows, step):
        hi = min(rows, lo + step)
        z = s["logits"][lo:hi].double()

        def at(name):
            v = s.get(name)
            return v[lo:hi] if isinstance(v, torch.Tensor) else v

        if case["op"] == "sample":
            parts.append(_exact_sample(z, at("u").double(), at("temperature"), at("top_k"),
                                       at("top_p"), at("min_p")))
        else:
            parts.append(_exact_distill(case, z, at("ids").long(), at("teacher").double(),
                                        at("weight"), at("grad_loss"), at("lse")))
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["op"] == "sample":
        out["tokens"] = None
    return out


def _exact_sample(z, u, temperature, top_k, top_p, min_p):
    n, V = z.shape

    def col(v):
        v = v if isinstance(v, torch.Tensor) else torch.full((n,), v, device=z.device)
        return v.double().unsqueeze(1)

    T, k, p, mp = col(temperature), col(top_k), col(top_p), col(min_p)
    greedy = T <= 0
    v, order = torch.sort(z, dim=1, descending=True, stable=True)
    top = v[:, :1]
    r = torch.exp((v - torch.where(torch.isinf(top), 0.0, top)) / torch.where(greedy, 1.0, T))
    place = torch.arange(V, device=z.device, dtype=torch.float64).expand(n, V)
    limit = torch.where(greedy, 1.0, torch.where(k < 1, float(V), k))
    r = torch.where(place < limit, r, 0.0)
    run_sum = r.cumsum(1)
    inside = (run_sum - r < p * run_sum[:, -1:]) | (p >= 1)
    cut = torch.where((inside & (r >= mp)) | (place == 0), r, 0.0)
    share = torch.zeros_like(cut).scatter_(1, order, cut)
    share = share / share.sum(1, keepdim=True)
    pick = torch.searchsorted(share.cumsum(1).contiguous(), u.unsqueeze(1).contiguous(), right=True)
    got = share.gather(1, pick.clamp(max=V - 1)).squeeze(1)
    return {"probs": torch.where(torch.isfinite(top.squeeze(1)), got, 0.0)}


def _exact_distill(case, z, ids, teacher, weight, grad_loss, lse):
    T = case["temperature"]
    logq = torch.log_softmax(teacher / T, dim=1)
    q = torch.exp(logq)
    n = z.shape[0]
    w = torch.ones(n, device=z.device).double() if weight is None else weight.double()
    norm = lse.double() if case["op"] == "distill_backward" else torch.logsumexp(z / T, dim=1)
    logp = z / T - norm.unsqueeze(1)
    out = {}
    if case["op"] != "distill_backward":
        out["loss"] = w * (q * (logq - logp.gather(1, ids))).sum(1)
        out["lse"] = torch.where(w != 0, norm, 0.0)
        if case["op"] == "distill_forward":
            return out
    up = w / T if grad_loss is None else grad_loss.double() * w / T
    diff = torch.exp(logp)
    diff.scatter_(1, ids, diff.gather(1, ids) - q)  # the teacher's ids are distinct
    out["grad"] = diff * up.unsqueeze(1)
    return out
