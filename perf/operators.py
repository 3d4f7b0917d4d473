"""Cases of the training objectives over rows of scores.

Four operators, each with its gradient:

* ``logp``: the log-probability of one label a row under a row of logits, and the gradient that
  a given gradient of it makes in the logits.
* ``policy``: a clipped policy loss with a KL term to a reference, over rows of logits.
* ``pref``: a preference loss over pairs of token sequences laid end to end.
* ``balance``: a router's top-k choice, its balance loss and per-expert counts.
"""
import math
import random

import torch

#: False: the operators in elementary torch operations; True: this repository's own calls.
own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
#: The most bytes of logits that a drawn case has: those of the largest listed one.
MOST = 8192 * 131072 * 2


def listed():
    return [
        # The token that a decoding step has just drawn, scored for the log of probabilities.
        {"name": "logp token", "op": "logp", "rows": 1, "n": 131072, "dtype": "bf16", "pad": 0,
         "ignored": 0.0, "closed": 0.0, "temperature": 1.0, "grad": False},
        # A reference model's scores of a batch of answers; a quarter of the rows are prompts.
        {"name": "logp score", "op": "logp", "rows": 4096, "n": 65536, "dtype": "bf16", "pad": 0,
         "ignored": 0.25, "closed": 0.01, "temperature": 1.0, "grad": False},
        # A supervised step in float32 on an odd vocabulary, stored in rows padded to 64.
        {"name": "logp train", "op": "logp", "rows": 1537, "n": 32003, "dtype": "f32", "pad": 61,
         "ignored": 0.1, "closed": 0.0, "temperature": 1.0, "grad": True},
        # A few rows of a small vocabulary in float16 with a scaled loss: latency counts.
        {"name": "policy small", "op": "policy", "rows": 96, "n": 8192, "dtype": "f16", "pad": 0,
         "ignored": 0.2, "closed": 0.0, "temperature": 1.0, "kl": 0.04, "scale": 4096.0},
        # An odd vocabulary with no padding (no row but the first aligned) at a sampling temperature.
        {"name": "policy odd", "op": "policy", "rows": 2047, "n": 50021, "dtype": "bf16", "pad": 0,
         "ignored": 0.15, "closed": 0.0, "temperature": 0.7, "kl": 0.05, "scale": 1.0},
        # A full micro-batch of answers on a large vocabulary, its last columns closed.
        {"name": "policy large", "op": "policy", "rows": 8192, "n": 131072, "dtype": "bf16", "pad": 0,
         "ignored": 0.3, "closed": 0.01, "temperature": 1.0, "kl": 0.02, "scale": 1.0},
        # Four short pairs in float32, a hinge on mean log-probabilities.
        {"name": "pref small", "op": "pref", "pairs": 4, "longest": 24, "n": 4096, "dtype": "f32",
         "pad": 0, "prompt": 0.2, "kind": "hinge", "average": True, "smooth": 0.0},
        # Ragged pairs on an odd vocabulary, prompts of nearly half of their tokens.
        {"name": "pref odd", "op": "pref", "pairs": 16, "longest": 201, "n": 32771, "dtype": "bf16",
         "pad": 0, "prompt": 0.4, "kind": "sigmoid", "average": False, "smooth": 0.0},
        # Long answers on a large vocabulary, with smoothed preferences.
        {"name": "pref large", "op": "pref", "pairs": 8, "longest": 512, "n": 131072, "dtype": "bf16",
         "pad": 0, "prompt": 0.25, "kind": "sigmoid", "average": False, "smooth": 0.1},
        # A decoding step's tokens at a router of 64 experts.
        {"name": "balance step", "op": "balance", "rows": 8, "n": 64, "dtype": "f32", "top_k": 2,
         "masked": 0.0, "closed": 0, "renormalize": False},
        # A sequence at a router of 128 experts, padding tokens masked, gates renormalised.
        {"name": "balance sequence", "op": "balance", "rows": 16384, "n": 128, "dtype": "bf16", "top_k": 8,
         "masked": 0.1, "closed": 0, "renormalize": True},
        # A whole batch at a router of 256 experts, three of them closed.
        {"name": "balance batch", "op": "balance", "rows": 131072, "n": 256, "dtype": "f32", "top_k": 8,
         "masked": 0.05, "closed": 3, "renormalize": False},
    ]


def spread(rng, low, high):
    """A whole number of low..high, even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["logp", "policy", "pref", "balance"])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    if op == "balance":
        n = spread(rng, 4, 512)
        return {"op": op, "rows": spread(rng, 1, 131072 * 256 * 4 // (n * SIZE[dtype])), "n": n, "dtype": dtype,
                "top_k": min(n, rng.choice([1, 2, 4, 6, 8])), "masked": rng.choice([0.0, 0.1, 0.5]),
                "closed": rng.choice([0, 0, n // 16]), "renormalize": rng.random() < 0.5}
    n = spread(rng, 300, 200003)
    pad = rng.choice([0, 0, -n % 64, rng.randrange(1, 64)])
    most = max(1, MOST // ((n + pad) * SIZE[dtype]))
    if op == "pref":
        pairs = spread(rng, 1, min(64, max(1, most // 4)))
        return {"op": op, "pairs": pairs, "longest": spread(rng, 1, max(1, min(1024, most // (2 * pairs)))), "n": n,
                "dtype": dtype, "pad": pad, "prompt": rng.uniform(0.0, 0.6), "kind": rng.choice(["sigmoid", "hinge", "squared"]),
                "average": rng.random() < 0.4, "smooth": rng.choice([0.0, 0.1])}
    case = {"op": op, "rows": spread(rng, 1, min(16384, most)), "n": n, "dtype": dtype, "pad": pad,
            "ignored": rng.choice([0.0, 0.1, 0.4]), "closed": rng.choice([0.0, 0.02]),
            "temperature": rng.choice([1.0, 1.0, 0.8])}
    if op == "logp":
        case["grad"] = rng.random() < 0.6
    else:
        case["kl"] = rng.choice([0.0, 0.05])
        case["scale"] = 4096.0 if dtype == "f16" else 1.0
    return case


def lengths(case):
    """The tokens of each sequence of a preference case, the chosen and the rejected of a pair in turn."""
    rng = random.Random(case["pairs"] * 1009 + case["longest"])
    return [rng.randint((case["longest"] + 1) // 2, case["longest"]) for _ in range(2 * case["pairs"])]


def prompts(case):
    """The leading tokens of each sequence that carry no label."""
    return [int(case["prompt"] * size) for size in lengths(case)]


def unlabelled(case):
    return int(case["ignored"] * case["rows"])


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def make_logits(case, rows, g):
    """Rows of a model's scores: a wide bulk and a few likely entries; the last columns closed with -inf."""
    n, dtype = case["n"], TYPES[case["dtype"]]
    x = torch.randn((rows, n + case.get("pad", 0)), generator=g, device="cuda", dtype=dtype).mul_(2.0)
    shut = int(n * case.get("closed", 0.0))
    x = x[:, :n]
    if shut:
        x[:, n - shut:] = -math.inf
    labels = torch.randint(0, n - shut, (rows,), generator=g, device="cuda")
    lift = 8.0 + 2.5 * torch.randn((rows,), generator=g, device="cuda")
    x[torch.arange(rows, device="cuda"), labels] = lift.to(dtype)
    return x, labels


def make_logp(x, labels, temperature):
    """The labels' log-probabilities, a block of rows at a time."""
    got = []
    for at in range(0, x.shape[0], 512):
        y = x[at:at + 512].float() / temperature
        got.append(y.gather(1, labels[at:at + 512, None])[:, 0] - torch.logsumexp(y, 1))
    return torch.cat(got)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op == "balance":
        rows, n = case["rows"], case["n"]
        x = normal(rows, n) + 0.7 * normal(1, n)
        if case["closed"]:
            x[:, torch.randperm(n, generator=g, device="cuda")[:case["closed"]]] = -math.inf
        s["logits"] = x.to(TYPES[case["dtype"]])
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.rand((rows,), generator=g, device="cuda") >= case["masked"]
        s["grad_gates"] = normal(rows, case["top_k"]) / rows
        s["grad_loss"] = 0.01
        return s
    if op == "pref":
        sizes = lengths(case)
        rows = sum(sizes)
        x, labels = make_logits(case, rows, g)
        offsets = [0]
        for size in sizes:
            offsets.append(offsets[-1] + size)
        quiet = torch.zeros(rows, dtype=torch.bool)
        for at, size in zip(offsets, prompts(case)):
            quiet[at:at + size] = True
        # What the reference model gave each token: near the policy, as it is early in training.
        s["ref"] = make_logp(x, labels, 1.0) + (1.0 if case["average"] else 0.15) * normal(rows)
        labels[quiet.cuda()] = -100
        s["logits"], s["labels"] = x, labels
        s["offsets"] = torch.tensor(offsets, device="cuda")
        s["beta"] = 2.0 if case["average"] else 0.1
        return s
    x, labels = make_logits(case, case["rows"], g)
    rows = case["rows"]
    if op == "policy":
        lp = make_logp(x, labels, case["temperature"])
        move = 0.2 * normal(rows)
        # The derivative jumps where the ratio meets a bound of the clip; no row is put within rounding of one.
        for edge in (math.log(0.8), math.log(1.28)):
            move = torch.where((move - edge).abs() < 1e-4, move + 1e-3, move)
        s["old"] = lp - move
        s["advantages"] = normal(rows)
        s["ref"] = lp + 0.3 * normal(rows) if case["kl"] else None
        s["low"], s["high"] = 0.2, 0.28
    elif case["grad"]:
        s["grad"] = -torch.rand((rows,), generator=g, device="cuda") / rows
        if case["dtype"] == "f16":
            s["grad"] = s["grad"] * 4096.0
    labels[torch.randperm(rows, generator=g, device="cuda")[:unlabelled(case)]] = -100
    s["logits"], s["labels"] = x, labels
    return s


# ---------------------------------------------------------------------------
# This repository's calls
# ---------------------------------------------------------------------------
def own_run(s):
    from convex_hull_pava_gb300 import objectives

    case, op = s["case"], s["case"]["op"]
    if op == "logp":
        logp, norm, _ = objectives.iso_token_logp(s["logits"], s["labels"], temperature=case["temperature"])
        if not case["grad"]:
            return {"logp": logp}
        return {"logp": logp, "dlogits": objectives.iso_token_logp_backward(
            s["grad"], s["logits"], s["labels"], norm, temperature=case["temperature"])}
    if op == "policy":
        r = objectives.iso_policy_loss(
            s["logits"], s["labels"], s["old"], s["advantages"], s["ref"], clip_low=s["low"], clip_high=s["high"],
            kl_coef=case["kl"], temperature=case["temperature"], grad_scale=case["scale"])
        return {"loss": r.loss, "stats": r.stats, "logp": r.logp, "dlogits": r.dlogits}
    if op == "pref":
        r = objectives.iso_preference_loss(
            s["logits"], s["labels"], s["offsets"], s["ref"], kind=case["kind"], beta=s["beta"],
            label_smoothing=case["smooth"], average=case["average"])
        return {"loss": r.loss, "margins": r.margins, "seq_logp": r.seq_logp, "dlogits": r.dlogits}
    r = objectives.iso_balance_loss(s["logits"], case["top_k"], s["mask"], renormalize=case["renormalize"])
    dlogits = objectives.iso_balance_loss_backward(s["logits"], r, grad_loss=s["grad_loss"], grad_gates=s["grad_gates"])
    return {"loss": r.loss, "counts": r.counts, "experts": r.experts, "gates": r.gates, "dlogits": dlogits}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def plain_logp(logits, labels, temperature):
    """(log-probabilities, with 0 at unlabelled rows; probabilities)"""
    x = logits.float() / temperature
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    at = labels.clamp(min=0)[:, None]
    logp = (x.gather(1, at) - torch.log(total))[:, 0]
    return torch.where(labels >= 0, logp, 0.0), e.div_(total)


def plain_grad(coef, p, labels, temperature, dtype):
    """coef (onehot - p) / temperature, with 0 at unlabelled rows."""
    coef = torch.where(labels >= 0, coef, 0.0)[:, None] / temperature
    d = p.mul_(-coef)
    at = labels.clamp(min=0)[:, None]
    d.scatter_(1, at, d.gather(1, at) + coef)
    return d.to(dtype)


def plain_policy(s):
    case = s["case"]
    logp, p = plain_logp(s["logits"], s["labels"], case["temperature"])
    live = (s["labels"] >= 0).float()
    w = live / live.sum().clamp(min=1.0)
    ratio = torch.exp(logp - s["old"])
    free = -s["advantages"] * ratio
    held = -s["advantages"] * ratio.clamp(1.0 - s["low"], 1.0 + s["high"])
    cut = (held > free).float()
    coef = w * free * (1.0 - cut)
    stats = [(w * torch.maximum(free, held)).sum(), torch.zeros((), device="cuda"), (w * cut).sum()]
    if s["ref"] is not None:
        d = s["ref"] - logp
        stats[1] = (w * (torch.expm1(d) - d)).sum()
        coef = coef - case["kl"] * w * torch.expm1(d)
    return {"loss": stats[0] + case["kl"] * stats[1], "stats": torch.stack(stats), "logp": logp,
            "dlogits": plain_grad(coef * case["scale"], p, s["labels"], case["temperature"], s["logits"].dtype)}


def plain_pref(s):
    case, offsets = s["case"], s["offsets"]
    logp, p = plain_logp(s["logits"], s["labels"], 1.0)
    at = torch.arange(logp.shape[0], device="cuda")
    inside = ((at >= offsets[:-1, None]) & (at < offsets[1:, None])).float()
    share = inside * (s["labels"] >= 0)
    if case["average"]:
        share = share / share.sum(1, keepdim=True).clamp(min=1.0)
    seq = (share * logp).sum(1)
    gain = (share * (logp - s["ref"])).sum(1).view(-1, 2)
    h = gain[:, 0] - gain[:, 1]
    beta, smooth = s["beta"], case["smooth"]
    margins = beta * h
    if case["kind"] == "sigmoid":
        over = torch.log1p(torch.exp(-margins.abs()))
        each = (1 - smooth) * (over + (-margins).clamp(min=0)) + smooth * (over + margins.clamp(min=0))
        slope = beta * (smooth / (1.0 + torch.exp(-margins)) - (1 - smooth) / (1.0 + torch.exp(margins)))
    elif case["kind"] == "hinge":
        each = (1.0 - margins).clamp(min=0)
        slope = -beta * (margins < 1.0).float()
    else:
        each = (h - 0.5 / beta) ** 2
        slope = 2.0 * (h - 0.5 / beta)
    slope = slope / margins.shape[0]
    coef = (torch.stack([slope, -slope], 1).view(-1, 1) * share).sum(0)
    return {"loss": each.mean(), "margins": margins, "seq_logp": seq,
            "dlogits": plain_grad(coef, p, s["labels"], 1.0, s["logits"].dtype)}


def plain_balance(s):
    case = s["case"]
    x, k, n = s["logits"].float(), case["top_k"], case["n"]
    rows = x.shape[0]
    live = torch.ones(rows, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    live = live & (x > -math.inf).any(1)
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    chosen = (value[:, :k] > -math.inf) & live[:, None]
    experts = torch.where(chosen, order[:, :k], -1)
    counts = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    counts = counts.scatter_add_(0, (experts + 1).reshape(-1), torch.ones_like(experts).reshape(-1))[1:]
    top = torch.where(live[:, None], value[:, :1], 0.0)
    e = torch.where(live[:, None], torch.exp(x - top), 0.0)
    p = e / torch.where(live, e.sum(1), 1.0)[:, None]
    tokens = live.sum().clamp(min=1).float()
    loss = n / (k * tokens * tokens) * (counts.float() * p.sum(0)).sum()
    at = experts.clamp(min=0).long()
    gates = torch.where(chosen, p.gather(1, at), 0.0)
    g = torch.where(chosen, s["grad_gates"], 0.0)
    u = (s["grad_loss"] * n / (k * tokens * tokens)) * counts.float()[None, :]
    if case["renormalize"]:
        gates = gates / torch.where(live, gates.sum(1), 1.0)[:, None]
        extra = gates * (g - (gates * g).sum(1, keepdim=True))
        d = p * (u - (p * u).sum(1, keepdim=True))
        d = d.scatter_add_(1, at, extra)
    else:
        u = u.expand(rows, n).scatter_add(1, at, g)
        d = p * (u - (p * u).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts, "experts": experts.to(torch.int32), "gates": gates,
            "dlogits": d.to(s["logits"].dtype)}


def plain_run(s):
    case = s["case"]
    if case["op"] == "policy":
        return plain_policy(s)
    if case["op"] == "pref":
        return plain_pref(s)
    if case["op"] == "balance":
        return plain_balance(s)
    if not case["grad"]:
        return {"logp": plain_logp(s["logits"], s["labels"], case["temperature"])[0]}
    logp, p = plain_logp(s["logits"], s["labels"], case["temperature"])
    return {"logp": logp, "dlogits": plain_grad(s["grad"], p, s["labels"], case["temperature"], s["logits"].dtype)}


def run(state):
    return own_run(state) if own else plain_run(state)


def work(case):
    b, n = SIZE[case["dtype"]], case["n"]
    if case["op"] == "balance":
        rows, k = case["rows"], case["top_k"]
        return {"bytes": 2 * rows * n * b + rows * k * 12 + n * 8 + (rows if case["masked"] else 0),
                "flops": rows * n * (12 + k)}
    if case["op"] == "pref":
        rows, live = sum(lengths(case)), sum(lengths(case)) - sum(prompts(case))
        return {"bytes": (live + rows) * n * b + rows * 12 + case["pairs"] * 28, "flops": 8 * live * n}
    rows = case["rows"]
    live = rows - unlabelled(case)
    if case["op"] == "policy":
        return {"bytes": (live + rows) * n * b + rows * (24 if case["kl"] else 20), "flops": 8 * live * n}
    if case["grad"]:
        return {"bytes": (live + rows) * n * b + rows * 16, "flops": 8 * live * n}
    return {"bytes": live * n * b + rows * 12, "flops": 4 * live * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits; the gradients by differentiating them
# ---------------------------------------------------------------------------
def exact_logp(logits, labels, temperature):
    x = logits.double().requires_grad_()
    nll = torch.nn.functional.nll_loss(torch.log_softmax(x / temperature, 1), labels, ignore_index=-100, reduction="none")
    return x, -nll


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return exact_balance(s)
    x, lp = exact_logp(s["logits"], s["labels"], case.get("temperature", 1.0))
    if case["op"] == "logp":
        if not case["grad"]:
            return {"logp": lp.detach()}
        return {"logp": lp.detach(), "dlogits": torch.autograd.grad(lp, x, s["grad"].double())[0]}
    if case["op"] == "policy":
        live = s["labels"] != -100
        if not bool(live.any()):
            return None
        a, new, old = s["advantages"].double()[live], lp[live], s["old"].double()[live]
        ratio = (new - old).exp()
        inner = torch.minimum(a * ratio, a * torch.clamp(ratio, 1 - s["low"], 1 + s["high"]))
        kl = torch.zeros_like(new)
        if s["ref"] is not None:
            kl = torch.exp(s["ref"].double()[live] - new) - 1 + (new - s["ref"].double()[live])
        loss = -inner.mean() + case["kl"] * kl.mean()
        cut = (inner < a * ratio).double().mean()
        d = torch.autograd.grad(loss * case["scale"], x)[0]
        return {"loss": loss.detach(), "stats": torch.stack([-inner.mean(), kl.mean(), cut]).detach(), "logp": lp.detach(),
                "dlogits": d}
    seq, reward = [], []
    ends = s["offsets"].tolist()
    for a, b in zip(ends, ends[1:]):
        live = s["labels"][a:b] != -100
        size = max(1, int(live.sum())) if case["average"] else 1
        seq.append(lp[a:b][live].sum() / size)
        reward.append(s["beta"] * (seq[-1] - s["ref"][a:b][live].double().sum() / size))
    seq, reward = torch.stack(seq), torch.stack(reward)
    margins = reward[0::2] - reward[1::2]
    if case["kind"] == "sigmoid":
        softplus = torch.nn.functional.softplus
        each = softplus(-margins) * (1 - case["smooth"]) + softplus(margins) * case["smooth"]
    elif case["kind"] == "hinge":
        each = torch.relu(1 - margins)
    else:
        each = (margins / s["beta"] - 1 / (2 * s["beta"])).square()
    d = torch.autograd.grad(each.mean(), x)[0]
    return {"loss": each.mean().detach(), "margins": margins.detach(), "seq_logp": seq.detach(), "dlogits": d}


def exact_balance(s):
    case = s["case"]
    x = s["logits"].double()
    rows, n, k = x.shape[0], case["n"], case["top_k"]
    live = torch.isfinite(x).any(1) if s["mask"] is None else s["mask"] & torch.isfinite(x).any(1)
    picked = torch.full((rows, k), -1, device=x.device)
    left = x.clone()
    for j in range(k):  # the largest that is left; of equal ones the first
        most = left.amax(1, keepdim=True)
        first = ((left == most) * torch.arange(n, 0, -1, device=x.device)).argmax(1)
        ok = live & (most[:, 0] > -math.inf)
        picked[:, j] = torch.where(ok, first, -1)
        left.scatter_(1, first[:, None], -math.inf)
    hit = picked >= 0
    counts = torch.bincount(picked[hit], minlength=n)
    y = x[live].requires_grad_()
    p = torch.softmax(y, 1)
    tokens = max(1, int(live.sum()))
    loss = n * (counts.double() / (k * tokens) * (p.sum(0) / tokens)).sum()
    gates = p.gather(1, picked[live].clamp(min=0)) * hit[live]
    if case["renormalize"]:
        gates = gates / gates.sum(1, keepdim=True)
    goal = s["grad_loss"] * loss + (gates * s["grad_gates"].double()[live]).sum()
    d = torch.zeros_like(x)
    d[live] = torch.autograd.grad(goal, y)[0]
    whole = torch.zeros((rows, k), dtype=torch.float64, device=x.device)
    whole[live] = gates.detach()
    return {"loss": loss.detach(), "counts": counts, "experts": picked.to(torch.int32), "gates": whole, "dlogits": d}
