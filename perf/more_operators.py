"""Cases of the choices over rows of scores, and of the states that follow them.

Three operators:

* ``route``: a router's choice of experts by softmax or sigmoid scores, with a bias for balance and
  groups of experts, its gates and per-expert counts, and the gradient that one of the gates makes
  in the scores.
* ``beam``: a step of beam search: the best continuations over a batch item's beams and vocabulary.
* ``reorder``: the states of beams put, in place, where their continuations are.
"""
import math

import torch

#: False: the operators in elementary torch operations; True: this repository's own calls.
own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i64": torch.int64}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "i64": 8}
#: The most bytes that a drawn case has: of a router's scores, of logits, of states.
MOST_ROUTE = 131072 * 256 * 4
MOST_BEAM = 64 * 8 * 131072 * 2
MOST_STATE = 16 * 64 * 8 * 1024 * 128 * 2


def listed():
    return [
        # A decoding step's tokens at a router of 64 experts with a balance bias: latency counts.
        {"name": "route step", "op": "route", "rows": 8, "n": 64, "dtype": "f32", "pad": 0, "score": "sigmoid", "bias": True,
         "groups": 1, "top_groups": 1, "best": 1, "top_k": 2, "masked": 0.0, "closed": 0, "renormalize": True, "scale": 1.0, "grad": False},
        # A sequence at a router of 128 experts, padding tokens masked, no groups.
        {"name": "route sequence", "op": "route", "rows": 16384, "n": 128, "dtype": "bf16", "pad": 0, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "best": 1, "top_k": 8, "masked": 0.1, "closed": 0, "renormalize": True, "scale": 1.0, "grad": True},
        # Groups of 20 experts by their best one, in padded rows, an odd number of tokens.
        {"name": "route odd", "op": "route", "rows": 4099, "n": 160, "dtype": "f16", "pad": 7, "score": "softmax", "bias": False,
         "groups": 8, "top_groups": 3, "best": 1, "top_k": 6, "masked": 0.0, "closed": 3, "renormalize": False, "scale": 16.0, "grad": True},
        # Many experts without groups, ten of them a token.
        {"name": "route wide", "op": "route", "rows": 8191, "n": 512, "dtype": "bf16", "pad": 0, "score": "softmax", "bias": True,
         "groups": 1, "top_groups": 1, "best": 1, "top_k": 10, "masked": 0.05, "closed": 0, "renormalize": True, "scale": 1.0, "grad": True},
        # A whole batch at a router of 256 experts: sigmoid scores, a balance bias, 4 of 8 groups by their best two.
        {"name": "route batch", "op": "route", "rows": 131072, "n": 256, "dtype": "f32", "pad": 0, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "best": 2, "top_k": 8, "masked": 0.05, "closed": 0, "renormalize": True, "scale": 2.5, "grad": True},
        # One question's four beams on a large vocabulary: latency counts.
        {"name": "beam token", "op": "beam", "batch": 1, "beams": 4, "n": 131072, "dtype": "bf16", "pad": 0, "keep": 8, "done": 0.0,
         "closed": 0.0, "temperature": 1.0},
        # A few questions in float32 on a small vocabulary, some beams ended, with a temperature.
        {"name": "beam small", "op": "beam", "batch": 8, "beams": 5, "n": 8192, "dtype": "f32", "pad": 0, "keep": 10, "done": 0.2,
         "closed": 0.0, "temperature": 0.7},
        # An odd vocabulary without padding: no row but the first aligned.
        {"name": "beam odd", "op": "beam", "batch": 37, "beams": 6, "n": 50021, "dtype": "bf16", "pad": 0, "keep": 6, "done": 0.1,
         "closed": 0.0, "temperature": 1.0},
        # A batch of answers for preference pairs on a large vocabulary, its last columns closed.
        {"name": "beam large", "op": "beam", "batch": 64, "beams": 8, "n": 131072, "dtype": "bf16", "pad": 0, "keep": 16, "done": 0.0,
         "closed": 0.01, "temperature": 1.0},
        # The tokens chosen so far.
        {"name": "reorder tokens", "op": "reorder", "batch": 64, "beams": 8, "tensors": 1, "heads": 1, "room": 2048, "used": 777, "dim": 1,
         "dtype": "i64", "moved": 5, "sources": 3},
        # One question's cache of keys and values, two thirds of its room in use.
        {"name": "reorder step", "op": "reorder", "batch": 1, "beams": 4, "tensors": 32, "heads": 8, "room": 1024, "used": 701, "dim": 128,
         "dtype": "bf16", "moved": 2, "sources": 2},
        # A batch's caches of keys and values.
        {"name": "reorder large", "op": "reorder", "batch": 8, "beams": 8, "tensors": 16, "heads": 8, "room": 1024, "used": 1000, "dim": 128,
         "dtype": "bf16", "moved": 6, "sources": 4},
    ]


def spread(rng, low, high):
    """A whole number of low..high, even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["route", "route", "beam", "beam", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        n = groups * spread(rng, 4, 512 // groups)
        top_groups = rng.randint(1, groups)
        return {"op": op, "rows": spread(rng, 1, MOST_ROUTE // (n * SIZE[dtype])), "n": n, "dtype": dtype, "pad": rng.choice([0, 0, 3]),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6, "groups": groups, "top_groups": top_groups,
                "best": rng.choice([1, 2]), "top_k": min(top_groups * (n // groups), rng.choice([1, 2, 4, 6, 8, 12])),
                "masked": rng.choice([0.0, 0.1, 0.5]), "closed": rng.choice([0, 0, n // 16]), "renormalize": rng.random() < 0.5,
                "scale": rng.choice([1.0, 2.5]), "grad": rng.random() < 0.7}
    if op == "beam":
        n, beams = spread(rng, 300, 200003), rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        pad = rng.choice([0, 0, -n % 64, rng.randrange(1, 64)])
        return {"op": op, "batch": spread(rng, 1, max(1, min(256, MOST_BEAM // ((n + pad) * SIZE[dtype] * beams)))), "beams": beams, "n": n,
                "dtype": dtype, "pad": pad, "keep": rng.choice([1, beams, beams, 2 * beams]), "done": rng.choice([0.0, 0.0, 0.2]),
                "closed": rng.choice([0.0, 0.02]), "temperature": rng.choice([1.0, 1.0, 0.8])}
    batch, beams, heads, dim = spread(rng, 1, 32), rng.choice([2, 3, 4, 5, 8, 12]), rng.choice([1, 2, 5, 8]), rng.choice([16, 36, 64, 128])
    tensors = spread(rng, 1, 32)
    room = spread(rng, 16, max(16, min(4096, MOST_STATE // (batch * beams * tensors * heads * dim * SIZE[dtype]))))
    moved = rng.randint(1, beams) if beams > 2 else 2
    return {"op": op, "batch": batch, "beams": beams, "tensors": tensors, "heads": heads, "room": room, "used": rng.randint(1, room),
            "dim": dim, "dtype": dtype, "moved": max(2, moved), "sources": rng.randint(2, max(2, moved))}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    dtype = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def chance(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    if case["op"] == "route":
        rows, n = case["rows"], case["n"]
        x = torch.empty((rows, n + case["pad"]), dtype=dtype, device="cuda")[:, :n]
        # A trained router: some experts are asked for more than others.
        x.copy_(normal(rows, n).add_(0.7 * normal(1, n)))
        if case["closed"]:
            x[:, torch.randperm(n, generator=g, device="cuda")[:case["closed"]]] = -math.inf
        s["logits"] = x
        s["mask"] = chance(rows) >= case["masked"] if case["masked"] else None
        # The bias moves in steps of a thousandth against the load.
        size = 100.0 if case["score"] == "sigmoid" else 10.0
        s["bias"] = torch.round(size * normal(n)) / 1000.0 if case["bias"] else None
        s["grad"] = normal(rows, case["top_k"]) / rows
        if case["dtype"] == "f16":
            s["grad"] *= 4096.0
        return s
    if case["op"] == "beam":
        batch, beams, n = case["batch"], case["beams"], case["n"]
        rows = batch * beams
        x = torch.randn((rows, n + case["pad"]), generator=g, device="cuda", dtype=dtype).mul_(2.0)[:, :n]
        shut = int(n * case["closed"])
        # A wide bulk and some likely tokens.
        likely = torch.randint(0, n - shut, (rows, 24), generator=g, device="cuda")
        x.scatter_(1, likely, (9.0 + 2.0 * normal(rows, 24)).to(dtype))
        if shut:
            x[:, n - shut:] = -math.inf
        s["logits"] = x
        s["scores"] = -(3.0 + 2.0 * chance(batch, beams)).cumsum(1)
        s["done"] = chance(batch, beams) < case["done"] if case["done"] else None
        s["end"] = 2
        return s
    batch, beams = case["batch"], case["beams"]
    shape = (batch * beams, case["heads"], case["room"], case["dim"])
    s["states"] = []
    for _ in range(case["tensors"]):
        if case["dtype"] == "i64":
            whole = torch.randint(0, 131072, shape, generator=g, device="cuda")
        else:
            whole = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
        s["states"].append(whole[:, :, :case["used"]])
    # `moved` beams of each item take over from `sources` of them, all in a ring: some only swap.
    order = chance(batch, beams).argsort(1)
    at = torch.arange(case["moved"], device="cuda")
    parents = torch.arange(beams, device="cuda").expand(batch, beams).clone()
    parents.scatter_(1, order[:, :case["moved"]], order[:, (at + 1) % case["sources"]])
    s["parents"] = parents.to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# This repository's calls
# ---------------------------------------------------------------------------
def own_run(s):
    from convex_hull_pava_gb300 import choices

    case = s["case"]
    if case["op"] == "route":
        r = choices.iso_route(
            s["logits"], case["top_k"], s["mask"], score=case["score"], bias=s["bias"], groups=case["groups"],
            top_groups=case["top_groups"], group_best=case["best"], renormalize=case["renormalize"], scale=case["scale"])
        out = {"gates": r.gates, "experts": r.experts, "counts": r.counts}
        if case["grad"]:
            out["dlogits"] = choices.iso_route_backward(s["grad"], s["logits"], r)
        return out
    if case["op"] == "beam":
        r = choices.iso_beam_choose(s["logits"], s["scores"], case["keep"], s["done"], end=s["end"], temperature=case["temperature"])
        return {"scores": r.scores, "beams": r.beams, "tokens": r.tokens}
    choices.iso_beam_reorder(s["states"], s["parents"])
    return s["states"]


# ---------------------------------------------------------------------------
# The plain forms.  What is ranked is computed in 64 bits: in 32, a choice between values next to each
# other would be that of their roundings.
# ---------------------------------------------------------------------------
def plain_route(s):
    case = s["case"]
    x, k, n = s["logits"].double(), case["top_k"], case["n"]
    rows = x.shape[0]
    open_ = x > -math.inf
    if s["mask"] is not None:
        open_ = open_ & s["mask"][:, None]
    live = open_.any(1, keepdim=True)
    if case["score"] == "softmax":
        e = torch.where(live, torch.exp(x - torch.where(live, x.amax(1, keepdim=True), 0.0)), 0.0)
        p = e / torch.where(live, e.sum(1, keepdim=True), 1.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    c = p if s["bias"] is None else p + s["bias"].double()
    c = torch.where(open_, c, -math.inf)
    if case["groups"] > 1:
        by_group = torch.sort(c.view(rows, case["groups"], -1), dim=2, descending=True)[0][:, :, :case["best"]]
        some = by_group[:, :, 0] > -math.inf
        of_group = torch.where(some, torch.where(by_group > -math.inf, by_group, 0.0).sum(2), -math.inf)
        first = torch.sort(of_group, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        kept = torch.zeros_like(some).scatter_(1, first, True)
        c = torch.where(kept[:, :, None], c.view(rows, case["groups"], -1), -math.inf).view(rows, n)
    value, order = torch.sort(c, dim=1, descending=True, stable=True)
    chosen = value[:, :k] > -math.inf
    experts = torch.where(chosen, order[:, :k], -1)
    counts = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    counts = counts.scatter_add_(0, (experts + 1).reshape(-1), torch.ones_like(experts).reshape(-1))[1:]
    at = experts.clamp(min=0)
    share = torch.where(chosen, p.gather(1, at), 0.0)
    if case["renormalize"]:
        share = share / torch.where(chosen[:, :1], share.sum(1, keepdim=True), 1.0)
    out = {"gates": (case["scale"] * share).float(), "experts": experts.to(torch.int32), "counts": counts}
    if case["grad"]:
        g = torch.where(chosen, case["scale"] * s["grad"].double(), 0.0)
        if case["renormalize"]:
            each = share * (g - (share * g).sum(1, keepdim=True))
            if case["score"] == "sigmoid":
                each = torch.where(chosen, each * (1.0 - p.gather(1, at)), 0.0)
            d = torch.zeros_like(x).scatter_add_(1, at, each)
        elif case["score"] == "sigmoid":
            d = torch.zeros_like(x).scatter_add_(1, at, torch.where(chosen, g * share * (1.0 - p.gather(1, at)), 0.0))
        else:
            u = torch.zeros_like(x).scatter_add_(1, at, g)
            d = p * (u - (p * u).sum(1, keepdim=True))
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def plain_beam(s):
    case = s["case"]
    batch, beams, n = case["batch"], case["beams"], case["n"]
    x = s["logits"].double() / case["temperature"]
    x = x - x.amax(1, keepdim=True)
    total = x - torch.log(torch.exp(x).sum(1, keepdim=True)) + s["scores"].double().view(-1, 1)
    if s["done"] is not None:
        ended = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
        ended[s["end"]] = 0.0
        total = torch.where(s["done"].view(-1, 1), s["scores"].double().view(-1, 1) + ended, total)
    value, order = torch.sort(total.view(batch, beams * n), dim=1, descending=True, stable=True)
    value, order = value[:, :case["keep"]], order[:, :case["keep"]]
    some = value > -math.inf
    return {"scores": value.float(), "beams": torch.where(some, order // n, -1).to(torch.int32), "tokens": torch.where(some, order % n, -1)}


def plain_reorder(s):
    batch, beams = s["parents"].shape
    rows = (s["parents"] + beams * torch.arange(batch, device="cuda")[:, None]).reshape(-1)
    return [x.copy_(x[rows]) for x in s["states"]]


def plain_run(s):
    op = s["case"]["op"]
    return plain_route(s) if op == "route" else plain_beam(s) if op == "beam" else plain_reorder(s)


def run(state):
    return own_run(state) if own else plain_run(state)


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "route":
        rows, n, k = case["rows"], case["n"], case["top_k"]
        size = rows * n * b + rows * k * 8 + n * (12 if case["bias"] else 8) + (rows if case["masked"] else 0)
        return {"bytes": size + (rows * n * b + rows * k * 4 if case["grad"] else 0), "flops": rows * n * (6 + (4 if case["grad"] else 0))}
    if case["op"] == "beam":
        rows = case["batch"] * case["beams"]
        return {"bytes": (1.0 - case["done"]) * rows * case["n"] * b + rows * 4 + case["batch"] * case["keep"] * 16,
                "flops": 4 * (1.0 - case["done"]) * rows * case["n"]}
    row = case["tensors"] * case["heads"] * case["used"] * case["dim"] * b
    return {"bytes": case["batch"] * (row * (case["moved"] + case["sources"]) + 4 * case["beams"]), "flops": 0}


# ---------------------------------------------------------------------------
# The definitions in 64 bits; the gradient by differentiating them
# ---------------------------------------------------------------------------
def best_of(value, count):
    """The places of the `count` largest of each row, of equal ones the first; -1 where only -inf is left."""
    left, found = value.clone(), []
    for _ in range(count):
        most, at = left.max(1)
        ties = left == most[:, None]
        at = ties.to(torch.uint8).argmax(1) if bool((ties.sum(1) > 1).any()) else at
        found.append(torch.where(most > -math.inf, at, -1))
        left.scatter_(1, at[:, None], -math.inf)
    return torch.stack(found, 1)


def exact_route(s):
    case = s["case"]
    n, k, size = case["n"], case["top_k"], case["n"] // case["groups"]
    x = s["logits"].double().requires_grad_()
    rows = x.shape[0]
    live = torch.isfinite(x).any(1)
    if s["mask"] is not None:
        live = live & s["mask"]
    p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    c = p.detach() if s["bias"] is None else p.detach() + s["bias"].double()
    c = c.masked_fill(~(live[:, None] & torch.isfinite(x)), -math.inf)
    if case["groups"] > 1:
        of_group = []
        for part in c.split(size, 1):
            at = best_of(part, min(case["best"], size))
            value = part.gather(1, at.clamp(min=0)).masked_fill(at < 0, 0.0).sum(1)
            of_group.append(value.masked_fill(at[:, 0] < 0, -math.inf))
        kept = best_of(torch.stack(of_group, 1), case["top_groups"])
        group = torch.arange(n, device="cuda") // size
        stays = torch.zeros((rows, n), dtype=torch.bool, device="cuda")
        for j in range(case["top_groups"]):
            stays |= group[None, :] == kept[:, j:j + 1]
        c = c.masked_fill(~stays, -math.inf)
    experts = best_of(c, k)
    hit = experts >= 0
    gates = p.gather(1, experts.clamp(min=0)).masked_fill(~hit, 0.0)
    if case["renormalize"]:
        gates = gates / gates.sum(1, keepdim=True).masked_fill(~hit[:, :1], 1.0)
    gates = gates * case["scale"]
    out = {"gates": gates.detach(), "experts": experts.to(torch.int32), "counts": torch.bincount(experts[hit], minlength=n)}
    if case["grad"]:
        d = torch.autograd.grad((gates * s["grad"].double()).masked_fill(~hit, 0.0).sum(), x)[0]
        out["dlogits"] = d.masked_fill(~live[:, None], 0.0)
    return out


def exact_beam(s):
    case = s["case"]
    scores, beams, tokens = [], [], []
    for item, logits in enumerate(s["logits"].split(case["beams"])):
        total = torch.log_softmax(logits.double() / case["temperature"], 1) + s["scores"][item, :, None].double()
        if s["done"] is not None:
            for b in s["done"][item].nonzero()[:, 0].tolist():
                total[b] = -math.inf
                total[b, s["end"]] = s["scores"][item, b].double()
        at = best_of(total.reshape(1, -1), case["keep"])[0]
        scores.append(total.reshape(-1)[at.clamp(min=0)].masked_fill(at < 0, -math.inf))
        beams.append(torch.where(at < 0, -1, at // case["n"]).to(torch.int32))
        tokens.append(torch.where(at < 0, -1, at % case["n"]))
    return {"scores": torch.stack(scores), "beams": torch.stack(beams), "tokens": torch.stack(tokens)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return exact_route(s)
    if case["op"] == "beam":
        return exact_beam(s)
    beams, parents = case["beams"], s["parents"].tolist()
    return [torch.stack([x[item * beams + b] for item, row in enumerate(parents) for b in row]) for x in s["states"]]
