"""The choices over rows of scores in 64 bits (numpy), from their definitions."""
import numpy as np


def shares(x, score):
    """Softmax or sigmoid of rows in 64 bits; a row with NaN or +inf has no softmax (NaN)."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(m), m, 0.0))
        return np.where(np.isfinite(m), e / e.sum(1, keepdims=True), np.nan)


def first(value, count):
    """The places of the `count` largest that are not -inf, equal ones by place; -1 where none is left."""
    order = sorted((i for i in range(len(value)) if value[i] > -np.inf), key=lambda i: (-value[i], i))[:count]
    return order + [-1] * (count - len(order))


def route(x, top_k, mask=None, score="softmax", bias=None, groups=1, top_groups=1, group_best=2,
          renormalize=False, scale=1.0):
    """(gates, experts, counts, shares of the chosen without scale)"""
    x = np.asarray(x, np.float64)
    tokens, n = x.shape
    p = shares(x, score)
    size = n // groups
    b = None if bias is None else np.asarray(bias, np.float64)
    experts = np.full((tokens, top_k), -1, np.int32)
    gates = np.zeros((tokens, top_k))
    counts = np.zeros(n, np.int64)
    for t in range(tokens):
        if mask is not None and not mask[t]:
            continue
        bad = score == "softmax" and not (x[t] < np.inf).all()
        q = np.where(np.isnan(p[t]), 0.0, p[t])
        closed = ~(x[t] > -np.inf)
        c = x[t].copy() if b is None else q + b   # without a bias the order is that of x
        if b is not None:
            closed |= ~(b > -np.inf)
        c[closed] = -np.inf
        if groups > 1:
            value = []
            for g in range(groups):
                top = [g * size + i for i in first(c[g * size:(g + 1) * size], group_best) if i >= 0]
                if not top:
                    value.append(-np.inf)
                elif b is None and group_best == 1:
                    value.append(c[top[0]])
                else:
                    value.append(sum(q[i] if b is None else c[i] for i in top))
            kept = first(value, top_groups)
            for g in range(groups):
                if g not in kept:
                    c[g * size:(g + 1) * size] = -np.inf
        e = first(c, top_k)
        experts[t] = e
        at = [i for i in e if i >= 0]
        counts[at] += 1
        if not at:
            continue
        with np.errstate(all="ignore"):
            if not renormalize:
                s = p[t, at]
            else:
                v = x[t, at]
                if score == "softmax":
                    s = np.exp(v - v.max())
                else:
                    low = min(v.max(), 0.0)
                    s = np.where(v > 0, 1.0 / (1.0 + np.exp(-v)), np.exp(v - low) / (1.0 + np.exp(np.minimum(v, 0.0))))
                s = s / s.sum()
        gates[t, :len(at)] = np.nan if bad else scale * s
    return gates, experts, counts


def route_grad(x, grad_gates, gates, experts, score="softmax", renormalize=False, scale=1.0):
    """The gradient of sum(grad_gates * gates) in x, from the formulas."""
    x = np.asarray(x, np.float64)
    g = np.asarray(grad_gates, np.float64)
    p = shares(x, score)
    d = np.zeros_like(x)
    for t in range(len(x)):
        hit = [i for i in range(experts.shape[1]) if experts[t, i] >= 0]
        if not hit:
            continue
        at, gt, gg = experts[t, hit], gates[t, hit], g[t, hit]
        if np.isnan(gt).any():
            d[t] = np.nan
            continue
        with np.errstate(all="ignore"):
            rest = 1.0 / (1.0 + np.exp(x[t, at])) if score == "sigmoid" else 1.0
        if renormalize:
            d[t, at] = gt * rest * (gg - (gt * gg).sum() / scale)
        elif score == "sigmoid":
            d[t, at] = gt * rest * gg
        else:
            u = np.zeros(x.shape[1])
            u[at] = scale * gg
            d[t] = p[t] * (u - (gt * gg).sum())
    return d


def log_probabilities(x, temperature):
    """x / T - log sum exp(x / T) of rows; NaN where a row has NaN, +inf or nothing but -inf."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        y = np.where(np.isfinite(m), (x - m) / temperature, np.nan)
        return y - np.log(np.exp(y).sum(1, keepdims=True))


def beam_choose(x, scores, keep, done=None, end=0, temperature=1.0):
    """(scores, beams, tokens, bad rows); x [batch * beams, n]"""
    scores = np.asarray(scores, np.float64)
    batch, beams = scores.shape
    x = np.asarray(x, np.float64)
    n = x.shape[1]
    lp = log_probabilities(x, temperature)
    out = np.full((batch, keep), -np.inf)
    parents = np.full((batch, keep), -1, np.int32)
    tokens = np.full((batch, keep), -1, np.int64)
    bad = np.zeros(batch * beams, bool)
    for i in range(batch):
        total = np.full((beams, n), -np.inf)
        for b in range(beams):
            r = i * beams + b
            if not np.isfinite(scores[i, b]):
                continue
            if done is not None and done[i, b]:
                total[b, end] = scores[i, b]
            elif np.isnan(lp[r]).any():
                bad[r] = True
            else:
                total[b] = scores[i, b] + lp[r]
        flat = total.reshape(-1)
        some = np.flatnonzero(flat > -np.inf)
        if len(some) > 4 * keep:
            edge = np.partition(flat[some], len(some) - keep)[len(some) - keep]
            some = some[flat[some] >= edge]
        order = some[np.lexsort((some, -flat[some]))][:keep]
        out[i, :len(order)] = flat[order]
        parents[i, :len(order)] = order // n
        tokens[i, :len(order)] = order % n
    return out, parents, tokens, bad
