"""The training objectives in 64 bits, row by row, from their formulas (numpy).

Independent of the package: only the tests use it.  Scores come as float64 arrays of the
values that the GPU sees (its float32, bfloat16 or float16 scores widened)."""
import numpy as np


def log_softmax(x, t=1.0):
    v = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        top = v.max() if v.size else -np.inf
        if not np.isfinite(top):
            return np.full(v.shape, np.nan)
        v = (v - top) / t
        return v - np.log(np.exp(v).sum())


def token_logp(x, labels, t=1.0):
    lp = np.zeros(len(labels))
    for r, l in enumerate(labels):
        if l >= 0:
            lp[r] = log_softmax(x[r], t)[l] if l < x.shape[1] else np.nan
    return lp


def grad_logits(coef, x, labels, t=1.0):
    """coef (onehot - p) / T, and the probabilities."""
    d = np.zeros(x.shape)
    p = np.zeros(x.shape)
    for r, l in enumerate(labels):
        if l < 0:
            continue
        p[r] = np.exp(log_softmax(x[r], t))
        d[r] = -coef[r] * p[r] / t
        if l < x.shape[1]:
            d[r, l] += coef[r] / t
    return d, p


def policy(x, labels, old, adv, ref=None, weights=None, low=0.2, high=0.2, kl_coef=0.0, t=1.0):
    """(loss, stats, lp, coef)"""
    lp = token_logp(x, labels, t)
    live = [r for r, l in enumerate(labels) if l >= 0]
    coef = np.zeros(len(labels))
    stats = np.zeros(3)
    for r in live:
        w = float(weights[r]) if weights is not None else 1.0 / len(live)
        q = np.exp(lp[r] - float(old[r]))
        a = float(adv[r])
        free, held = -a * q, -a * min(max(q, 1.0 - low), 1.0 + high)
        if held > free:
            stats[0] += w * held
            stats[2] += w
        else:
            stats[0] += w * free
            coef[r] = w * free
        if ref is not None:
            d = float(ref[r]) - lp[r]
            stats[1] += w * (np.exp(d) - 1.0 - d)
            coef[r] += kl_coef * w * (1.0 - np.exp(d))
    return stats[0] + (kl_coef if ref is not None else 0.0) * stats[1], stats, lp, coef


def preference(x, labels, offsets, ref=None, kind="sigmoid", beta=0.1, smooth=0.0, average=False):
    """(loss, margins, seq, lp, coef)"""
    lp = token_logp(x, labels)
    pairs = len(offsets) // 2
    seq = np.zeros(2 * pairs)
    gain = np.zeros(2 * pairs)
    share = np.zeros(2 * pairs)
    for s in range(2 * pairs):
        rows = [r for r in range(offsets[s], offsets[s + 1]) if labels[r] >= 0]
        share[s] = 1.0 / max(1, len(rows)) if average else 1.0
        seq[s] = share[s] * sum(lp[r] for r in rows)
        gain[s] = share[s] * sum(lp[r] - (float(ref[r]) if ref is not None else 0.0) for r in rows)
    h = gain[0::2] - gain[1::2]
    z = beta * h
    if kind == "sigmoid":
        each = (1 - smooth) * np.logaddexp(0.0, -z) + smooth * np.logaddexp(0.0, z)
        slope = beta * (smooth / (1 + np.exp(-z)) - (1 - smooth) / (1 + np.exp(z)))
    elif kind == "hinge":
        each = np.maximum(0.0, 1.0 - z)
        slope = np.where(z < 1.0, -beta, 0.0)
    else:
        each = (h - 1.0 / (2.0 * beta)) ** 2
        slope = 2.0 * (h - 1.0 / (2.0 * beta))
    coef = np.zeros(len(labels))
    for s in range(2 * pairs):
        for r in range(offsets[s], offsets[s + 1]):
            if labels[r] >= 0:
                coef[r] = (1 if s % 2 == 0 else -1) * slope[s // 2] * share[s] / pairs
    return (each.mean() if pairs else 0.0), z, seq, lp, coef


def balance(x, top_k, mask=None, renormalize=False):
    """(loss, counts, experts, gates, live)"""
    tokens, n = x.shape
    counts = np.zeros(n, np.int64)
    experts = np.full((tokens, top_k), -1, np.int32)
    gates = np.zeros((tokens, top_k))
    total = np.zeros(n)
    live = 0
    for t in range(tokens):
        if (mask is not None and not mask[t]) or not (x[t] > -np.inf).any():
            continue
        live += 1
        p = np.exp(log_softmax(x[t]))
        total += p
        order = sorted((e for e in range(n) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))[:top_k]
        for i, e in enumerate(order):
            experts[t, i] = e
            gates[t, i] = p[e]
            counts[e] += 1
        if renormalize:
            gates[t] /= gates[t].sum()
    loss = n / (top_k * live * live) * (counts * total).sum() if live else 0.0
    return loss, counts, experts, gates, live


def balance_grad(x, top_k, mask, renormalize, g_loss, g_gates):
    tokens, n = x.shape
    loss, counts, experts, gates, live = balance(x, top_k, mask, renormalize)
    d = np.zeros(x.shape)
    for t in range(tokens):
        if (mask is not None and not mask[t]) or not (x[t] > -np.inf).any():
            continue
        p = np.exp(log_softmax(x[t]))
        u = g_loss * n / (top_k * live * live) * counts.astype(np.float64)
        picked = [(i, e) for i, e in enumerate(experts[t]) if e >= 0]
        if not renormalize:
            for i, e in picked:
                u[e] += g_gates[t, i]
        d[t] = p * (u - (p * u).sum())
        if renormalize:
            mean = sum(gates[t, i] * g_gates[t, i] for i, _ in picked)
            for i, e in picked:
                d[t, e] += gates[t, i] * (g_gates[t, i] - mean)
    return d
