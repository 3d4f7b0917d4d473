"""The training objectives on the GPU against their 64-bit forms.

Tolerances (written before the first run).
* A log-probability: the score's difference and its scaling round at 2^-24 each, the
  exponential's relative error is 2^-22, the sum of n terms in float32 adds sqrt(adds) * 2^-25
  in a chain of at most 1,024 adds (1e-6); the result rounds at 2^-24 of itself.  Together
  under LP = 4e-6 * (1 + |lp|).
* A probability: that of the exponential, 2^-22 + |v| 2^-23 with v the exponent's argument in
  base 2, and the sum's: p * (4e-6 + 1.2e-7 |v|).
* A gradient element: the coefficient's error on |d|, the probability's error times |c| / T,
  the label's cancellation |c| / T * 2^-22, one rounding to the type (half a unit: 2^-24, 2^-8,
  2^-11 relative; float16 subnormals 2^-25 absolute).
* A coefficient: exp turns the log-probability's absolute error into a relative one, so
  LP(lp) * (its own size + what the KL term adds), and a few roundings (1e-6).
* Means over rows: the mean of the rows' bounds."""
import numpy as np
import pytest

import objectives_ref as ref

pytestmark = pytest.mark.gpu

TYPES = ("f32", "bf16", "f16")
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}


def tor(dtype):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]


def lp_tol(lp):
    return 4e-6 * (1.0 + np.abs(lp))


def put(v, dtype="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda().to(tor(dtype))


def ids(v):
    import torch
    return torch.from_numpy(np.ascontiguousarray(v, np.int64)).cuda()


def wide(t):
    return t.detach().double().cpu().numpy()


def make(rows, n, dtype, seed, pad=0, shift=0, closed=0.0, ignored=0.2):
    """(scores on the GPU as a view of rows padded by `pad` that starts `shift` elements into its
    buffer, the values they have, labels)"""
    import torch
    rng = np.random.default_rng(seed)
    buf = torch.full((rows * (n + pad) + shift,), float("nan"), dtype=tor(dtype), device="cuda")
    x = buf[shift:].view(rows, n + pad)[:, :n]
    x.copy_(put(2.0 * rng.standard_normal((rows, n)), dtype))
    open_ = max(1, n - int(closed * n))
    x[:, open_:] = -float("inf")
    labels = rng.integers(0, open_, rows)
    lift = put(6.0 + 2.0 * rng.standard_normal(rows), dtype)
    x[torch.arange(rows, device="cuda"), ids(labels)] = lift
    if rows > 1:
        labels[rng.permutation(rows)[:int(ignored * rows)]] = -100
    return x, wide(x), labels, rng


def check_grad(got, x, labels, coef, coef_tol, dtype, t=1.0, scale=1.0):
    want, p = ref.grad_logits(coef * scale, x, labels, t)
    with np.errstate(all="ignore"):
        v = np.where(p > 0, np.abs(np.log2(np.maximum(p, 1e-300))), 0.0)
        c = (np.abs(coef * scale) / t)[:, None]
        ct = (coef_tol * abs(scale) / t)[:, None]
        tol = c * p * (4e-6 + 1.2e-7 * v) + ct * p + HALF[dtype] * np.abs(want) * 1.001 + TINY[dtype] + 1e-12 * c
    for r, l in enumerate(labels):
        if l >= 0:
            tol[r, l] += c[r, 0] * 2.0 ** -22 + ct[r, 0]
    off = np.abs(wide(got) - want) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


SIZES = [(1, 1), (3, 1), (2, 2), (5, 7), (4, 8), (3, 31), (3, 33), (2, 255), (5, 256), (3, 257), (9, 1000),
         (700, 130), (4, 4096), (3, 8191), (3, 8192), (5, 20011), (3, 32771), (2, 65536), (2, 131075), (1, 131072),
         (1, 200003), (2, 600011)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", SIZES)
def test_token_logp(cuda_ok, rows, n, dtype):
    from convex_hull_pava_gb300 import objectives as obj
    for pad, shift, t in ((0, 0, 1.0), (5, 0, 0.7), (-n % 64, 3, 1.3)):
        x, xw, labels, rng = make(rows, n, dtype, seed=n + pad, pad=pad, shift=shift, closed=0.1)
        lp, norm, st = obj.iso_token_logp(x, ids(labels), temperature=t)
        want = ref.token_logp(xw, labels, t)
        assert (np.abs(wide(lp) - want) <= lp_tol(want)).all()
        assert (wide(lp)[labels < 0] == 0).all() and not st.any()
        g = rng.standard_normal(rows).astype(np.float32)
        d = obj.iso_token_logp_backward(put(g), x, ids(labels), norm, temperature=t, grad_scale=3.0)
        assert d.dtype == x.dtype and d.shape == x.shape
        check_grad(d, xw, labels, g.astype(np.float64), np.zeros(rows), dtype, t, 3.0)
        assert (wide(d)[labels < 0] == 0).all()


def policy_inputs(xw, labels, rng, t):
    lp = ref.token_logp(xw, labels, t)
    move = 0.25 * rng.standard_normal(len(labels))
    for edge in (np.log(0.8), np.log(1.3)):   # away from the clip's corners by more than LP
        move = np.where(np.abs(move - edge) < 1e-3, move + 4e-3, move)
    old = np.where(labels >= 0, lp - move, np.nan)       # not used where there is no label
    adv = np.where(labels >= 0, rng.standard_normal(len(labels)), np.nan)
    base = np.where(labels >= 0, lp + 0.3 * rng.standard_normal(len(labels)), np.nan)
    return [v.astype(np.float32) for v in (old, adv, base)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_policy_loss(cuda_ok, rows, n, dtype, kl):
    from convex_hull_pava_gb300 import objectives as obj
    for pad, shift, t, weighted in ((0, 0, 1.0, False), (3, 1, 0.8, True)):
        x, xw, labels, rng = make(rows, n, dtype, seed=7 * n + pad, pad=pad, shift=shift, closed=0.05)
        old, adv, base = policy_inputs(xw, labels, rng, t)
        w = rng.uniform(0.1, 1.0, rows).astype(np.float32) if weighted else None
        scale = 64.0
        r = obj.iso_policy_loss(x, ids(labels), put(old), put(adv), put(base) if kl else None,
                                None if w is None else put(w), clip_low=0.2, clip_high=0.3, kl_coef=kl,
                                temperature=t, grad_scale=scale)
        loss, stats, lp, coef = ref.policy(xw, labels, old, adv, base if kl else None, w, 0.2, 0.3, kl, t)
        assert (np.abs(wide(r.logp) - lp) <= lp_tol(lp)).all()
        live = labels >= 0
        ww = np.where(live, w if w is not None else 1.0 / max(1, live.sum()), 0.0).astype(np.float64)
        with np.errstate(all="ignore"):
            size = np.where(live, np.abs(adv) * np.exp(lp - old) + (kl * np.exp(base - lp) if kl else 0.0), 0.0)
        coef_tol = ww * size * (lp_tol(lp) + 1e-6)
        assert (np.abs(wide(r.coef) - coef) <= coef_tol).all()
        bound = coef_tol.sum() + 1e-6 * abs(loss) + 1e-7
        assert abs(float(r.loss) - loss) <= bound
        kl_bound = (ww * (lp_tol(lp) + 1e-6) * np.where(live, np.exp(np.where(live, base - lp, 0.0)) + 1, 0)).sum()
        assert np.abs(wide(r.stats) - stats).max() <= bound + kl_bound + 1e-6 * ww.sum()
        assert not r.row_status.any()
        check_grad(r.dlogits, xw, labels, coef, coef_tol, dtype, t, scale)
        again = obj.iso_policy_loss(x, ids(labels), put(old), put(adv), put(base) if kl else None,
                                    None if w is None else put(w), clip_low=0.2, clip_high=0.3, kl_coef=kl,
                                    temperature=t, grad_scale=scale)
        for a, b in zip(r, again):
            assert a is b or bool((a.isnan() | (a == b)).all())
        without = obj.iso_policy_loss(x, ids(labels), put(old), put(adv), put(base) if kl else None,
                                      None if w is None else put(w), clip_low=0.2, clip_high=0.3, kl_coef=kl,
                                      temperature=t, want_grad=False)
        assert without.dlogits is None and abs(float(without.loss) - loss) <= bound


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("sizes,n", [((1, 1), 300), ((3, 0, 2, 5), 1000), ((0, 0), 50), ((40, 33, 1, 70, 8, 9), 8195),
                                     ((6, 7), 131072), ((2, 3, 4, 1), 70001)])
def test_preference_loss(cuda_ok, sizes, n, kind, dtype):
    from convex_hull_pava_gb300 import objectives as obj
    for average, smooth, with_ref, extra in ((False, 0.1, True, 0), (True, 0.0, True, 3), (False, 0.0, False, 1)):
        off = np.concatenate([[0], np.cumsum(sizes)]) + extra
        rows = int(off[-1]) + extra        # `extra` rows before and after all sequences
        if rows == 0:
            rows = 1
        x, xw, labels, rng = make(rows, n, dtype, seed=n + rows, closed=0.02)
        lp = ref.token_logp(xw, labels)
        base = np.where(labels >= 0, lp + 0.2 * rng.standard_normal(rows), np.nan).astype(np.float32)
        beta = 0.5 if average else 0.1
        r = obj.iso_preference_loss(x, ids(labels), ids(off), put(base) if with_ref else None, kind=kind, beta=beta,
                                    label_smoothing=smooth, average=average, grad_scale=8.0)
        loss, z, seq, lp, coef = ref.preference(xw, labels, off.tolist(), base if with_ref else None, kind, beta,
                                                smooth if kind == "sigmoid" else 0.0, average)
        # a margin: the errors of its tokens' log-probabilities
        z_tol, pairs = np.zeros(len(z)), len(z)
        for s in range(2 * pairs):
            inside = [q for q in range(off[s], off[s + 1]) if labels[q] >= 0]
            share = 1.0 / max(1, len(inside)) if average else 1.0
            err = share * sum(lp_tol(lp[q]) for q in inside)
            assert abs(float(r.seq_logp[s]) - seq[s]) <= err + 1e-6 * abs(seq[s])
            z_tol[s // 2] += beta * err
        z_tol += 1e-6 * np.abs(z)
        assert (np.abs(wide(r.margins) - z) <= z_tol).all()
        # slopes: 1 in z for the sigmoid and the hinge, 2 / beta^2 (z - 1/2) for the square
        steep = 2.0 / beta ** 2 * np.abs(z - 0.5) if kind == "squared" else np.ones(pairs)
        assert abs(float(r.loss) - loss) <= (steep * z_tol).mean() + 1e-6 * abs(loss) + 1e-7
        curve = (2.0 / beta if kind == "squared" else beta * 0.25 if kind == "sigmoid" else 0.0) * z_tol / pairs
        coef_tol = np.zeros(rows)
        for s in range(2 * pairs):
            coef_tol[off[s]:off[s + 1]] = curve[s // 2]
        coef_tol += 1e-6 * np.abs(coef)
        assert (np.abs(wide(r.coef) - coef) <= coef_tol).all()
        assert not r.row_status.any() and not r.pair_status.any()
        check_grad(r.dlogits, xw, labels, coef, coef_tol, dtype, 1.0, 8.0)


ROUTERS = [(1, 1, 1), (1, 4, 2), (7, 5, 5), (33, 32, 1), (64, 33, 8), (100, 64, 2), (257, 128, 8), (90, 160, 6),
           (40, 256, 8), (31, 300, 32), (17, 512, 8), (9, 1000, 4), (5, 1024, 32), (3000, 8, 2)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,n,k", ROUTERS)
@pytest.mark.parametrize("renormalize", [False, True])
def test_balance_loss(cuda_ok, tokens, n, k, renormalize, dtype):
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    for pad, masked in ((0, False), (3, True)):
        rng = np.random.default_rng(tokens + n + pad)
        raw = rng.standard_normal((tokens, n + pad))
        if tokens > 3:
            raw[:, : n // 3] = np.round(raw[:, : n // 3])      # ties
            raw[1, n // 2:] = -np.inf                          # closed experts, perhaps under k open
            raw[2] = -np.inf                                   # nothing open
            raw[3] = -0.0
            raw[3, ::2] = 0.0                                  # equal zeros of both signs
        x = put(raw, dtype)[:, :n]
        xw = wide(x)
        mask = rng.random(tokens) < 0.7 if masked else None
        mt = None if mask is None else torch.from_numpy(mask).cuda()
        r = obj.iso_balance_loss(x, k, mt, renormalize=renormalize)
        loss, counts, experts, gates, live = ref.balance(xw, k, mask, renormalize)
        assert int(r.live) == live
        assert np.array_equal(r.counts.cpu().numpy(), counts)
        assert np.array_equal(r.experts.cpu().numpy(), experts)
        assert np.abs(wide(r.gates) - gates).max() <= 4e-6
        assert abs(float(r.loss) - loss) <= 1e-5 * (1 + abs(loss))
        gg = rng.standard_normal((tokens, k)).astype(np.float32)
        for g_gates in (gg, None):
            d = obj.iso_balance_loss_backward(x, r, grad_loss=0.5, grad_gates=None if g_gates is None else put(gg))
            want = ref.balance_grad(xw, k, mask, renormalize, 0.5, gg.astype(np.float64) if g_gates is not None else 0 * gg)
            # each element is p (u - mean u): p to 4e-6, u's largest entry times the sums' 1e-5
            top = np.abs(gg).max() + 0.5 * n * counts.max(initial=0) / max(1, k * live * live)
            assert np.abs(wide(d) - want).max() <= 1e-5 * top + (HALF[dtype] * np.abs(want)).max() + TINY[dtype]
            assert d.dtype == x.dtype


def test_infinities_nan_and_lowest_values(cuda_ok):
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    for dtype in TYPES:
        low = torch.finfo(tor(dtype)).min
        for n in (5, 900, 40000):
            x = torch.zeros((8, n), dtype=tor(dtype), device="cuda")
            x[0] = low                      # masked by the lowest value throughout: even
            x[1, 1:] = low                  # one open entry
            x[2] = -float("inf")            # nothing open
            x[3, n - 1] = float("nan")
            x[4, 2] = float("inf")
            x[5, 1:] = -float("inf")        # one open entry, the label closed
            x[6, 3] = low
            labels = ids([0, 0, 0, 0, 0, 1, 0, n])
            lp, norm, st = obj.iso_token_logp(x, labels)
            got, st = wide(lp), st.cpu().numpy()
            assert abs(got[0] + np.log(n)) <= 4e-6 * (1 + np.log(n))
            assert abs(got[1]) <= 4e-6
            assert np.isnan(got[[2, 3, 4, 7]]).all() and got[5] == -np.inf
            assert abs(got[6] + np.log(n - 1)) <= 4e-6 * (1 + np.log(n))
            assert list(st) == [0, 0, 1, 1, 1, 0, 0, 8]
            ones = torch.ones(8, device="cuda")
            d = wide(obj.iso_token_logp_backward(ones, x, labels, norm))
            assert np.isnan(d[2]).all() and np.isnan(d[3]).all()
            assert np.abs(d[1]).max() <= 4e-6
            assert abs(d[0, 0] - (1 - 1 / n)) <= 4e-6 + HALF[dtype] and np.isfinite(d[0]).all()
            assert d[5, 0] == -1 and d[5, 1] == 1 and (d[5, 2:] == 0).all()
            # the neighbours of bad rows are as they are alone
            alone, _, _ = obj.iso_token_logp(x[6:7], labels[6:7])
            assert float(alone) == got[6]


def test_rows_without_labels(cuda_ok):
    """No row, or no labelled row: zeros, and scores of NaN in unlabelled rows do not matter."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x = torch.full((4, 77), float("nan"), device="cuda")
    none = torch.full((4,), float("nan"), device="cuda")
    r = obj.iso_policy_loss(x, ids([-1] * 4), none, none, none, none, kl_coef=0.1)
    assert float(r.loss) == 0 and not r.stats.any() and not r.dlogits.any() and not r.logp.any()
    r = obj.iso_preference_loss(x, ids([-1] * 4), ids([0, 2, 4]), none)
    assert abs(float(r.loss) - np.log(2)) < 1e-6 and not r.dlogits.any() and not r.seq_logp.any()
    e = torch.empty((0, 77), device="cuda")
    z = torch.empty(0, device="cuda")
    zi = torch.empty(0, dtype=torch.int64, device="cuda")
    r = obj.iso_policy_loss(e, zi, z, z)
    assert float(r.loss) == 0 and r.dlogits.shape == (0, 77)
    r = obj.iso_preference_loss(e, zi, ids([0]))
    assert float(r.loss) == 0
    lp, norm, _ = obj.iso_token_logp(e, zi)
    assert lp.shape == (0,) and obj.iso_token_logp_backward(z, e, zi, norm).shape == (0, 77)
    b = obj.iso_balance_loss(e, 3)
    assert float(b.loss) == 0 and int(b.live) == 0 and not b.counts.any()
    assert obj.iso_balance_loss_backward(e, b).shape == (0, 77)


def test_offsets_out_of_order(cuda_ok):
    """A pair whose offsets are out of order or range is flagged and NaN, and nothing is read or
    written outside; the other pairs keep their margins."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(12, 40, "f32", 3, ignored=0.0)
    good = obj.iso_preference_loss(x, ids(labels), ids([0, 3, 6, 9, 12]))
    r = obj.iso_preference_loss(x, ids(labels), ids([0, 3, 6, 9, 1 << 40]))
    assert r.pair_status.tolist() == [0, 4]
    assert float(r.margins[0]) == float(good.margins[0]) and bool(r.margins[1].isnan()) and bool(r.loss.isnan())
    r = obj.iso_preference_loss(x, ids(labels), ids([-5, 3, 6, 9, 12]))
    assert r.pair_status.tolist() == [4, 0] and float(r.margins[1]) == float(good.margins[1])
    r = obj.iso_preference_loss(x, ids(labels), ids([6, 3, 6, 9, 12]))
    assert r.pair_status.tolist() == [4, 0]


def test_gradients_against_differences(cuda_ok):
    """Directional central differences of the losses in float32: step 2e-2, truncation step^2 / 6
    times a third derivative of at most 4, losses off by 2e-6 each."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    step, tol = 2e-2, 4e-4 / 6 * 4 + 2e-6 / 2e-2
    x, xw, labels, rng = make(24, 37, "f32", 11)
    old, adv, base = policy_inputs(xw, labels, rng, 1.0)
    li, args = ids(labels), [put(v) for v in policy_inputs(xw, labels, np.random.default_rng(3), 1.0)]
    # far from the clip's corners: the step moves a ratio by up to step * |direction|
    args[0] = put(np.where(labels >= 0, ref.token_logp(xw, labels) - 0.05 * rng.standard_normal(24), 0))
    mask = torch.ones(24, dtype=torch.uint8, device="cuda")
    gg = put(rng.standard_normal((24, 3)) / 24)
    off = ids([0, 5, 11, 18, 24])

    def direction():
        d = rng.standard_normal(x.shape)
        return put(d / np.sqrt((d * d).sum(1, keepdims=True)))

    def policy(v):
        return obj.iso_policy_loss(v, li, *args, kl_coef=0.2)

    def pref(v):
        return obj.iso_preference_loss(v, li, off, args[2], beta=0.3, label_smoothing=0.1)

    for _ in range(4):
        d = direction()
        for f in (policy, pref):
            num = (float(f(x + step * d).loss) - float(f(x - step * d).loss)) / (2 * step)
            assert abs(num - float((f(x).dlogits.double() * d.double()).sum())) <= tol
    # the router's choice jumps: only directions of small size that change no choice are compared
    x = x.contiguous()
    r = obj.iso_balance_loss(x, 3, mask)
    d = obj.iso_balance_loss_backward(x, r, grad_loss=0.4, grad_gates=gg)
    used = 0
    for _ in range(40):
        u = direction()
        up, down = obj.iso_balance_loss(x + step * u, 3, mask), obj.iso_balance_loss(x - step * u, 3, mask)
        if not (torch.equal(up.experts, r.experts) and torch.equal(down.experts, r.experts)):
            continue
        used += 1
        goal = [0.4 * float(v.loss) + float((v.gates.double() * gg.double()).sum()) for v in (up, down)]
        assert abs((goal[0] - goal[1]) / (2 * step) - float((d.double() * u.double()).sum())) <= tol
    assert used > 0


def test_autograd(cuda_ok):
    """The differentiable calls give the explicit ones' gradients, times the upstream gradient,
    also the second time through a kept graph."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(20, 501, "f32", 5, pad=3)
    li = ids(labels)
    old, adv, base = [put(v) for v in policy_inputs(xw, labels, rng, 0.9)]
    xr = x.detach().clone().requires_grad_()
    x = xr.detach()   # bits are compared: the explicit calls take the very same rows

    def grad(loss, scale):
        return torch.autograd.grad(loss * scale, xr, retain_graph=True)[0]

    lp = obj.token_logp(xr, li, 0.9)
    assert torch.equal(lp.detach(), obj.iso_token_logp(x, li, temperature=0.9)[0])
    g = put(rng.standard_normal(20))
    d = torch.autograd.grad(lp, xr, g)[0]
    assert torch.equal(d, obj.iso_token_logp_backward(g, x, li, obj.iso_token_logp(x, li, temperature=0.9)[1], temperature=0.9))

    r = obj.iso_policy_loss(x, li, old, adv, base, kl_coef=0.1, temperature=0.9)
    loss, stats, logp = obj.policy_loss(xr, li, old, adv, base, kl_coef=0.1, temperature=0.9)
    assert torch.equal(loss.detach(), r.loss) and torch.equal(stats, r.stats) and not logp.requires_grad
    first = grad(loss, 1.0)
    assert torch.equal(first, r.dlogits)
    kept = first.clone()
    second = grad(loss, 3.0)
    assert torch.equal(first, kept)   # the first gradient is the caller's now
    assert torch.allclose(second, 3 * kept, rtol=1e-5, atol=1e-12)
    loss, _, _ = obj.policy_loss(xr, li, old, adv, base, kl_coef=0.1, temperature=0.9)
    assert torch.allclose(grad(loss, -0.25), -0.25 * kept, rtol=1e-5, atol=1e-12)

    off = ids([0, 4, 10, 17, 20])
    r = obj.iso_preference_loss(x, li, off, base)
    loss, margins, _ = obj.preference_loss(xr, li, off, base)
    assert torch.equal(loss.detach(), r.loss) and torch.equal(margins, r.margins)
    assert torch.equal(grad(loss, 1.0), r.dlogits)
    assert torch.allclose(grad(loss, 2.0), 2 * r.dlogits, rtol=1e-5, atol=1e-12)
    with torch.no_grad():
        assert not obj.preference_loss(xr, li, off, base)[0].requires_grad

    b = obj.iso_balance_loss(x, 4)
    loss, gates, counts, experts = obj.balance_loss(xr, 4)
    gg = put(rng.standard_normal((20, 4)))
    d = torch.autograd.grad(0.3 * loss + (gates * gg).sum(), xr)[0]
    want = obj.iso_balance_loss_backward(x, b, grad_loss=0.3, grad_gates=gg)
    assert torch.allclose(d, want, rtol=1e-5, atol=1e-9) and torch.equal(counts, b.counts)
    loss, gates, _, _ = obj.balance_loss(xr, 4)
    d = torch.autograd.grad(gates.sum(), xr)[0]
    assert torch.allclose(d, obj.iso_balance_loss_backward(x, b, grad_loss=0.0, grad_gates=torch.ones_like(gg)), atol=1e-9)


def test_streams_and_graphs(cuda_ok):
    """A side stream given by `stream`, and a captured call replayed on new inputs."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(64, 5000, "bf16", 9)
    li = ids(labels)
    old, adv, base = [put(v) for v in policy_inputs(xw, labels, rng, 1.0)]
    want = obj.iso_policy_loss(x, li, old, adv, base, kl_coef=0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = obj.iso_policy_loss(x, li, old, adv, base, kl_coef=0.1, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    off = ids([0, 10, 30, 50, 64])
    held = torch.zeros_like(x)
    obj.iso_preference_loss(held, li, off, base)
    obj.iso_balance_loss(held[:, :200], 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = obj.iso_policy_loss(held, li, old, adv, base, kl_coef=0.1)
        b = obj.iso_preference_loss(held, li, off, base)
        c = obj.iso_balance_loss(held[:, :200], 4)
        d = obj.iso_balance_loss_backward(held[:, :200], c)
    for _ in range(2):
        held.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(a, want):
            assert torch.equal(u, v)
        assert torch.equal(b.dlogits, obj.iso_preference_loss(x, li, off, base).dlogits)
        e = obj.iso_balance_loss(x[:, :200], 4)
        assert torch.equal(c.counts, e.counts) and torch.equal(d, obj.iso_balance_loss_backward(x[:, :200], e))


def test_rows_far_apart(cuda_ok):
    """Row offsets past 32 bits, in the scores and in the gradient."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    n, stride = 1001, (1 << 31) + 7
    buf = torch.empty(2 * stride + n, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(buf, (3, n), (stride, 1))
    x, xw, labels, rng = make(3, n, "bf16", 21, ignored=0.0)
    far.copy_(x)
    outbuf = torch.empty(2 * stride + n, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(outbuf, (3, n), (stride, 1))
    old, adv, base = [put(v) for v in policy_inputs(xw, labels, rng, 1.0)]
    want = obj.iso_policy_loss(x, ids(labels), old, adv, base, kl_coef=0.1)
    got = obj.iso_policy_loss(far, ids(labels), old, adv, base, kl_coef=0.1, out=out)
    assert abs(float(want.loss) - float(got.loss)) <= 1e-6
    assert (wide(want.dlogits) - wide(out)).__abs__().max() <= 2.0 ** -8 * wide(want.dlogits).__abs__().max()
    b = obj.iso_balance_loss(x, 5)
    bf = obj.iso_balance_loss(far, 5)
    assert torch.equal(b.experts, bf.experts)
    d = obj.iso_balance_loss_backward(far, bf, out=out)
    assert torch.equal(out, obj.iso_balance_loss_backward(x, b)) and d is out


def test_refusals(cuda_ok):
    import torch
    import convex_hull_pava_gb300 as chp
    from convex_hull_pava_gb300 import objectives as obj
    x = torch.zeros((4, 16), device="cuda")
    li, f = ids([0, 1, 2, 3]), torch.zeros(4, device="cuda")

    def no(call, *args, **kw):
        with pytest.raises((ValueError, chp.IsoError)):
            call(*args, **kw)

    no(obj.iso_token_logp, x.double(), li)
    no(obj.iso_token_logp, x.t(), ids([0] * 16))
    no(obj.iso_token_logp, x, li.int())
    no(obj.iso_token_logp, x, li[:3])
    no(obj.iso_token_logp, x, li.cpu())
    no(obj.iso_token_logp, x[:, :0], li)
    no(obj.iso_token_logp, x.view(2, 2, 16), li)
    for t in (0.0, -1.0, float("nan"), float("inf")):
        no(obj.iso_token_logp, x, li, temperature=t)
    lp, norm, _ = obj.iso_token_logp(x, li)
    no(obj.iso_token_logp_backward, f.double(), x, li, norm)
    no(obj.iso_token_logp_backward, f, x, li, norm[:3])
    no(obj.iso_token_logp_backward, f, x, li, norm, out=x.half())
    no(obj.iso_token_logp_backward, f, x, li, norm, out=x[:, :1].expand(4, 16))
    no(obj.iso_token_logp_backward, f, x, li, norm, changed_only=True)
    no(obj.iso_policy_loss, x, li, f[:3], f)
    no(obj.iso_policy_loss, x, li, f, f.half())
    no(obj.iso_policy_loss, x, li, f, f, f.view(2, 2))
    no(obj.iso_policy_loss, x, li, f, f, weights=f.cpu())
    no(obj.iso_policy_loss, x, li, f, f, clip_low=1.5)
    no(obj.iso_policy_loss, x, li, f, f, clip_high=-0.1)
    no(obj.iso_policy_loss, x, li, f, f, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    no(obj.iso_preference_loss, x, li, ids([0, 2, 3, 4]))
    no(obj.iso_preference_loss, x, li, ids([0, 2, 4]).int())
    no(obj.iso_preference_loss, x, li, ids([0, 2, 4]), kind="other")
    no(obj.iso_preference_loss, x, li, ids([0, 2, 4]), beta=0.0)
    no(obj.iso_preference_loss, x, li, ids([0, 2, 4]), label_smoothing=2.0)
    no(obj.iso_preference_loss, x, li, ids([0, 2, 4]), f[:2])
    no(obj.iso_balance_loss, x, 0)
    no(obj.iso_balance_loss, x, 17)
    no(obj.iso_balance_loss, x[0], 1)
    no(obj.iso_balance_loss, torch.zeros((2, 1025), device="cuda"), 2)
    no(obj.iso_balance_loss, x, 2, torch.ones(3, dtype=torch.bool, device="cuda"))
    no(obj.iso_balance_loss, x, 2, torch.ones(4, device="cuda"))
    b = obj.iso_balance_loss(x, 2)
    no(obj.iso_balance_loss_backward, x[:3], b)
    no(obj.iso_balance_loss_backward, x, b, grad_gates=f)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n,ignored", [(5000, 70, 0.3), (4100, 1999, 0.5), (1500, 5003, 0.25), (90, 131072, 0.3),
                                            (1100, 6000, 0.999), (1100, 6000, 0.0)])
def test_many_rows(cuda_ok, rows, n, ignored, dtype):
    """More rows than the GPU takes at once, with and without a label, in one call of each."""
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(rows, n, dtype, seed=rows, ignored=ignored)
    lp, norm, st = obj.iso_token_logp(x, ids(labels))
    want = ref.token_logp(xw, labels)
    assert (np.abs(wide(lp) - want) <= lp_tol(want)).all() and not st.any()
    g = rng.standard_normal(rows).astype(np.float32)
    check_grad(obj.iso_token_logp_backward(put(g), x, ids(labels), norm), xw, labels, g.astype(np.float64),
               np.zeros(rows), dtype)
    old, adv, _ = policy_inputs(xw, labels, rng, 1.0)
    r = obj.iso_policy_loss(x, ids(labels), put(old), put(adv), clip_high=0.3, grad_scale=1024.0)
    loss, stats, lp, coef = ref.policy(xw, labels, old, adv, high=0.3)
    live = labels >= 0
    with np.errstate(all="ignore"):
        size = np.where(live, np.abs(adv) * np.exp(lp - old), 0.0) / max(1, live.sum())
    coef_tol = size * (lp_tol(lp) + 1e-6)
    assert (np.abs(wide(r.coef) - coef) <= coef_tol).all()
    assert abs(float(r.loss) - loss) <= coef_tol.sum() + 1e-6 * abs(loss) + 1e-7
    check_grad(r.dlogits, xw, labels, coef, coef_tol, dtype, 1.0, 1024.0)
    off = np.linspace(0, rows, 2 * min(40, rows // 2) + 1).astype(np.int64)
    r = obj.iso_preference_loss(x, ids(labels), ids(off), beta=0.01, average=True)
    loss, z, seq, lp, coef = ref.preference(xw, labels, off.tolist(), beta=0.01, average=True)
    assert np.abs(wide(r.margins) - z).max() <= 0.02 * lp_tol(lp).max() + 1e-6 * np.abs(z).max()
    assert (np.abs(wide(r.logp) - lp) <= lp_tol(lp)).all()
    check_grad(r.dlogits, xw, labels, coef, 1e-5 * np.abs(coef), dtype)


def test_gradient_over_the_scores(cuda_ok):
    """`out` may be the scores themselves."""
    from convex_hull_pava_gb300 import objectives as obj
    for rows, n, dtype in ((40, 300, "bf16"), (9, 30011, "bf16"), (3, 131072, "f32"), (2, 600011, "bf16")):
        x, xw, labels, rng = make(rows, n, dtype, seed=n)
        old, adv, base = [put(v) for v in policy_inputs(xw, labels, rng, 1.0)]
        want = obj.iso_policy_loss(x, ids(labels), old, adv, base, kl_coef=0.1).dlogits
        y = x.clone()
        obj.iso_policy_loss(y, ids(labels), old, adv, base, kl_coef=0.1, out=y)
        assert bool((y == want).all())
        lp, norm, _ = obj.iso_token_logp(x, ids(labels))
        want = obj.iso_token_logp_backward(adv.nan_to_num(), x, ids(labels), norm)
        y = x.clone()
        obj.iso_token_logp_backward(adv.nan_to_num(), y, ids(labels), norm, out=y)
        assert bool((y == want).all())


def test_example_runs(cuda_ok):
    """The example that trains on calibrated, ranked rewards."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "post_training.py")
    spec = importlib.util.spec_from_file_location("post_training", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = np.array(example.main(6))
    assert history.shape == (6, 3) and np.isfinite(history).all()
    # balance is 1 when even; a sigmoid preference loss is positive
    assert (history[:, 1] > 0.9).all() and (history[:, 2] > 0).all()


def test_kernel_times_can_be_read(cuda_ok):
    """The library's per-kernel timing covers these calls."""
    import torch
    import convex_hull_pava_gb300 as chp
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(2000, 700, "f32", 2)
    li, off = ids(labels), ids([0, 500, 1000, 1700, 2000])
    zero = torch.zeros(2000, device="cuda")
    chp.profile_enable(True)
    try:
        seen = []
        for call in (lambda: obj.iso_policy_loss(x, li, zero, zero), lambda: obj.iso_preference_loss(x, li, off),
                     lambda: obj.iso_balance_loss(x, 4)):
            call()
            times = chp.profile_read()
            seen.append([name for name, _ in times])
            assert all(ms >= 0 for _, ms in times)
    finally:
        chp.profile_enable(False)
    assert seen[0][-1] == "policy_rows" and seen[1][-1] == "score_backward" and seen[2] == ["balance_tokens", "balance_finish"]


def test_more_rows_than_a_grid_dimension(cuda_ok):
    """Over 65,535 rows, of one CTA and of one warp each."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    for rows, n in ((66000, 2600), (530000, 9)):
        x = torch.randn((rows, n), device="cuda", dtype=torch.bfloat16)
        labels = torch.randint(-1, n, (rows,), device="cuda")
        g = torch.randn(rows, device="cuda")
        lp, norm, _ = obj.iso_token_logp(x, labels)
        want = torch.log_softmax(x.double(), 1)
        at = want.gather(1, labels.clamp(min=0)[:, None])[:, 0].where(labels >= 0, 0)
        assert bool(((lp - at).abs() <= 4e-6 * (1 + at.abs())).all())
        d = want.exp_().mul_(-g.double()[:, None])
        d.scatter_add_(1, labels.clamp(min=0)[:, None], g.double()[:, None])
        d[labels < 0] = 0
        got = obj.iso_token_logp_backward(g, x, labels, norm).double()
        # half a unit of bfloat16 relative, and the probabilities' error
        assert bool(((got - d).abs() <= 2.0 ** -8 * d.abs() + 5e-6 * g.double().abs()[:, None]).all())
