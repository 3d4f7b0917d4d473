"""The 64-bit forms of the training objectives against differences and closed forms, and the
library's host-side argument checks (no GPU)."""
import ctypes

import numpy as np
import pytest

import convex_hull_pava_gb300 as chp
import objectives_ref as ref

STEP = 1e-5
# central differences in float64: STEP^2 third derivatives + 2^-52 / STEP rounding, scaled by
# values of about 10
TOL = 1e-8


def differences(f, x):
    d = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        if not np.isfinite(x[i]):
            continue
        up, down = x.copy(), x.copy()
        up[i] += STEP
        down[i] -= STEP
        d[i] = (f(up) - f(down)) / (2 * STEP)
    return d


def scores(rows, n, seed=0, closed=True):
    rng = np.random.default_rng(seed)
    x = 1.5 * rng.standard_normal((rows, n))
    if closed and n > 3:
        x[:, 2] = -np.inf
    labels = rng.integers(0, 2 if n > 2 else n, rows)
    labels[1 % rows] = -100 if rows > 1 else labels[0]
    return rng, x, labels


@pytest.mark.parametrize("t", [1.0, 0.7])
@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient(t, kl):
    rng, x, labels = scores(6, 5)
    lp = ref.token_logp(x, labels, t)
    old, adv, base = lp + 0.3 * rng.standard_normal(6), rng.standard_normal(6), lp + 0.4 * rng.standard_normal(6)
    args = (labels, old, adv, base if kl else None)
    coef = ref.policy(x, *args, kl_coef=kl, t=t)[3]
    d, _ = ref.grad_logits(coef, x, labels, t)
    assert np.abs(d - differences(lambda v: ref.policy(v, *args, kl_coef=kl, t=t)[0], x)).max() <= TOL


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient(kind, average):
    rng, x, labels = scores(9, 5, 1)
    off = [0, 3, 5, 5, 9]   # one empty sequence
    base = ref.token_logp(x, labels) + 0.3 * rng.standard_normal(9)
    kw = dict(kind=kind, beta=0.6, smooth=0.1 if kind == "sigmoid" else 0.0, average=average)
    coef = ref.preference(x, labels, off, base, **kw)[4]
    d, _ = ref.grad_logits(coef, x, labels)
    num = differences(lambda v: ref.preference(v, labels, off, base, **kw)[0], x)
    assert np.abs(d - num).max() <= TOL * 10


@pytest.mark.parametrize("renormalize", [False, True])
def test_balance_gradient(renormalize):
    rng, x, _ = scores(6, 7, 2)
    x[4] = -np.inf
    mask = np.array([1, 1, 0, 1, 1, 1])
    g = rng.standard_normal((6, 3))

    def goal(v):
        loss, _, _, gates, _ = ref.balance(v, 3, mask, renormalize)
        return 0.7 * loss + (gates * g).sum()

    d = ref.balance_grad(x, 3, mask, renormalize, 0.7, g)
    assert np.abs(d - differences(goal, x)).max() <= TOL
    loss, counts, experts, gates, live = ref.balance(x, 3, mask, renormalize)
    assert live == 4 and counts.sum() == 12 and (experts[[2, 4]] == -1).all()


def test_even_router_has_loss_one():
    x = np.log(np.ones((8, 4)))
    for t in range(8):
        x[t, t % 4] += 1e-9
    assert abs(ref.balance(x, 1)[0] - 1.0) < 1e-6


def test_objective_argument_checks():
    """Refused before any CUDA call."""
    lib = chp.load_library()
    p, ws = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x100000)
    bad, no_ws = chp.ISO_ERR_INVALID_ARG, chp.ISO_ERR_WORKSPACE

    need0 = lib.iso_token_logp_workspace_bytes(4000)
    assert need0 > 0 and lib.iso_token_logp_workspace_bytes(-1) == 0 and lib.iso_token_logp_workspace_bytes(1) == 0

    def logp(x=p, dt=0, rows=4000, n=10, stride=10, labels=p, t=1.0, lp=p, norm=p, w=ws, wb=need0):
        return lib.iso_token_logp(x, dt, rows, n, stride, labels, t, lp, norm, w, wb, None, None)

    assert logp(rows=0, x=None, labels=None, lp=None, norm=None) == chp.ISO_OK
    for kw in (dict(x=None), dict(dt=3), dict(dt=-1), dict(rows=-1), dict(n=0), dict(n=1 << 31), dict(stride=-1),
               dict(rows=1 << 31), dict(rows=1 << 30, stride=1 << 30), dict(labels=None), dict(t=0.0), dict(t=-1.0),
               dict(t=float("nan")), dict(t=float("inf")), dict(t=1e-39), dict(lp=None), dict(norm=None)):
        assert logp(**kw) == bad, kw
    for kw in (dict(w=None), dict(wb=need0 - 1), dict(w=ctypes.c_void_p(0x100010))):
        assert logp(**kw) == no_ws, kw

    def back(x=p, norm=p, g=p, changed=0, out=p, out_stride=10, n=10):
        return lib.iso_token_logp_backward(x, 1, 4, n, 10, p, 1.0, norm, g, 1.0, None, changed, out, out_stride, None)

    for kw in (dict(x=None), dict(norm=None), dict(g=None), dict(changed=2), dict(out=None), dict(out_stride=9), dict(n=0)):
        assert back(**kw) == bad, kw

    need = lib.iso_policy_loss_workspace_bytes(4)
    assert need > 0 and lib.iso_policy_loss_workspace_bytes(-1) == 0

    def policy(x=p, old=p, adv=p, lo=0.2, hi=0.2, loss=p, stats=p, coef=p, out=p, out_stride=10, w=ws, wb=need):
        return lib.iso_policy_loss(x, 0, 4, 10, 10, p, 1.0, old, adv, None, None, lo, hi, 0.0, 1.0, loss, stats, p, p,
                                   coef, out, out_stride, w, wb, None, None)

    for kw in (dict(x=None), dict(old=None), dict(adv=None), dict(lo=-0.1), dict(lo=1.5), dict(hi=-1.0),
               dict(lo=float("nan")), dict(loss=None), dict(stats=None), dict(coef=None), dict(out_stride=3)):
        assert policy(**kw) == bad, kw
    for kw in (dict(w=None), dict(wb=need - 1), dict(w=ctypes.c_void_p(0x100010))):
        assert policy(**kw) == no_ws, kw

    need2 = lib.iso_preference_loss_workspace_bytes(4, 2)
    assert need2 > 0 and lib.iso_preference_loss_workspace_bytes(4, -1) == 0

    def pref(x=p, off=p, pairs=2, kind=0, beta=0.1, smooth=0.0, avg=0, loss=p, margins=p, seq=p, coef=p, w=ws, wb=need2):
        return lib.iso_preference_loss(x, 2, 4, 10, 10, p, off, pairs, None, kind, beta, smooth, avg, 1.0, loss,
                                       margins, seq, p, p, coef, p, 10, w, wb, None, None, None)

    for kw in (dict(x=None), dict(off=None), dict(pairs=-1), dict(kind=3), dict(kind=-1), dict(beta=0.0),
               dict(beta=float("nan")), dict(smooth=-0.1), dict(smooth=1.1), dict(avg=2), dict(loss=None),
               dict(margins=None), dict(seq=None), dict(coef=None)):
        assert pref(**kw) == bad, kw
    for kw in (dict(w=None), dict(wb=need2 - 1)):
        assert pref(**kw) == no_ws, kw

    need3 = lib.iso_balance_loss_workspace_bytes(4, 10)
    assert need3 > 0 and lib.iso_balance_loss_workspace_bytes(4, 1025) == 0

    def balance(x=p, n=10, k=2, renorm=0, loss=p, counts=p, chosen=p, gates=p, live=p, w=ws, wb=need3, stride=None):
        return lib.iso_balance_loss(x, 0, 4, n, stride or n, k, None, renorm, loss, counts, chosen, gates, live, w, wb, None)

    for kw in (dict(x=None), dict(n=0), dict(n=1025), dict(k=0), dict(k=11), dict(n=64, k=33), dict(renorm=2),
               dict(loss=None), dict(counts=None), dict(chosen=None), dict(gates=None), dict(live=None)):
        assert balance(**kw) == bad, kw
    for kw in (dict(w=None), dict(wb=need3 - 1)):
        assert balance(**kw) == no_ws, kw

    def balance_back(x=p, counts=p, gates=p, out=p, out_stride=10, k=2):
        return lib.iso_balance_loss_backward(x, 0, 4, 10, 10, k, None, 0, counts, p, gates, p, None, 1.0, None, out,
                                             out_stride, None)

    for kw in (dict(x=None), dict(counts=None), dict(gates=None), dict(out=None), dict(out_stride=9), dict(k=0)):
        assert balance_back(**kw) == bad, kw


def test_objective_bindings_refuse_host_tensors():
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x, labels = torch.zeros(2, 4), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        obj.iso_token_logp(x, labels)
    with pytest.raises(ValueError):
        obj.iso_policy_loss(x, labels, torch.zeros(2), torch.zeros(2))
    with pytest.raises(ValueError):
        obj.iso_preference_loss(x, labels, torch.tensor([0, 1, 2]))
    with pytest.raises(ValueError):
        obj.iso_balance_loss(x, 2)
