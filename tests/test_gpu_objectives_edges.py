"""The training objectives on the GPU where scores, places and offsets are out of the ordinary,
against their 64-bit forms.  Tolerances are those derived in test_gpu_objectives.py unless a test
says otherwise."""
import numpy as np
import pytest

import objectives_ref as ref
from test_gpu_objectives import HALF, TINY, check_grad, ids, lp_tol, make, policy_inputs, put, tor, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,n,k", [(9, 5, 2), (1000, 64, 3), (700, 256, 8), (33, 1000, 32)])
def test_router_gradient_over_the_scores(cuda_ok, tokens, n, k, dtype):
    """A router's gradient written over its scores is the one written elsewhere."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    rng = np.random.default_rng(n)
    for renormalize in (False, True):
        x = put(rng.standard_normal((tokens, n)), dtype)
        gg = put(rng.standard_normal((tokens, k)))
        r = obj.iso_balance_loss(x, k, renormalize=renormalize)
        want = obj.iso_balance_loss_backward(x, r, grad_loss=0.5, grad_gates=gg)
        y = x.clone()
        assert obj.iso_balance_loss_backward(y, r, grad_loss=0.5, grad_gates=gg, out=y) is y
        assert torch.equal(y, want)


@pytest.mark.parametrize("rows,n,dtype", [(40, 300, "bf16"), (9, 30011, "bf16"), (300, 2049, "f16"), (4, 131072, "f32")])
def test_preference_gradient_over_the_scores(cuda_ok, rows, n, dtype):
    """A preference loss's gradient written over its scores is the one written elsewhere."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(rows, n, dtype, seed=n)
    off = ids(np.linspace(0, rows, 5).astype(np.int64))
    want = obj.iso_preference_loss(x, ids(labels), off)
    y = x.clone()
    got = obj.iso_preference_loss(y, ids(labels), off, out=y)
    assert got.dlogits is y and torch.equal(y, want.dlogits) and torch.equal(got.loss, want.loss)


@pytest.mark.parametrize("offsets,status,as_if", [
    ([0, 6, 3, 6, 9], [4, 0], [3, 3, 3, 6, 9]),                     # a pair out of order over a good one's rows
    ([0, 3, 6, 9, 3, 5, 9], [0, 4, 4], [0, 3, 6, 6, 6, 6, 6]),      # two in order about one that is not
    ([5, 2, 5, 7, 9, 1 << 40, 0, 3, 5], [4, 0, 4, 4], [5, 5, 5, 7, 9, 9, 9, 9, 9]),   # the last starts before the second
    ([9, 9, 9, 3, 3, 6, 9], [0, 4, 0], [3, 3, 3, 3, 3, 6, 9]),      # an empty one holds no rows
    ([0, 3, 6, 9, 4, 4, 4], [0, 4, 0], [0, 3, 6, 6, 6, 6, 6]),
    ([0, 3, 6, 9, 6, 6, 6, 8, 12], [0, 4, 0, 0], [0, 3, 6, 6, 6, 6, 6, 8, 12]),
])
def test_pairs_that_share_rows(cuda_ok, offsets, status, as_if):
    """Each row's coefficient is that of the one pair that may write it, whatever the others' offsets
    are: the same bits as where the flagged pairs are empty."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(12, 40, "f32", 3, ignored=0.0)
    base = put(ref.token_logp(xw, labels) + 0.2 * rng.standard_normal(12))
    want = obj.iso_preference_loss(x, ids(labels), ids(as_if), base, beta=0.3)
    assert not want.pair_status.any() and bool((want.coef != 0).any())
    for _ in range(5):
        r = obj.iso_preference_loss(x, ids(labels), ids(offsets), base, beta=0.3)
        assert r.pair_status.tolist() == status
        assert r.margins.isnan().tolist() == [s != 0 for s in status] and bool(r.loss.isnan())
        assert r.seq_logp.isnan().tolist() == [s != 0 for s in status for _ in range(2)]
        assert torch.equal(r.coef, want.coef) and torch.equal(r.dlogits, want.dlogits)


def test_many_pairs_out_of_order(cuda_ok):
    """More pairs than the GPU takes at once, of which some are out of order: whatever CTA has a pair, it
    knows the rows before it."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    rng = np.random.default_rng(9)
    pairs, rows = 3000, 9000
    off = np.sort(rng.integers(0, rows + 1, 2 * pairs + 1))
    off[rng.integers(0, 2 * pairs, 300)] += rng.integers(-12, 13, 300)
    off[77], off[5000] = -5, rows + 1
    x, xw, labels, _ = make(rows, 20, "f32", 6)
    status, last = [], 0
    for q in range(pairs):
        a, b, c = off[2 * q:2 * q + 3]
        order = 0 <= a <= b <= c <= rows
        status.append(0 if order and (a == c or a >= last) else 4)
        if order and a < c:
            last = max(last, c)
    r = obj.iso_preference_loss(x, ids(labels), ids(off), beta=0.5)
    assert r.pair_status.tolist() == status and 10 < np.count_nonzero(status) < pairs
    assert torch.equal(r.margins.isnan().cpu(), torch.tensor(status) != 0) and bool(r.loss.isnan())
    # the coefficients that are left: each row's of the pair that holds it
    want = np.zeros(rows)
    lp = ref.token_logp(xw, labels)
    for q in np.flatnonzero(np.array(status) == 0):
        a, b, c = off[2 * q:2 * q + 3]
        z = 0.5 * (lp[a:b].sum() - lp[b:c].sum())
        slope = -0.5 / (1 + np.exp(z)) / pairs
        want[a:b], want[b:c] = slope, -slope
    want[labels < 0] = 0
    # a margin is beta times its tokens' log-probabilities (at most 40), a coefficient's slope in it beta / 4
    assert np.abs(wide(r.coef) - want).max() <= (0.5 / 4 * 0.5 * 40 * lp_tol(lp).max() + 1e-6) / pairs


def test_many_pairs(cuda_ok):
    """More pairs than a grid has CTAs, most of them short or empty, in order."""
    from convex_hull_pava_gb300 import objectives as obj
    rng = np.random.default_rng(8)
    sizes = rng.integers(0, 3, 2 * 1500)
    off = np.concatenate([[0], np.cumsum(sizes)])
    x, xw, labels, _ = make(int(off[-1]), 50, "f32", 5)
    r = obj.iso_preference_loss(x, ids(labels), ids(off), beta=0.5)
    loss, z, seq, lp, coef = ref.preference(xw, labels, off.tolist(), beta=0.5)
    assert not r.pair_status.any()
    # a margin is beta times at most four log-probabilities; a coefficient's slope in it is at most beta / 4
    off_by = 0.5 * 4 * lp_tol(lp).max() + 1e-6 * np.abs(z).max()
    assert np.abs(wide(r.margins) - z).max() <= off_by
    assert np.abs(wide(r.coef) - coef).max() <= (0.5 / 4 * off_by + 1e-6 * 0.5) / 1500


# Sizes of scores between the ordinary ones and the type's lowest value: masks by a large negative
# number, large positive scores, and ordinary scores at a small temperature.
FAR = [1e4, -1e4, 1e5, -1e5, 1e7, -1e7, 3e8, -1e9, -1e10, 1e12, -1e12, -1e20, 1e29, -3e30]


def far_rows(n, dtype, rng, sizes=FAR):
    """Two rows for each of the sizes that the type holds: about it throughout, and about it with some
    entries elsewhere (below a large score, above a mask).  The last entries are closed."""
    import torch
    most = torch.finfo(tor(dtype)).max
    step = {"f32": 2.0 ** -23, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]
    rows = []
    for size in [v for v in sizes if abs(v) < most / 2]:
        unit = 2.0 ** np.floor(np.log2(abs(size))) * step     # neighbouring numbers of the type
        even = size + unit * np.round(3 * rng.random(n)) * (unit < 4)
        other = even.copy()
        other[: (n + 1) // 3] = -abs(size) * rng.uniform(0.5, 1.0, (n + 1) // 3) if size > 0 else \
            3.0 * rng.standard_normal((n + 1) // 3)
        for row in (even, other):
            row = row.copy()
            if n > 4:
                row[-(n // 8) - 1:] = -np.inf
            rows.append(row)
    x = put(np.array(rows), dtype)
    return x, wide(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [1, 4, 33, 1000, 8191, 40000, 600011])
def test_scores_of_any_size(cuda_ok, n, dtype):
    """Log-probabilities, policy and preference losses of rows of large scores, at temperatures that
    make them larger, and of ordinary rows at a small temperature.

    The exponent of a term is (x - m) / T in base 2 whatever m is, off by 2^-22 of itself; log p is off by
    that of the label's, within LP as elsewhere."""
    from convex_hull_pava_gb300 import objectives as obj
    rng = np.random.default_rng(n)
    long_ = n > 100000   # (fewer of these)
    x, xw = far_rows(n, dtype, rng, [1e4, -1e4, -1e9] if long_ else FAR)
    rows = len(xw)
    plain = put(3.0 * rng.standard_normal((rows, n)), dtype)
    for v, w, temperatures in ((x, xw, (0.3,) if long_ else (1.0, 0.3, 50.0)), (plain, wide(plain), (1e-5,) if long_ else (1e-3, 1e-5))):
        # a label near the top (the others have no probability in 32 bits)
        labels = np.array([rng.choice(np.flatnonzero(r >= r.max() - 1e-6 * abs(r.max()))) for r in w])
        li = ids(labels)
        for t in temperatures:
            want = ref.token_logp(w, labels, t)
            lp, norm, st = obj.iso_token_logp(v, li, temperature=t)
            assert not st.any() and (np.abs(wide(lp) - want) <= lp_tol(want)).all(), (t, wide(lp), want)
            g = rng.standard_normal(rows).astype(np.float32)
            d = obj.iso_token_logp_backward(put(g), v, li, norm, temperature=t, grad_scale=t)
            check_grad(d, w, labels, g.astype(np.float64), np.zeros(rows), dtype, t, t)
            old, adv, base = policy_inputs(w, labels, rng, t)
            r = obj.iso_policy_loss(v, li, put(old), put(adv), put(base), clip_high=0.3, kl_coef=0.1, temperature=t,
                                    grad_scale=t)
            loss, stats, plp, coef = ref.policy(w, labels, old, adv, base, None, 0.2, 0.3, 0.1, t)
            assert not r.row_status.any() and (np.abs(wide(r.logp) - plp) <= lp_tol(plp)).all()
            size = np.abs(adv) * np.exp(plp - old) + 0.1 * np.exp(base - plp)
            coef_tol = size / rows * (lp_tol(plp) + 1e-6)
            assert (np.abs(wide(r.coef) - coef) <= coef_tol).all()
            check_grad(r.dlogits, w, labels, coef, coef_tol, dtype, t, t)
        # three sequences of one row each and one of all the rest
        off = np.arange(5).tolist()
        off[4] = rows
        want, z, seq, lp, coef = ref.preference(w, labels, off, beta=0.1)
        r = obj.iso_preference_loss(v, li, ids(off), beta=0.1)
        z_tol = 0.1 * lp_tol(lp).sum() + 1e-6 * np.abs(z).max()
        assert np.abs(wide(r.margins) - z).max() <= z_tol and abs(float(r.loss) - want) <= z_tol + 1e-6 * abs(want)
        check_grad(r.dlogits, w, labels, coef, 0.05 / 4 * z_tol + 1e-6 * np.abs(coef), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_states_of_far_and_near_scores_meet(cuda_ok, dtype):
    """Rows whose stretches hold scores on both sides of where exponents are formed another way (about
    2,800 at a temperature of 1): each thread's, warp's and CTA's sums are against a score of their own."""
    from convex_hull_pava_gb300 import objectives as obj
    rng = np.random.default_rng(4)
    for n in (70, 3000, 66000, 600011):
        for sign in (1, -1):
            row = sign * 2839.0 + rng.uniform(-6.0, 6.0, (6, n))
            row[1, : n // 2] -= 8.0
            row[2, n // 2:] -= 8.0
            row[3] = np.sort(row[3])
            row[4] = np.sort(row[4])[::-1]
            row[5, ::7] = -5000.0
            x = put(row, dtype)
            w = wide(x)
            labels = w.argmax(1)
            lp, norm, st = obj.iso_token_logp(x, ids(labels))
            want = ref.token_logp(w, labels)
            assert not st.any() and (np.abs(wide(lp) - want) <= lp_tol(want)).all()
            one = put(np.ones(6))
            zero = put(np.zeros(6))
            r = obj.iso_policy_loss(x, ids(labels), put(want), one, want_grad=False)
            assert (np.abs(wide(r.logp) - want) <= lp_tol(want)).all()
            check_grad(obj.iso_token_logp_backward(one, x, ids(labels), norm), w, labels, np.ones(6), np.zeros(6), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k", [(4, 2), (16, 3), (32, 1), (64, 8), (256, 8), (300, 32), (1000, 4)])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_scores_of_any_size(cuda_ok, n, k, renormalize, dtype):
    """A router's tokens with large scores beside ordinary ones: choice, gates, loss and gradient."""
    from convex_hull_pava_gb300 import objectives as obj
    rng = np.random.default_rng(n)
    far, fw = far_rows(n, dtype, rng)
    x = put(np.concatenate([fw, rng.standard_normal((20, n))]), dtype)
    xw = wide(x)
    r = obj.iso_balance_loss(x, k, renormalize=renormalize)
    loss, counts, experts, gates, live = ref.balance(xw, k, None, renormalize)
    assert int(r.live) == live and np.array_equal(r.counts.cpu().numpy(), counts)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.abs(wide(r.gates) - gates).max() <= 4e-6
    assert abs(float(r.loss) - loss) <= 1e-5 * (1 + abs(loss))
    gg = rng.standard_normal((len(xw), k)).astype(np.float32)
    d = obj.iso_balance_loss_backward(x, r, grad_loss=0.5, grad_gates=put(gg))
    want = ref.balance_grad(xw, k, None, renormalize, 0.5, gg.astype(np.float64))
    top = np.abs(gg).max() + 0.5 * n * counts.max() / (k * live * live)
    assert np.abs(wide(d) - want).max() <= 1e-5 * top + (HALF[dtype] * np.abs(want)).max() + TINY[dtype]


# (scores' width, scores a row, gradient's width, type): the scores' rows start where 128 bytes do, the
# gradient's do not, and the row's last words are near the end of a CTA's (or a warp's) share.
LAYOUTS = [(16384, 8191, 8191, "bf16"), (8192, 8192, 8193, "bf16"), (8192, 8185, 8191, "f16"), (131072, 131071, 131071, "bf16"),
           (4096, 1023, 1023, "f32"), (4096, 4093, 4093, "f32"), (4096, 4096, 4097, "f32"), (2048, 2048, 2049, "bf16"),
           (64, 17, 19, "f16"), (16384, 16381, 16387, "f16")]


@pytest.mark.parametrize("width,n,out_width,dtype", LAYOUTS)
def test_gradient_aligned_otherwise_than_the_scores(cuda_ok, width, n, out_width, dtype):
    """A gradient whose rows start at other places within 16 bytes than the scores': all of every row is
    written, zeros where the row has no label, and nothing else."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    rows = 40
    rng = np.random.default_rng(n)
    buf = torch.full((rows, width), float("nan"), dtype=tor(dtype), device="cuda")
    x = buf[:, :n]
    x.copy_(put(2.0 * rng.standard_normal((rows, n)), dtype))
    xw = wide(x)
    labels = rng.integers(0, n, rows)
    labels[rng.permutation(rows)[: rows // 2]] = -100
    li = ids(labels)
    lp, norm, _ = obj.iso_token_logp(x, li)
    g = rng.standard_normal(rows).astype(np.float32)
    lp_ = ref.token_logp(xw, labels)
    off = ids([0, 10, 20, 30, 40])

    def poisoned():
        t = torch.full((rows, out_width), float("nan"), dtype=tor(dtype), device="cuda")
        return t, t[:, :n]

    live = labels >= 0
    shares = ref.preference(xw, labels, [0, 10, 20, 30, 40])[4]
    ratio = np.where(live, -g / max(1, live.sum()), 0.0)   # (old is lp: a ratio of 1)
    for call, coef, coef_tol in (
            (lambda out: obj.iso_token_logp_backward(put(g), x, li, norm, out=out), g.astype(np.float64), np.zeros(rows)),
            # a margin's error is beta times those of its tokens, a coefficient's beta / 4 / pairs times that
            (lambda out: obj.iso_preference_loss(x, li, off, out=out), shares,
             0.1 / 4 / 2 * 0.1 * lp_tol(lp_)[live].sum() + 1e-6 * np.abs(shares)),
            (lambda out: obj.iso_policy_loss(x, li, put(lp_), put(g), out=out), ratio, np.abs(ratio) * (lp_tol(lp_) + 1e-6))):
        whole, out = poisoned()
        call(out)
        assert bool((out[li < 0] == 0).all())
        assert bool(whole[:, n:].isnan().all())
        check_grad(out, xw, labels, coef, coef_tol, dtype)


def test_outputs_of_no_rows(cuda_ok):
    """Of an empty batch every output is empty."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    e = torch.empty((0, 77), device="cuda")
    z = torch.empty(0, device="cuda")
    zi = torch.empty(0, dtype=torch.int64, device="cuda")
    for r in (obj.iso_policy_loss(e, zi, z, z), obj.iso_preference_loss(e, zi, ids([0])),
              obj.iso_preference_loss(e, zi, ids([0, 0, 0]))):
        assert r.norm.shape == (0, 2) and r.coef.shape == (0,) and r.row_status.shape == (0,) and r.logp.shape == (0,)
        assert not r.row_status.any() and len(list(r)) == len(r)
    assert r.pair_status.tolist() == [0] and r.margins.tolist() == [0.0]


def test_router_sums_over_many_tokens(cuda_ok):
    """The probabilities of 2^26 equal tokens: their sum is exact up to 64 additions in float32 (2^-25
    each, 1.9e-6 in all), a probability's error (4e-7) and the loss's last roundings (2e-7)."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    row = torch.tensor([0.3, -0.2, 0.75, -1.0], device="cuda", dtype=torch.bfloat16)
    x = row.repeat(1 << 26, 1)
    r = obj.iso_balance_loss(x, 1)
    p = float(torch.softmax(row.double(), 0)[2])
    assert r.counts.tolist() == [0, 0, 1 << 26, 0] and int(r.live) == 1 << 26
    assert abs(float(r.loss) - 4 * p) <= 3e-6 * 4 * p
    # and of tokens that one CTA takes alone
    r = obj.iso_balance_loss(x[:7], 1)
    assert abs(float(r.loss) - 4 * p) <= 3e-6 * 4 * p


def test_first_calls_from_several_threads(cuda_ok):
    """A process's first calls, from several threads at once, each on a stream of its own."""
    import os
    import subprocess
    import sys
    program = """
import threading
import torch
from convex_hull_pava_gb300 import objectives as obj
g = torch.Generator(device="cuda").manual_seed(1)
x = [torch.randn((n, v), device="cuda", generator=g) for n, v in ((70, 900), (90, 9000), (30, 70000), (5, 300001))]
labels = [torch.arange(len(v), device="cuda") % 7 for v in x]
zero = [torch.zeros(len(v), device="cuda") for v in x]
torch.cuda.synchronize()
got, at = [None] * 8, threading.Barrier(8)

def run(i):
    at.wait()
    with torch.cuda.stream(torch.cuda.Stream()):
        got[i] = [t for v, l, z in zip(x, labels, zero)
                  for t in (obj.iso_token_logp(v, l)[0], obj.iso_policy_loss(v, l, z, z + 1).dlogits, obj.iso_balance_loss(v[:, :64], 4).loss)]
        torch.cuda.current_stream().synchronize()

threads = [threading.Thread(target=run, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_no_second_derivatives(cuda_ok):
    """The gradients carry no graph of their own: a second derivative is refused, not left out."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x = torch.randn((6, 9), device="cuda", requires_grad=True)
    labels, zero = ids([0, 1, 2, 3, 4, 5]), torch.zeros(6, device="cuda")
    for loss in (lambda: obj.token_logp(x, labels).square().sum(), lambda: obj.policy_loss(x, labels, zero, zero + 1)[0],
                 lambda: obj.preference_loss(x, labels, ids([0, 3, 6]))[0], lambda: obj.balance_loss(x, 2)[1].square().sum()):
        first, = torch.autograd.grad(loss(), x)
        again, = torch.autograd.grad(loss(), x, create_graph=True)
        assert torch.equal(first, again)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(again.square().sum() + x.square().sum(), x)


def test_infinite_margins(cuda_ok):
    """A sequence with a token of probability 0: the pair's loss is its formula's limit, in which a term
    that the smoothing gives no weight has no part."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x = torch.zeros((4, 8), device="cuda")
    x[:, 5] = -float("inf")
    for rejected, chosen in ((5, 1), (1, 5)):
        labels, off = ids([chosen, rejected, 2, 3]), ids([0, 1, 2, 3, 4])
        sign = 1.0 if rejected == 5 else -1.0
        for smooth, want in ((0.0, 0.0 if sign > 0 else np.inf), (1.0, np.inf if sign > 0 else 0.0), (0.1, np.inf)):
            r = obj.iso_preference_loss(x, labels, off, beta=0.5, label_smoothing=smooth)
            assert r.margins.tolist() == [sign * np.inf, 0.0]
            got = float(r.loss)
            assert got == np.inf if want == np.inf else abs(got - np.log(2) / 2) <= 1e-6
            # the slope: -(1 - smooth) sigmoid(-z) + smooth sigmoid(z), halved over the pairs, times beta
            slope = 0.25 * (smooth if sign > 0 else smooth - 1.0)
            assert np.abs(wide(r.coef)[:2] - [slope, -slope]).max() <= 1e-6


def test_kl_term_without_weight(cuda_ok):
    """A KL weight of 0 leaves no KL term, however far the reference's log-probability is (its
    exponential leaves float32's range)."""
    from convex_hull_pava_gb300 import objectives as obj
    x, labels, lp = put(np.zeros((4, 6))), ids([0, 1, 2, 3]), float(-np.log(6.0))
    base = put([lp, lp + 150.0, lp, lp])
    r = obj.iso_policy_loss(x, labels, put([lp] * 4), put([1.0] * 4), base, kl_coef=0.0)
    # a ratio of 1: off by the log-probability's 1e-5
    assert abs(float(r.loss) + 1.0) <= 2e-5 and np.abs(wide(r.coef) + 0.25).max() <= 0.25 * 2e-5
    assert float(r.stats[1]) == np.inf and bool(r.dlogits.isfinite().all())


def test_advantage_of_zero(cuda_ok):
    """An advantage of 0 leaves no policy term, however small the old probability is (the ratio leaves
    float32's range)."""
    from convex_hull_pava_gb300 import objectives as obj
    x, labels, lp = put(np.zeros((4, 6))), ids([0, 1, 2, 3]), float(-np.log(6.0))
    r = obj.iso_policy_loss(x, labels, put([lp, lp - 200.0, lp, lp - 200.0]), put([1.0, 0.0, -1.0, -0.0]))
    assert abs(float(r.loss)) <= 1e-5 and wide(r.coef).tolist()[1::2] == [0.0, 0.0]
    assert np.abs(wide(r.coef)[[0, 2]] - [-0.25, 0.25]).max() <= 1e-5 and not wide(r.dlogits)[1::2].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_labels_past_the_end(cuda_ok, dtype):
    """A label that is not below n: no log-probability and no gradient, in every call."""
    from convex_hull_pava_gb300 import objectives as obj
    for n in (7, 900, 9000):
        x, xw, labels, rng = make(9, n, dtype, seed=n, ignored=0.0)
        good = ids(labels)
        labels[[1, 4, 8]] = [n, n + 7, 1 << 40]
        bad = np.isin(np.arange(9), [1, 4, 8])
        li, one = ids(labels), put(np.ones(9))
        lp, norm, st = obj.iso_token_logp(x, li)
        assert np.array_equal(np.isnan(wide(lp)), bad) and np.array_equal(st.cpu().numpy(), 8 * bad)
        d = wide(obj.iso_token_logp_backward(one, x, li, norm))
        want = wide(obj.iso_token_logp_backward(one, x, good, norm))
        assert np.isnan(d[bad]).all() and np.array_equal(d[~bad], want[~bad])
        r = obj.iso_policy_loss(x, li, one, one)
        assert np.isnan(wide(r.dlogits)[bad]).all() and np.isfinite(wide(r.dlogits)[~bad]).all()
        r = obj.iso_preference_loss(x, li, ids([0, 1, 2, 3, 4, 5, 6, 7, 8]))
        assert r.margins.isnan().tolist() == [True, False, True, False]


@pytest.mark.parametrize("n", [4, 8, 16, 30, 64, 256, 600])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_scores_of_nan(cuda_ok, n, renormalize):
    """A NaN or +inf makes the gates and the gradient of its token NaN, at any number of experts, and the
    loss; the other tokens are as they are alone."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x = torch.randn((40, n), device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    want = obj.iso_balance_loss(x, 3, renormalize=renormalize)
    x[5, 1], x[17, n - 1] = float("nan"), float("inf")
    r = obj.iso_balance_loss(x, 3, renormalize=renormalize)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[5, 17]] = True
    assert bool(r.gates[bad].isnan().all()) and torch.equal(r.gates[~bad], want.gates[~bad])
    assert torch.equal(r.experts[~bad], want.experts[~bad]) and bool((r.experts[5] != 1).all()) and int(r.experts[17, 0]) == n - 1
    assert bool(r.loss.isnan())
    d = obj.iso_balance_loss_backward(x, r, grad_gates=torch.ones_like(r.gates))
    assert bool(d[bad].isnan().all()) and bool(d[~bad].isfinite().all())


def test_router_of_many_experts_in_a_graph(cuda_ok):
    """More than 512 experts, whose sums take more shared memory than a kernel has by itself, captured."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x = torch.randn((3000, 1000), device="cuda")
    held = torch.zeros_like(x)
    obj.iso_balance_loss(held, 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = obj.iso_balance_loss(held, 4)
    held.copy_(x)
    graph.replay()
    want = obj.iso_balance_loss(x, 4)
    assert torch.equal(r.loss, want.loss) and torch.equal(r.experts, want.experts) and torch.equal(r.counts, want.counts)


@pytest.mark.parametrize("n", [5, 1000, 50021])
def test_one_row_without_a_rows_dimension(cuda_ok, n):
    """Scores [n] with a label of no dimension: as the one row [1, n]."""
    import torch
    from convex_hull_pava_gb300 import objectives as obj
    x, xw, labels, rng = make(1, n, "bf16", seed=n)
    li, one = ids(labels), put(np.ones(1))
    lp, norm, st = obj.iso_token_logp(x[0], li[0])
    assert lp.shape == () and torch.equal(lp, obj.iso_token_logp(x, li)[0][0])
    d = obj.iso_token_logp_backward(one[0], x[0], li[0], norm)
    assert d.shape == (n,) and torch.equal(d, obj.iso_token_logp_backward(one, x, li, norm)[0])
    r, want = obj.iso_policy_loss(x[0], li[0], lp, one[0]), obj.iso_policy_loss(x, li, lp[None], one)
    assert r.coef.shape == () and torch.equal(r.dlogits, want.dlogits[0]) and torch.equal(r.loss, want.loss)
    r, want = obj.iso_preference_loss(x[0], li[0], ids([0, 1, 1])), obj.iso_preference_loss(x, li, ids([0, 1, 1]))
    assert torch.equal(r.dlogits, want.dlogits[0]) and torch.equal(r.loss, want.loss)
