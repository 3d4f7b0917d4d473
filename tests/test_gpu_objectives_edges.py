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
    ([5, 2, 5, 7, 9, 1 << 40, 0, 3, 5], [4, 0, 4, 0], [0, 0, 0, 3, 5, 5, 5, 7, 9]),
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
