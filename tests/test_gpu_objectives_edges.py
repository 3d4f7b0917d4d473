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
