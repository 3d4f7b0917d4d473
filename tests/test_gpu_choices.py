"""The choices over rows of scores on the GPU against their 64-bit forms.

Choices (experts, beams, tokens, counts) are equal to the 64-bit form's, also between values that float32
cannot tell apart.  Tolerances of the rest (written before the first run).
* A share: the exponential 2^-22 and its exponent rounded at 2^-24 |v| log 2 with v up to 1.45 |x - m|
  (softmax) or 1.45 |x| (sigmoid), a sum of up to 1,024 terms in chains of at most 37 (32 of a lane, 5 of a
  warp) at 2^-24, a quotient at 2^-23; a renormalised one has two such shares:
  relative 5e-6 + 2.5e-7 |x|, |x| the largest of the token's finite scores.
* A gradient element: products of the above, |d| times twice that, and where terms cancel (g less a
  mean) that of scale |g| times the share; one rounding to the type, 2^-24, 2^-8, 2^-11 relative, float16
  subnormals 2^-25 absolute.
* A beam's score: the log of a sum as the objectives' log-probabilities, 4e-6 absolute, and one
  rounding to float32, 2^-24 of itself."""
import numpy as np
import pytest

import choices_ref as ref

pytestmark = pytest.mark.gpu

TYPES = ("f32", "bf16", "f16")
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}


def tor(dtype):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]


def rows_of(v, dtype, pad=0, shift=0):
    """v's values as a view of rows padded by `pad` that starts `shift` elements into its buffer."""
    import torch
    rows, n = v.shape
    buf = torch.full((rows * (n + pad) + shift,), float("nan"), dtype=tor(dtype), device="cuda")
    x = buf[shift:].view(rows, n + pad)[:, :n]
    x.copy_(torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda())
    return x


def wide(t):
    return t.detach().double().cpu().numpy()


def put(v, dtype=np.float32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(v, dtype)).cuda()


def check_route(x, top_k, mask=None, bias=None, grad_seed=1, out=None, **options):
    """Runs a router forward and backward and compares with the 64-bit form."""
    from convex_hull_pava_gb300 import choices
    v = wide(x)
    scale, score, renormalize = options.get("scale", 1.0), options.get("score", "softmax"), options.get("renormalize", False)
    r = choices.iso_route(x, top_k, None if mask is None else put(mask, bool), bias=None if bias is None else put(bias), **options)
    gates, experts, counts = ref.route(v, top_k, mask, bias=bias, **options)
    np.testing.assert_array_equal(r.experts.cpu().numpy(), experts)
    np.testing.assert_array_equal(r.counts.cpu().numpy(), counts)
    finite = np.where(np.isfinite(v), np.abs(v), 0.0)
    spread = 2.0 * finite.max(1, keepdims=True) if score == "softmax" else finite.max(1, keepdims=True)
    rel = 5e-6 + 2.5e-7 * spread
    got = wide(r.gates)
    assert (np.isnan(got) == np.isnan(gates)).all()
    ok = ~np.isnan(gates)
    err = np.where(ok, np.abs(got - np.where(ok, gates, 0.0)), 0.0)
    assert (err <= rel * np.where(ok, np.abs(gates), 0.0) + 1e-37).all(), (err / np.maximum(np.abs(gates), 1e-30)).max()
    rng = np.random.default_rng(grad_seed)
    g = rng.standard_normal((v.shape[0], top_k)).astype(np.float32)
    d = choices.iso_route_backward(put(g), x, r, out=out)
    if score == "sigmoid" and out is None:   # without the scores that the forward has kept
        again = choices.iso_route_backward(put(g), x, choices.Route(r.gates, r.experts, r.counts, score, r.renormalize, r.scale))
        np.testing.assert_array_equal(wide(again), wide(d))
    want = ref.route_grad(v, g, gates, experts, score, renormalize, scale)
    dtype = str(x.dtype).split(".")[1]
    dtype = {"float32": "f32", "bfloat16": "bf16", "float16": "f16"}[dtype]
    got = wide(d)
    assert (np.isnan(got) == np.isnan(want)).all()
    ok = ~np.isnan(want)
    p = np.where(np.isnan(ref.shares(v, score)), 0.0, ref.shares(v, score))
    if renormalize:   # a renormalised gate stands for the share
        p = np.zeros_like(p)
        for t in range(len(v)):
            at = experts[t][experts[t] >= 0]
            p[t, at] = np.nan_to_num(gates[t, :len(at)]) / scale
    size = scale * np.abs(g).max(1, keepdims=True) * p
    tol = 2 * rel * (np.abs(np.where(ok, want, 0.0)) + 2 * size) + HALF[dtype] * np.abs(np.where(ok, want, 0.0)) + TINY[dtype]
    err = np.where(ok, np.abs(got - np.where(ok, want, 0.0)), 0.0)
    assert (err <= tol).all(), (err - tol).max()
    return r


ROUTERS = [  # tokens, experts, top_k, groups, top_groups
    (1, 1, 1, 1, 1), (3, 5, 2, 1, 1), (40, 8, 8, 1, 1), (33, 16, 4, 4, 2), (7, 24, 2, 3, 2), (65, 64, 6, 8, 3), (129, 160, 6, 8, 3),
    (70, 256, 8, 8, 4), (70, 256, 8, 1, 1), (9, 384, 8, 1, 1), (31, 512, 10, 32, 5), (5, 1024, 32, 4, 2), (6, 1000, 32, 10, 10),
    (2, 96, 32, 32, 11), (300, 128, 1, 1, 1), (17, 33, 3, 11, 1), (12, 500, 20, 5, 3)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,n,k,groups,top_groups", ROUTERS)
def test_route(cuda_ok, tokens, n, k, groups, top_groups, score, dtype):
    seed = tokens * 7 + n
    rng = np.random.default_rng(seed)
    for turn, (renormalize, biased, best) in enumerate([(True, True, 2), (False, False, 1), (True, False, 2), (False, True, 1)]):
        v = rng.standard_normal((tokens, n)) + 0.7 * rng.standard_normal((1, n))
        bias = np.round(0.1 * rng.standard_normal(n), 3).astype(np.float32) if biased else None
        mask = rng.random(tokens) < 0.8 if turn % 2 else None
        x = rows_of(v, dtype, pad=[0, 0, 3, 8][turn], shift=[0, 1, 0, 0][turn])
        check_route(x, k, mask, bias, score=score, groups=groups, top_groups=top_groups, group_best=best,
                    renormalize=renormalize, scale=[1.0, 2.5, 1.0, 0.125][turn])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,k,groups", [(8, 3, 2), (32, 8, 1), (64, 6, 4), (256, 8, 8), (600, 20, 6)])
def test_route_equal_scores(cuda_ok, n, k, groups, score):
    """Few distinct scores and biases: equal values, also of groups, go to the lowest index."""
    rng = np.random.default_rng(n + k)
    v = rng.integers(-2, 3, (50, n)) * 0.5
    v[:5] = 1.25
    for bias in (None, np.zeros(n, np.float32), (rng.integers(0, 3, n) / 64).astype(np.float32)):
        for best in (1, 2):
            check_route(rows_of(v, "bf16"), k, None, bias, score=score, groups=groups, top_groups=max(1, groups // 2),
                        group_best=best, renormalize=best == 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n", [16, 48, 256, 700])
def test_route_choices_that_float32_cannot_tell(cuda_ok, n, score):
    """A bias that makes pairs of experts equal but for its own rounding to float32 (a part in 10^8): the
    choice is that of the exact sums."""
    rng = np.random.default_rng(n)
    tokens = 200 if n < 300 else 40
    v = rng.standard_normal((1, n)).astype(np.float32)
    p = ref.shares(v, score)[0]
    bias = np.zeros(n, np.float32)
    half = n // 2
    bias[half:2 * half] = (p[:half] - p[half:2 * half]).astype(np.float32)
    x = np.repeat(v, tokens, 0)
    assert len(set(np.round(p[:half], 6))) > half // 2
    check_route(rows_of(x, "f32"), min(8, n // 4), None, bias, score=score, renormalize=True)
    # and as sums of a group's two
    check_route(rows_of(x, "f32"), 4, None, bias, score=score, groups=4, top_groups=2, group_best=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,groups", [(7, 1), (16, 4), (40, 1), (256, 8), (640, 5)])
def test_route_closed_nan_and_infinite(cuda_ok, n, groups, dtype):
    """Closed experts, tokens with fewer open ones than places, NaN, +inf, the types' lowest values."""
    import torch
    rng = np.random.default_rng(n)
    k = min(5, n // groups)
    low = float(torch.finfo(tor(dtype)).min)
    v = np.clip(rng.standard_normal((24, n)), -3, 3)
    v[0] = -np.inf
    v[1, 1:] = -np.inf
    v[2, ::2] = -np.inf
    v[3, 0] = np.nan
    v[4, n - 1] = np.inf
    v[5] = np.nan
    v[6, : n // 2] = np.nan
    v[7] = low
    v[8, 1:] = low
    v[9, ::2] = -np.inf
    v[9, 1::2] = low
    v[10] = np.inf
    v[11, 0], v[11, 1:] = np.nan, -np.inf
    v[12] = -60000.0
    v[13] = 3e4
    v[14, : n - 1] = -200.0
    bias = (0.05 * rng.standard_normal(n)).astype(np.float32)
    bias[n // 3] = -np.inf
    bias[n // 2] = np.nan
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            for b in (None, bias):
                keep = np.ones(24, bool)
                if b is None and groups > 1 and score == "softmax":
                    keep[[4, 10]] = False   # which groups a token without probabilities takes is not promised
                check_route(rows_of(v[keep], dtype), k, None, b, score=score, renormalize=renormalize, groups=groups,
                            top_groups=max(1, groups - 1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_route_one_renormalised_gate(cuda_ok, dtype, score):
    """The renormalised gate of one expert alone is the scale, whatever its score, and has no gradient at all."""
    from convex_hull_pava_gb300 import choices
    rng = np.random.default_rng(8)
    for n, k, groups, scale in ((40, 1, 1, 2.5), (256, 1, 8, 0.3), (1000, 1, 1, 1.0), (90, 1, 9, 7.0), (8, 4, 1, 2.5)):
        v = 2.0 * rng.standard_normal((500, n))
        if k > 1:
            v[:, 1:] = -np.inf   # more places than open experts
        r = choices.iso_route(rows_of(v, dtype), k, score=score, groups=groups, renormalize=True, scale=scale)
        assert (wide(r.gates)[:, 0] == np.float32(scale)).all() and (wide(r.gates)[:, 1:] == 0).all()
        d = choices.iso_route_backward(put(rng.standard_normal((500, k))), rows_of(v, dtype), r)
        assert (wide(d) == 0).all()


def test_route_empty(cuda_ok):
    import torch
    from convex_hull_pava_gb300 import choices
    r = choices.iso_route(torch.empty(0, 8, device="cuda"), 2)
    assert r.gates.shape == (0, 2) and r.experts.shape == (0, 2) and r.counts.tolist() == [0] * 8
    assert choices.iso_route_backward(torch.empty(0, 2, device="cuda"), torch.empty(0, 8, device="cuda"), r).shape == (0, 8)
    r = choices.iso_route(torch.randn(5, 8, device="cuda"), 2, torch.zeros(5, dtype=torch.bool, device="cuda"))
    assert (r.experts == -1).all() and (r.gates == 0).all() and r.counts.sum() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k", [(5, 2), (64, 3), (256, 8), (1000, 32)])
@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True), ("sigmoid", False)])
def test_route_gradient_over_the_scores(cuda_ok, n, k, score, renormalize, dtype):
    from convex_hull_pava_gb300 import choices
    rng = np.random.default_rng(n)
    x = rows_of(rng.standard_normal((300, n)), dtype, pad=3)
    r = choices.iso_route(x, k, score=score, renormalize=renormalize)
    g = put(rng.standard_normal((300, k)))
    want = choices.iso_route_backward(g, x, r).clone()
    got = choices.iso_route_backward(g, x, r, out=x)
    assert got is x and bool((got == want).all())


def test_route_many_tokens(cuda_ok):
    """More tokens than a launch holds at once: each token as alone, and the counts of all."""
    import torch
    from convex_hull_pava_gb300 import choices
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((200003, 20), generator=g, device="cuda")
    b = 0.1 * torch.randn(20, generator=g, device="cuda")
    options = dict(score="sigmoid", bias=b, groups=4, top_groups=2, renormalize=True)
    r = choices.iso_route(x, 3, **options)
    for at in (0, 77777, 199000):
        part = choices.iso_route(x[at:at + 1003], 3, **options)
        assert bool((part.experts == r.experts[at:at + 1003]).all()) and bool((part.gates == r.gates[at:at + 1003]).all())
    assert bool((torch.bincount(r.experts.reshape(-1).long(), minlength=20) == r.counts).all())
    again = choices.iso_route(x, 3, **options)
    assert bool((again.gates == r.gates).all()) and bool((again.experts == r.experts).all())


def test_route_autograd(cuda_ok):
    import torch
    from convex_hull_pava_gb300 import choices
    x = torch.randn(50, 32, device="cuda", requires_grad=True)
    bias = torch.zeros(32, device="cuda")
    gates, experts, counts = choices.route(x, 4, score="sigmoid", bias=bias, renormalize=True, scale=2.0)
    assert not experts.requires_grad and not counts.requires_grad and gates.requires_grad
    w = torch.randn(50, 4, device="cuda")
    got, = torch.autograd.grad((gates * w).sum(), x, retain_graph=True)
    s = torch.sigmoid(x.double())
    top = s.gather(1, experts.long())
    want, = torch.autograd.grad((2 * top / top.sum(1, keepdim=True) * w).sum(), x)
    assert (got - want).abs().max() <= 1e-5
    again, = torch.autograd.grad(gates.sum() * 0 + (gates * w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        again.sum().backward()


# ---------------------------------------------------------------------------
# Beams
# ---------------------------------------------------------------------------
def check_beams(x, scores, keep, done=None, end=0, temperature=1.0):
    from convex_hull_pava_gb300 import choices
    want, parents, tokens, bad = ref.beam_choose(wide(x), scores, keep, done, end, temperature)
    r = choices.iso_beam_choose(x, put(scores), keep, None if done is None else put(done, bool), end=end, temperature=temperature)
    np.testing.assert_array_equal(r.beams.cpu().numpy(), parents)
    np.testing.assert_array_equal(r.tokens.cpu().numpy(), tokens)
    got = wide(r.scores)
    some = np.isfinite(want)
    assert (np.isfinite(got) == some).all() and (got[~some] == -np.inf).all()
    err = np.abs(got[some] - want[some])
    assert (err <= 4e-6 + 2.0 ** -24 * np.abs(want[some])).all(), err.max()
    np.testing.assert_array_equal(r.row_status.cpu().numpy() != 0, bad)
    return r


BEAMS = [  # batch, beams, n, keep
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 10), (1, 2, 300, 64), (5, 4, 1000, 8), (3, 5, 8192, 10), (1, 4, 131072, 8),
    (2, 32, 2049, 64), (40, 6, 5021, 6), (1, 1, 600011, 64), (200, 4, 333, 4), (2, 16, 50021, 32)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,beams,n,keep", BEAMS)
def test_beam_choose(cuda_ok, batch, beams, n, keep, dtype):
    rng = np.random.default_rng(batch * 31 + n)
    rows = batch * beams
    for turn in range(2):
        v = 2.0 * rng.standard_normal((rows, n))
        v[np.arange(rows), rng.integers(0, n, rows)] = 9.0 + rng.standard_normal(rows)
        if turn:
            v[:, n - n // 50:] = -np.inf
        scores = -np.cumsum(1.0 + rng.random((batch, beams)), 1)
        scores = scores.astype(np.float32).astype(np.float64)
        done = rng.random((batch, beams)) < 0.3 if turn else None
        x = rows_of(v, dtype, pad=[0, 5][turn], shift=[0, 3][turn])
        check_beams(x, scores, keep, done, end=n // 2, temperature=[1.0, 0.7][turn])


def test_beam_dead_beams_and_first_step(cuda_ok):
    """Beams that are not in use yet (-inf), and other scores that are no numbers: their rows are not read."""
    rng = np.random.default_rng(0)
    v = rng.standard_normal((12, 3000))
    v[1] = np.nan
    v[6:8] = np.nan
    scores = np.array([[0.0, -np.inf, -np.inf, -np.inf], [-1.0, -2.0, np.inf, np.nan], [-np.inf] * 4])
    r = check_beams(rows_of(v, "f32"), scores, 8)
    assert (r.row_status == 0).all() and (r.beams[2] == -1).all() and (r.beams[0] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_beam_infinities_nan_and_lowest_values(cuda_ok, dtype):
    import torch
    rng = np.random.default_rng(1)
    low = float(torch.finfo(tor(dtype)).min)
    v = np.clip(2 * rng.standard_normal((16, 2500)), -9, 9)
    v[0, 7] = np.nan
    v[1, 2499] = np.inf
    v[2] = -np.inf
    v[3, 5:] = -np.inf
    v[4] = low
    v[5, 1:] = low
    v[6, :1250] = low
    v[7, 3:] = low
    v[7, :3] = -np.inf
    v[9] = 60000.0
    v[10, ::2] = -60000.0
    v[11, 0] = 60000.0
    scores = np.tile(-np.arange(4) / 4.0, (4, 1))
    check_beams(rows_of(v, dtype), scores, 12)
    check_beams(rows_of(v, dtype, shift=1), scores, 3, temperature=0.25)


@pytest.mark.parametrize("n", [40, 700, 5000, 70001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_equal_scores(cuda_ok, n, dtype):
    """Rows of one score, of few, and equal beams: the lowest beam, then the lowest token."""
    rng = np.random.default_rng(n)
    v = np.zeros((18, n))
    v[3:6] = rng.integers(0, 2, (3, n))
    v[6:9] = rng.integers(0, 2, (1, n))
    v[9:12] = rng.standard_normal((1, n))
    v[12:15, n // 2:] = 1.0
    v[15] = 1.0
    scores = np.zeros((6, 3))
    for keep in (1, 7, 64):
        check_beams(rows_of(v, dtype), scores, keep)
        check_beams(rows_of(v, dtype, pad=1), scores, keep)   # equal rows at unequal places in memory


@pytest.mark.parametrize("n", [50, 3001, 131072])
def test_beam_choices_that_float32_cannot_tell(cuda_ok, n):
    """Scores that make the best continuations of two beams equal but for the scores' own rounding (about
    1e-9): the order is that of the exact totals."""
    rng = np.random.default_rng(n)
    batch = 12
    v = (2.0 * rng.standard_normal((2 * batch, n))).astype(np.float32).astype(np.float64)
    scores = np.zeros((batch, 2))
    best = ref.log_probabilities(v, 1.0).max(1)
    for i in range(batch):   # the second's score puts its best beside the first's, both scores small
        scores[i, 1] = np.float32(best[2 * i] - best[2 * i + 1])
    r = check_beams(rows_of(v, "f32"), scores, 4)
    top = wide(r.scores)[:, :2]
    assert (np.abs(top[:, 0] - top[:, 1]) < 1e-6).all()


def test_beam_far_scores(cuda_ok):
    """Scores so large against the temperature that float32 products lose their fraction."""
    rng = np.random.default_rng(4)
    v = (1e6 + rng.integers(0, 8, (8, 900)) / 2.0)
    v[4:] = rng.standard_normal((4, 900))
    scores = -rng.random((4, 2)).astype(np.float32).astype(np.float64)
    check_beams(rows_of(v, "f32"), scores, 6, temperature=0.05)
    check_beams(rows_of(v, "f32"), scores, 6, temperature=1e-6)


def test_beam_empty(cuda_ok):
    import torch
    from convex_hull_pava_gb300 import choices
    r = choices.iso_beam_choose(torch.empty(0, 10, device="cuda"), torch.empty(0, 3, device="cuda"), 4)
    assert r.scores.shape == (0, 4) and r.tokens.shape == (0, 4) and r.row_status.numel() == 0


# ---------------------------------------------------------------------------
# States
# ---------------------------------------------------------------------------
def moved(x, parents):
    batch, beams = parents.shape
    p = np.where((parents >= 0) & (parents < beams), parents, np.arange(beams))
    return (p + beams * np.arange(batch)[:, None]).reshape(-1)


@pytest.mark.parametrize("batch,beams", [(1, 1), (1, 2), (3, 4), (5, 7), (2, 16), (3, 32)])
def test_reorder(cuda_ok, batch, beams):
    """Swaps, copies and rings at once, over types, views and places that are aligned otherwise; what is
    not in use stays as it was."""
    import torch
    from convex_hull_pava_gb300 import choices
    rng = np.random.default_rng(beams)
    rows = batch * beams
    parents = rng.integers(0, beams, (batch, beams))
    parents[0] = np.roll(np.arange(beams), 1)
    if batch > 2:
        parents[1] = np.arange(beams)   # nothing moves
        parents[2, 0], parents[2, beams - 1] = -1, beams   # left as they are
    at = torch.from_numpy(moved(None, parents)).cuda()
    whole, views = [], []

    def state(shape, dtype, cut=None):
        t = torch.randint(0, 100, shape, device="cuda").to(dtype)
        whole.append(t)
        views.append(t if cut is None else cut(t))

    state((rows, 3, 40, 16), torch.bfloat16, lambda t: t[:, :, :33])
    state((rows, 2, 9, 36), torch.float16, lambda t: t[:, :, :7])
    state((rows, 777), torch.int64)
    state((rows, 1001), torch.uint8)
    state((rows, 5, 11), torch.float32, lambda t: t[:, 1:4, 3:9])
    state((batch, beams, 70), torch.bool)
    state((rows,), torch.float64)
    state((4, rows, 30, 8), torch.bfloat16, lambda t: t.transpose(0, 1)[:, :, :20])
    state((rows, 20, 3, 8), torch.float32, lambda t: t.transpose(1, 2))
    state((rows, 6000), torch.bfloat16, lambda t: t[:, 1:5000])
    state((rows, 0), torch.float32)
    state((rows, 4, 2, 5, 8), torch.bfloat16, lambda t: t[:, 2])
    want = []
    for t, x in zip(whole, views):
        before = t.clone()
        y = x.clone() if x.shape[0] == rows else x.reshape(rows, -1).clone()
        x.copy_(y[at].view(x.shape))
        want.append(t.clone())
        t.copy_(before)
    assert choices.iso_beam_reorder(views, torch.from_numpy(parents.astype(np.int32)).cuda()) is None
    for t, w in zip(whole, want):
        assert torch.equal(t, w)


def test_reorder_many_states(cuda_ok):
    """More states than one launch takes."""
    import torch
    from convex_hull_pava_gb300 import choices
    states = [torch.randn(6, i + 1, device="cuda") for i in range(150)]
    want = [x[[2, 0, 0, 3, 5, 4]] for x in states]
    choices.iso_beam_reorder(states, torch.tensor([[2, 0, 0], [0, 2, 1]], dtype=torch.int32, device="cuda"))
    assert all(torch.equal(x, y) for x, y in zip(states, want))


def test_reorder_far_apart(cuda_ok):
    """Rows more than 2^32 bytes apart."""
    import torch
    from convex_hull_pava_gb300 import choices
    big = torch.zeros(3, (1 << 31) + 64, dtype=torch.bfloat16, device="cuda")
    big[:, -9:] = torch.arange(27, device="cuda").view(3, 9).to(torch.bfloat16)
    choices.iso_beam_reorder(big[:, -9:], torch.tensor([[1, 2, 0]], dtype=torch.int32, device="cuda"))
    assert big[:, -9:].int().tolist() == [list(range(9, 18)), list(range(18, 27)), list(range(9))]


# ---------------------------------------------------------------------------
# Together, on streams, in graphs, refused
# ---------------------------------------------------------------------------
def test_search_of_a_routed_model(cuda_ok):
    """Beam search over a small routed recurrent model, its states moved behind the beams: each beam's
    state and score are those of its own tokens, run from the start."""
    import torch
    from convex_hull_pava_gb300 import choices, objectives
    torch.manual_seed(2)
    batch, beams, steps, n, width, experts = 3, 4, 6, 1000, 32, 8
    embed, head = torch.randn(n, width, device="cuda"), torch.randn(width, n, device="cuda") / 4
    to_router, inside = torch.randn(width, experts, device="cuda"), torch.randn(experts, width, width, device="cuda") / 4

    def advance(h, token):
        h = h + embed[token]
        gates, at, _ = choices.route(h @ to_router, 2, score="sigmoid", renormalize=True)
        each = torch.einsum("rw,ewv->rev", h, inside).gather(1, at.long()[..., None].expand(-1, -1, width))
        return torch.tanh(h + (gates[..., None] * each).sum(1))

    rows = batch * beams
    h = advance(torch.zeros(rows, width, device="cuda"), torch.zeros(rows, dtype=torch.long, device="cuda"))
    history = torch.full((rows, steps), -1, dtype=torch.long, device="cuda")
    scores = torch.full((batch, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    for step in range(steps):
        r = choices.iso_beam_choose(h @ head, scores, beams)
        choices.iso_beam_reorder([h, history[:, :step]], r.beams)
        history[:, step] = r.tokens.view(-1)
        scores = r.scores
        h = advance(h, r.tokens.view(-1))
    again = advance(torch.zeros(rows, width, device="cuda"), torch.zeros(rows, dtype=torch.long, device="cuda"))
    total = torch.zeros(rows, device="cuda")
    for step in range(steps):
        total += objectives.iso_token_logp(again @ head, history[:, step].contiguous())[0]
        again = advance(again, history[:, step])
    assert (again - h).abs().max() < 1e-4 and (total - scores.view(-1)).abs().max() < 1e-3
    assert len({tuple(t) for t in history.tolist()}) >= beams


def test_routes_agree_with_the_balance_loss(cuda_ok):
    """By softmax, without bias and groups, the choice and the counts are the balance loss's."""
    import torch
    from convex_hull_pava_gb300 import choices, objectives
    x = torch.randn(3000, 96, device="cuda").to(torch.bfloat16)
    mask = torch.rand(3000, device="cuda") < 0.9
    a, b = choices.iso_route(x, 6, mask, renormalize=True), objectives.iso_balance_loss(x, 6, mask, renormalize=True)
    assert torch.equal(a.experts, b.experts) and torch.equal(a.counts, b.counts)
    assert (a.gates - b.gates).abs().max() < 1e-6


def test_streams_and_graphs(cuda_ok):
    """A side stream given by `stream`, and captured calls replayed on new inputs, two graphs with a
    workspace in common."""
    import torch
    from convex_hull_pava_gb300 import choices
    g = torch.Generator(device="cuda").manual_seed(9)

    def inputs(n):
        return (torch.randn((12, n), generator=g, device="cuda"), -torch.rand((4, 3), generator=g, device="cuda"),
                torch.randn((12, 64), generator=g, device="cuda"), torch.randn((12, 5), generator=g, device="cuda"))

    def work(x, scores, y, w, state, workspace=None):
        c = choices.iso_beam_choose(x, scores, 3, workspace=workspace)
        choices.iso_beam_reorder(state, c.beams)
        r = choices.iso_route(y, 5, score="sigmoid", renormalize=True)
        return c.scores, c.tokens, c.beams, r.gates, r.counts, choices.iso_route_backward(w, y, r), state

    sizes = (9000, 4001)
    first = [inputs(n) for n in sizes]
    state = [torch.randn(12, 50, device="cuda") for _ in sizes]
    side = torch.cuda.Stream()
    want = work(*first[0], state[0].clone())
    torch.cuda.synchronize()
    c = choices.iso_beam_choose(first[0][0], first[0][1], 3, stream=side)
    moved_state = state[0].clone()
    torch.cuda.synchronize()
    choices.iso_beam_reorder(moved_state, c.beams, stream=side)
    r = choices.iso_route(first[0][2], 5, score="sigmoid", renormalize=True, stream=side)
    d = choices.iso_route_backward(first[0][3], first[0][2], r, stream=side)
    side.synchronize()
    for p, q in zip((c.scores, c.tokens, c.beams, r.gates, r.counts, d, moved_state), want):
        assert torch.equal(p, q)

    workspace = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for x, s in zip(first, state):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(work(*x, s, workspace=workspace))
        graphs.append(graph)
    for turn in range(3):
        new = [inputs(n) for n in sizes]
        expect = []
        for old, x, s in zip(first, new, state):
            for p, q in zip(old, x):
                p.copy_(q)
            s.normal_(generator=g)
            expect.append(work(*x, s.clone()))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, expect):
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_refusals(cuda_ok):
    import torch
    from convex_hull_pava_gb300 import IsoError, choices
    x = torch.randn(6, 16, device="cuda")
    ok = choices.iso_route(x, 2)
    g = torch.zeros(6, 2, device="cuda")
    bad = [
        lambda: choices.iso_route(x[0], 2), lambda: choices.iso_route(x.double(), 2), lambda: choices.iso_route(x.t(), 2),
        lambda: choices.iso_route(x, 0), lambda: choices.iso_route(x, 17), lambda: choices.iso_route(x, 2, score="tanh"),
        lambda: choices.iso_route(x, 2, torch.ones(5, dtype=torch.bool, device="cuda")),
        lambda: choices.iso_route(x, 2, torch.ones(6, device="cuda")), lambda: choices.iso_route(x, 2, bias=torch.zeros(16)),
        lambda: choices.iso_route(x, 2, bias=torch.zeros(15, device="cuda")),
        lambda: choices.iso_route(x, 2, bias=torch.zeros(16, device="cuda", dtype=torch.bfloat16)),
        lambda: choices.iso_route(x, 2, groups=3), lambda: choices.iso_route(x, 2, groups=4, top_groups=5),
        lambda: choices.iso_route(x, 5, groups=4, top_groups=1), lambda: choices.iso_route(x, 2, groups=2, group_best=3),
        lambda: choices.iso_route_backward(g, x, (1, 2)), lambda: choices.iso_route_backward(g[:5], x, ok),
        lambda: choices.iso_route_backward(g.double(), x, ok), lambda: choices.iso_route_backward(g, x[:5], ok),
        lambda: choices.iso_route_backward(g, x[:, :8].contiguous(), ok),
        lambda: choices.iso_route_backward(g, x, ok, out=torch.empty(6, 16, device="cuda", dtype=torch.bfloat16)),
        lambda: choices.iso_beam_choose(x, torch.zeros(2, 2, device="cuda"), 2),
        lambda: choices.iso_beam_choose(x, torch.zeros(6, device="cuda"), 2),
        lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda", dtype=torch.float64), 2),
        lambda: choices.iso_beam_choose(x, torch.zeros(2, 3), 2), lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 0),
        lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 65),
        lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 2, torch.zeros(3, 2, dtype=torch.bool, device="cuda")),
        lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 2, torch.zeros(2, 3, dtype=torch.bool, device="cuda"), end=16),
        lambda: choices.iso_beam_choose(torch.randn(99, 16, device="cuda"), torch.zeros(3, 33, device="cuda"), 2),
        lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 2, workspace=torch.empty(4, device="cuda")),
        lambda: choices.iso_beam_reorder(x, torch.zeros(2, 3, device="cuda")),
        lambda: choices.iso_beam_reorder(x, torch.zeros(6, dtype=torch.int32, device="cuda")),
        lambda: choices.iso_beam_reorder(x[:5], torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
        lambda: choices.iso_beam_reorder([x, x], torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
        lambda: choices.iso_beam_reorder([x, x.cpu()], torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
        lambda: choices.iso_beam_reorder(torch.zeros(6, 4, 4, 4, device="cuda")[:, :2, :2, :2], torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
        lambda: choices.iso_beam_reorder(x.clone().requires_grad_(), torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: choices.iso_route(x, 2, scale=0.0), lambda: choices.iso_route(x, 2, scale=float("nan")),
                 lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 2, temperature=0.0),
                 lambda: choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: choices.iso_beam_reorder(x[:1].expand(6, 16), torch.zeros(2, 3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(IsoError):
            call()


def test_kernel_times_can_be_read(cuda_ok):
    import torch
    import convex_hull_pava_gb300 as chp
    from convex_hull_pava_gb300 import choices
    chp.profile_enable(True)
    try:
        x = torch.randn(6, 64, device="cuda")
        r = choices.iso_route(x, 2)
        assert [name for name, _ in chp.profile_read()] == ["route"]
        choices.iso_route_backward(torch.zeros(6, 2, device="cuda"), x, r)
        assert [name for name, _ in chp.profile_read()] == ["route_backward"]
        c = choices.iso_beam_choose(x, torch.zeros(2, 3, device="cuda"), 3)
        assert [name for name, _ in chp.profile_read()] == ["beam_rows", "beam_join"]
        choices.iso_beam_reorder(x, c.beams)
        assert [name for name, _ in chp.profile_read()] == ["beam_reorder"]
    finally:
        chp.profile_enable(False)
