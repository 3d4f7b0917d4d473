"""The choices over rows of scores on the GPU: calls that the documentation allows and that are easily got wrong."""
import threading

import numpy as np
import pytest

import choices_ref as ref
from test_gpu_choices import check_beams, check_route, put, rows_of, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups", [(8, 2), (64, 8), (256, 8), (300, 3)])
def test_route_bias_of_infinity(cuda_ok, n, groups, score):
    """A bias of +inf puts its experts first (by index among themselves), and their groups."""
    rng = np.random.default_rng(n)
    v = rng.standard_normal((60, n))
    bias = (0.05 * rng.standard_normal(n)).astype(np.float32)
    bias[[1, n // 2, n - 1]] = np.inf
    bias[n // 3] = -np.inf
    for best in (1, 2):
        for k in (1, 2, min(5, n // groups)):
            check_route(rows_of(v, "f32"), k, None, bias, score=score, groups=groups, top_groups=max(1, groups // 2), group_best=best,
                        renormalize=True)
            check_route(rows_of(v, "f32"), k, None, bias, score=score, renormalize=best == 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_that_float32_cannot_tell(cuda_ok, score):
    """Groups that are each other's copies but for a bias of a part in 10^8 of their sums."""
    rng = np.random.default_rng(11)
    groups, size = 8, 32
    half = rng.standard_normal((1, size)).astype(np.float32)
    v = np.tile(half, (100, groups))
    bias = (1e-9 * rng.integers(-8, 9, groups * size)).astype(np.float32)
    for best in (1, 2):
        check_route(rows_of(v, "f32"), 6, None, bias, score=score, groups=groups, top_groups=3, group_best=best)


def test_route_scores_of_any_size(cuda_ok):
    rng = np.random.default_rng(3)
    for size in (1e-30, 1e-3, 50.0, 3e3, 1e6, 1e30):
        v = size * rng.standard_normal((40, 96))
        for score in ("softmax", "sigmoid"):
            for renormalize in (False, True):
                check_route(rows_of(v, "f32"), 5, score=score, renormalize=renormalize)
                if size <= 50.0:
                    check_route(rows_of(v, "f32"), 5, None, np.linspace(-0.1, 0.1, 96).astype(np.float32), score=score, renormalize=renormalize)


def test_rows_that_are_one_row(cuda_ok):
    """Rows of a stride of 0 (a broadcast row) are read as they are."""
    import torch
    from convex_hull_pava_gb300 import choices
    x = torch.randn(1, 640, device="cuda")
    a, b = choices.iso_route(x.expand(30, 640), 4, renormalize=True), choices.iso_route(x, 4, renormalize=True)
    assert bool((a.experts == b.experts).all()) and bool((a.gates == b.gates).all()) and int(a.counts.sum()) == 120
    g = torch.randn(30, 4, device="cuda")
    d = choices.iso_route_backward(g, x.expand(30, 640), a)
    assert d.shape == (30, 640) and d.is_contiguous()
    scores = torch.tensor([[-1.0, -1.0, -2.0]], device="cuda")
    c = choices.iso_beam_choose(x.expand(3, 640), scores, 5)
    want, parents, tokens, _ = ref.beam_choose(np.repeat(wide(x), 3, 0), wide(scores), 5)
    np.testing.assert_array_equal(c.beams.cpu().numpy(), parents)
    np.testing.assert_array_equal(c.tokens.cpu().numpy(), tokens)


@pytest.mark.parametrize("n", [300, 9000, 131072, 300007])
def test_beam_first_step_of_many_beams(cuda_ok, n):
    """One beam in use of 32, the most places: its continuations fill them."""
    rng = np.random.default_rng(n)
    v = rng.standard_normal((32, n)) * 2.0
    scores = np.full((1, 32), -np.inf)
    scores[0, 17] = -0.25
    check_beams(rows_of(v, "bf16"), scores, 64)
    done = np.zeros((1, 32), bool)
    done[0, 3] = True
    scores[0, 3] = -9.0
    check_beams(rows_of(v, "bf16"), scores, 64, done, end=n - 1)


@pytest.mark.parametrize("n", [2000, 40000])
def test_beam_few_open_scores(cuda_ok, n):
    """Rows that are closed but for a stretch or some places: fewer open scores than places, and than threads."""
    rng = np.random.default_rng(n)
    for some in (1, 3, 70, 400):
        v = np.full((12, n), -np.inf)
        for r in range(12):
            at = rng.choice(n, some, replace=False) if r % 2 else n - some + np.arange(some)
            v[r, at] = rng.standard_normal(some)
        check_beams(rows_of(v, "f32", shift=1), np.tile(-np.arange(3) / 2.0, (4, 1)), 64)


def test_beam_rows_of_few_scores_and_many(cuda_ok):
    """More rows than the GPU holds CTAs, of sizes around its units."""
    rng = np.random.default_rng(6)
    for n, batch in ((3, 700), (127, 500), (1024, 300), (4104, 260), (8190, 200)):
        v = 2.0 * rng.standard_normal((batch * 2, n))
        check_beams(rows_of(v, "f16"), -rng.random((batch, 2)).astype(np.float32).astype(np.float64), 3)


def test_beam_large_and_small_temperatures(cuda_ok):
    rng = np.random.default_rng(9)
    v = (rng.integers(-8000, 8000, (8, 3000)) / 1024.0)
    for t in (1e-4, 0.01, 30.0, 1e5):
        check_beams(rows_of(v, "f32"), -rng.random((2, 4)).astype(np.float32).astype(np.float64), 9, temperature=t)


def test_workspace_of_any_contents(cuda_ok):
    """Nothing is read of a workspace that the call has not written: not-a-numbers and large numbers in it change nothing."""
    import torch
    from convex_hull_pava_gb300 import choices, load_library
    g = torch.Generator(device="cuda").manual_seed(2)
    for batch, beams, n in ((3, 4, 70001), (150, 5, 900), (1, 2, 20)):
        x = torch.randn((batch * beams, n), generator=g, device="cuda")
        scores = -torch.rand((batch, beams), generator=g, device="cuda")
        need = load_library().iso_beam_choose_workspace_bytes(batch, beams, n, 0, 7)
        got = []
        for fill in (0, 0xff, 0x7f, 0x42):
            w = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            got.append(choices.iso_beam_choose(x, scores, 7, workspace=w))
        for r in got[1:]:
            assert torch.equal(r.scores, got[0].scores) and torch.equal(r.tokens, got[0].tokens) and torch.equal(r.beams, got[0].beams)


def test_saved_states_notice_the_move(cuda_ok):
    """A graph that has saved a state for its gradient does not take it for what it was."""
    import torch
    from convex_hull_pava_gb300 import choices
    w = torch.randn(4, device="cuda", requires_grad=True)
    h = torch.randn(6, 4, device="cuda")
    y = (h * w).sum()
    choices.iso_beam_reorder(h, torch.tensor([[1, 0, 2], [0, 2, 1]], dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError):
        y.backward()
    with torch.inference_mode():
        t = torch.arange(6, device="cuda")
        choices.iso_beam_reorder(t, torch.tensor([[1, 0, 2], [0, 2, 1]], dtype=torch.int32, device="cuda"))
    assert t.tolist() == [1, 0, 2, 3, 5, 4]


def test_calls_from_several_threads(cuda_ok):
    """Calls at the same time on streams of their own."""
    import torch
    from convex_hull_pava_gb300 import choices
    g = torch.Generator(device="cuda").manual_seed(4)
    work = []
    for n in (4000, 9001, 30000, 800):
        work.append((torch.randn((20, n), generator=g, device="cuda"), -torch.rand((5, 4), generator=g, device="cuda"),
                     torch.randn((3000, 64), generator=g, device="cuda")))

    def run(x, scores, y):
        c = choices.iso_beam_choose(x, scores, 6)
        r = choices.iso_route(y, 4, score="sigmoid", renormalize=True)
        return c.scores, c.tokens, r.gates, r.experts, r.counts, choices.iso_route_backward(r.gates, y, r)

    want = [run(*w) for w in work]
    torch.cuda.synchronize()
    bad = []

    def one(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = run(*work[i])
                stream.synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=one, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_route_captured_gradient(cuda_ok):
    """A training step through the router, captured and replayed."""
    import torch
    from convex_hull_pava_gb300 import choices
    x = torch.randn(64, 40, device="cuda", requires_grad=True)
    w = torch.randn(64, 3, device="cuda")

    def step():
        gates, _, _ = choices.route(x, 3, score="sigmoid", renormalize=True)
        return torch.autograd.grad((gates * w).sum(), x)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = step()
    for _ in range(2):
        with torch.no_grad():
            x.normal_()
        w.normal_()
        graph.replay()
        got = d.clone()
        assert torch.equal(got, step())
