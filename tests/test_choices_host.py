"""The choices' host side: what is refused (no GPU), and the 64-bit forms on worked cases."""
import ctypes

import numpy as np
import pytest

import choices_ref as ref
import convex_hull_pava_gb300 as chp
from convex_hull_pava_gb300 import choices

P = ctypes.c_void_p(0x1000)
WS = ctypes.c_void_p(0x100000)
BAD = chp.ISO_ERR_INVALID_ARG


def route_args(**change):
    a = dict(logits=P, dtype=0, tokens=4, experts=16, stride=16, top_k=2, mask=None, bias=None, score=0, groups=1,
             top_groups=1, group_best=2, renormalize=0, scale=1.0, counts=P, chosen=P, gates=P, picked=None, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(counts=None), dict(chosen=None), dict(gates=None), dict(dtype=3), dict(dtype=-1),
    dict(tokens=-1), dict(experts=0), dict(experts=1025, stride=1025), dict(stride=-1),
    dict(stride=1 << 39), dict(top_k=0), dict(top_k=17), dict(experts=64, stride=64, top_k=33), dict(score=2),
    dict(score=-1), dict(groups=0), dict(groups=3), dict(experts=64, stride=64, groups=64, top_groups=64),
    dict(groups=4, top_groups=0), dict(groups=4, top_groups=5), dict(groups=8, top_groups=1, top_k=3),
    dict(groups=4, top_groups=2, group_best=0), dict(groups=4, top_groups=2, group_best=3), dict(renormalize=2),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))])
def test_route_refusals(change):
    assert chp.load_library().iso_route(*route_args(**change)) == BAD


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(chosen=None), dict(gates=None), dict(grad=None), dict(out=None), dict(top_k=0),
    dict(score=2), dict(renormalize=-1), dict(scale=0.0), dict(out_stride=15), dict(tokens=-3), dict(dtype=7)])
def test_route_backward_refusals(change):
    a = dict(logits=P, dtype=0, tokens=4, experts=16, stride=16, top_k=2, score=0, renormalize=0, scale=1.0, chosen=P,
             gates=P, picked=None, grad=P, out=P, out_stride=16, stream=None)
    a.update(change)
    assert chp.load_library().iso_route_backward(*a.values()) == BAD


def beam_args(**change):
    a = dict(logits=P, dtype=1, batch=2, beams=3, n=100, stride=100, scores=P, done=None, end=0, temperature=1.0, keep=4,
             out=P, parents=P, tokens=P, ws=WS, ws_bytes=1 << 30, status=None, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(scores=None), dict(out=None), dict(parents=None), dict(tokens=None), dict(dtype=3),
    dict(batch=-1), dict(batch=1 << 31), dict(batch=1 << 30), dict(beams=0), dict(beams=33), dict(n=0), dict(n=1 << 31),
    dict(stride=-1), dict(stride=1 << 39), dict(keep=0), dict(keep=65), dict(done=P, end=-1), dict(done=P, end=100),
    dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
    dict(temperature=1e-39), dict(temperature=1e60)])
def test_beam_refusals(change):
    assert chp.load_library().iso_beam_choose(*beam_args(**change)) == BAD


def test_beam_workspace():
    lib = chp.load_library()
    need = lib.iso_beam_choose_workspace_bytes(2, 3, 100, 1, 4)
    assert need > 0
    for ws, size in ((None, 0), (WS, need - 1), (ctypes.c_void_p(0x100010), need)):
        assert lib.iso_beam_choose(*beam_args(ws=ws, ws_bytes=size)) == chp.ISO_ERR_WORKSPACE
    assert lib.iso_beam_choose_workspace_bytes(64, 8, 131072, 1, 16) > need
    for bad in ((-1, 3, 100, 1, 4), (2, 33, 100, 1, 4), (2, 3, 0, 1, 4), (2, 3, 100, 5, 4), (2, 3, 100, 1, 65)):
        assert lib.iso_beam_choose_workspace_bytes(*bad) == 0
    assert lib.iso_beam_choose(*beam_args(batch=0, logits=None, scores=None, ws=None, ws_bytes=0)) == chp.ISO_OK


def reorder(states, batch=2, beams=3, parents=P, count=None):
    table = (ctypes.c_int64 * (5 * len(states)))(*[v or 0 for s in states for v in s])   # iso_state: five 64-bit numbers
    return chp.load_library().iso_beam_reorder(table, len(states) if count is None else count, batch, beams, parents, None)


@pytest.mark.parametrize("state", [
    (None, 64, 1, 0, 64), (0x1000, -64, 1, 0, 64), (0x1000, 64, -1, 0, 64), (0x1000, 64, 1, 0, -1),
    (0x1000, 63, 1, 0, 64),            # rows overlap
    (0x1000, 0, 1, 0, 64),
    (0x1000, 256, 4, 63, 64),          # runs overlap
    (0x1000, 192, 4, 64, 64),          # rows overlap the runs of others
    (0x1000, 64, 4, 64 * 6 - 1, 64),   # runs of rows overlap
    (0x1000, 1 << 60, 1, 0, 64)])
def test_reorder_refusals(state):
    assert reorder([state]) == BAD
    assert reorder([(0x1000, 64, 1, 0, 64)] * 2 + [state]) == BAD


def test_reorder_arguments():
    good = (0x1000, 64, 1, 0, 64)
    assert reorder([good], beams=0) == BAD and reorder([good], beams=33) == BAD and reorder([good], batch=-1) == BAD
    assert reorder([good], parents=None) == BAD and reorder([good], count=-1) == BAD
    assert reorder([good], batch=0, parents=None) == chp.ISO_OK and reorder([], parents=None) == chp.ISO_OK
    assert reorder([(None, 0, 0, 0, 64), (None, 0, 5, 0, 0)], beams=1) == chp.ISO_OK   # nothing to move


def test_host_tensors_refused():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        choices.iso_route(x, 2)
    with pytest.raises(ValueError):
        choices.iso_beam_choose(x, torch.zeros(2, 2), 2)
    with pytest.raises(ValueError):
        choices.iso_beam_reorder([x], torch.zeros(2, 2, dtype=torch.int32))


def layout(x, rows, batch):
    return choices._layout(x.shape, x.stride(), rows, batch)


def test_layouts_of_states():
    import torch
    x = torch.empty(6, 4, 10, 8)
    assert layout(x, 6, 2) == (320, 1, 0, 320)
    assert layout(x[:, :, :7], 6, 2) == (320, 4, 80, 56)
    assert layout(x.view(2, 3, 4, 10, 8)[:, :, :, :7], 6, 2) == (320, 4, 80, 56)
    assert layout(x.transpose(1, 2), 6, 2) == (320, 1, 0, 320)          # dimensions in any order
    assert layout(x.transpose(0, 1), 4, 2) == (80, 6, 320, 80)           # rows inside runs
    assert layout(x[:, 1:3, :7, :5], 6, 2) is None                        # two dimensions apart
    assert layout(x[:, :, :1, :], 6, 2) == (320, 4, 80, 8)
    assert layout(x[:, 0, 0, 0], 6, 2) == (320, 1, 0, 1)
    assert layout(torch.empty(2, 6)[:, ::2], 6, 2) == (2, 1, 0, 1)
    assert layout(torch.empty(2, 4, 5)[:, :3], 6, 2) is None              # batch and beams do not make one dimension


def test_reference_on_worked_cases():
    gates, experts, counts = ref.route([[1.0, 2.0, 2.0, -np.inf]], 3)
    assert experts.tolist() == [[1, 2, 0]] and counts.tolist() == [1, 1, 1, 0]
    z = 2 * np.exp(1.0) + 1.0
    assert np.allclose(gates[0], [np.exp(1.0) / z, np.exp(1.0) / z, 1.0 / z])
    # groups: the sum of two decides, not the best one
    x = np.log([[0.4, 0.01, 0.3, 0.29]])
    assert ref.route(x, 1, groups=2, top_groups=1)[1].tolist() == [[2]]
    assert ref.route(x, 1, groups=2, top_groups=1, group_best=1)[1].tolist() == [[0]]
    # the bias moves the choice, not the gate
    gates, experts, _ = ref.route([[0.0, 0.0]], 1, score="sigmoid", bias=[0.0, 0.1], scale=2.0)
    assert experts.tolist() == [[1]] and gates.tolist() == [[1.0]]
    s, b, t, bad = ref.beam_choose(np.log([[0.5, 0.5], [0.9, 0.1]]), [[0.0, -0.1]], 3)
    assert b.tolist() == [[1, 0, 0]] and t.tolist() == [[0, 0, 1]] and not bad.any()
    assert np.allclose(s, [[np.log(0.9) - 0.1, np.log(0.5), np.log(0.5)]])
    s, b, t, _ = ref.beam_choose(np.zeros((2, 2)), [[-1.0, -0.5]], 4, done=np.array([[0, 1]]), end=1)
    assert b.tolist() == [[1, 0, 0, -1]] and t.tolist() == [[1, 0, 1, -1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 12))
    g = rng.standard_normal((5, 4))
    options = dict(score=score, renormalize=renormalize, scale=1.7, groups=3, top_groups=2)
    gates, experts, _ = ref.route(x, 4, **options)
    d = ref.route_grad(x, g, gates, experts, score, renormalize, 1.7)
    h = 1e-6
    for t in range(5):
        for e in range(12):
            y = x.copy()
            y[t, e] += h
            up = (ref.route(y, 4, **options)[0] * g).sum()
            y[t, e] -= 2 * h
            assert abs((up - (ref.route(y, 4, **options)[0] * g).sum()) / (2 * h) - d[t, e]) < 1e-8
