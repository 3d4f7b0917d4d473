"""Choices over rows of scores, and the states that follow them.

Beside the objectives: the experts that a router gives its tokens to, with the
gradient of its gates; the continuations that beam search keeps, of which
preference pairs and ranked answers are made; and the states of the beams that
they continue.

Explicit calls (same names and arguments as the C ABI of ``include/iso.h``, which
states the formulas, the masks and the errors in full):

* :func:`iso_route`, :func:`iso_route_backward`
* :func:`iso_beam_choose`
* :func:`iso_beam_reorder` -- in place

Differentiable in the scores (autograd): :func:`route` (first derivatives only).

Scores are float32, bfloat16 or float16 CUDA tensors, contiguous within a row (rows
may be strided).  A choice is that of the exact values, equal ones by the lowest
index.  Calls run on ``stream`` (default: the current one); what they allocate
belongs to it.
"""
from __future__ import annotations

import ctypes

from . import _torch
from . import objectives as _obj
from .objectives import (MAX_EXPERTS, MAX_TOP_K, _check, _check_out, _done, _elsewhere, _like,
                         _own_workspace, _ptr, _scores)

MAX_GROUPS = 32   # ISO_MAX_GROUPS
MAX_BEAMS = 32    # ISO_MAX_BEAMS
MAX_KEEP = 64     # ISO_MAX_KEEP
SCORES = {"softmax": 0, "sigmoid": 1}


class Route:
    """What :func:`iso_route` returns."""
    _fields = ("gates", "experts", "counts", "score", "renormalize", "scale", "picked")
    __slots__ = _fields

    def __init__(self, gates, experts, counts, score, renormalize, scale, picked=None):
        self.gates, self.experts, self.counts, self.picked = gates, experts, counts, picked
        self.score, self.renormalize, self.scale = score, renormalize, scale

    def __iter__(self):
        return (getattr(self, name) for name in self._fields)

    def __len__(self):
        return len(self._fields)


class BeamChoice:
    """What :func:`iso_beam_choose` returns."""
    _fields = ("scores", "beams", "tokens", "row_status")
    __slots__ = ("scores", "beams", "tokens", "_buf", "_rows")

    def __init__(self, scores, beams, tokens, buf, rows):
        self.scores, self.beams, self.tokens, self._buf, self._rows = scores, beams, tokens, buf, rows

    @property
    def row_status(self):
        return self._buf[self._buf.numel() - self._rows:]   # the call's workspace is in front of it

    def __iter__(self):
        return (getattr(self, name) for name in self._fields)

    def __len__(self):
        return len(self._fields)


def _mask(t, name, shape, device):
    """A bool or uint8 tensor (a bool is a byte of 0 or 1)."""
    torch = _torch()
    dtype = torch.bool if getattr(t, "dtype", None) == torch.bool else torch.uint8
    _check(t, name, dtype, shape, device)


def _router(logits, top_k, score):
    code, tokens, experts, stride, dev = _scores(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    if experts > MAX_EXPERTS or not 1 <= top_k <= min(experts, MAX_TOP_K):
        raise ValueError(f"at most {MAX_EXPERTS} experts, and 1 <= top_k <= min(experts, {MAX_TOP_K})")
    how = SCORES.get(score)
    if how is None:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    return _torch(), code, tokens, experts, stride, dev, how


def iso_route(logits, top_k: int, mask=None, *, score: str = "softmax", bias=None, groups: int = 1,
              top_groups: int = 1, group_best: int = 2, renormalize: bool = False,
              scale: float = 1.0, want_grad: bool = True, stream=None):
    """A router's choice of ``top_k`` experts for each row of ``logits`` ``[tokens, experts]``, by
    "softmax" or "sigmoid" scores and a ``bias`` (float32 ``[experts]``) that moves the choice and
    not the gates; with ``groups`` above 1, among the experts of the ``top_groups`` groups whose
    ``group_best`` (1 or 2) largest scores have the largest sum.  ``mask``: bool or uint8
    ``[tokens]``, false where a token takes no part.  Returns a :class:`Route`: ``gates`` (float32
    ``[tokens, top_k]``: ``scale`` times the scores, with ``renormalize`` divided by their sum),
    ``experts`` (int32, -1 where none), ``counts`` (int64 ``[experts]``), ``picked`` (with "sigmoid": the
    scores of the chosen, float32, which the backward takes instead of gathering them; None
    without ``want_grad``)."""
    torch, code, tokens, experts, stride, dev, how = _router(logits, top_k, score)
    if mask is not None:
        _mask(mask, "mask", logits.shape[:1], dev)
    if bias is not None:
        _check(bias, "bias", torch.float32, logits.shape[1:], dev)
    if not 1 <= groups <= MAX_GROUPS or experts % groups or not 1 <= top_groups <= groups:
        raise ValueError(f"groups must divide the experts, up to {MAX_GROUPS}, and 1 <= top_groups <= groups")
    if top_k > top_groups * (experts // groups):
        raise ValueError("top_k must not be more than the experts of top_groups groups")
    if group_best not in (1, 2):
        raise ValueError("group_best must be 1 or 2")
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_route(logits, top_k, mask, score=score, bias=bias, groups=groups,
                             top_groups=top_groups, group_best=group_best, renormalize=renormalize,
                             scale=scale, want_grad=want_grad)
    counts = torch.empty(experts, dtype=torch.int64, device=dev)
    chosen = torch.empty((tokens, top_k), dtype=torch.int32, device=dev)
    gates = torch.empty((tokens, top_k), dtype=torch.float32, device=dev)
    renormalize = bool(renormalize)
    picked = torch.empty((tokens, top_k), dtype=torch.float32, device=dev) if how and want_grad else None
    _done(_obj._abi.iso_route(
        logits.data_ptr(), code, tokens, experts, stride, top_k, _ptr(mask), _ptr(bias), how, groups,
        top_groups, group_best, renormalize, scale, counts.data_ptr(), chosen.data_ptr(),
        gates.data_ptr(), _ptr(picked), _obj._raw_stream(dev.index)), "iso_route")
    return Route(gates, chosen, counts, score, renormalize, scale, picked)


def iso_route_backward(grad_gates, logits, result, *, out=None, stream=None):
    """The gradient of ``sum(grad_gates * gates)`` in the logits, ``result`` being
    :func:`iso_route`'s for them.  ``out`` may be the logits themselves."""
    if not isinstance(result, Route):
        raise ValueError("result must be iso_route's")
    shape = result.experts.shape
    torch, code, tokens, experts, stride, dev, how = _router(logits, shape[1], result.score)
    if shape[0] != tokens or result.counts.numel() != experts or result.experts.device != dev:
        raise ValueError("logits must have the shape and device that result was made for")
    _check(grad_gates, "grad_gates", torch.float32, shape, dev)
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_route_backward(grad_gates, logits, result, out=out)
    if out is None:
        out, out_stride = _like(torch, logits, tokens, experts, stride)
    else:
        out_stride = _check_out(out, logits)
    _done(_obj._abi.iso_route_backward(
        logits.data_ptr(), code, tokens, experts, stride, shape[1], how, result.renormalize,
        result.scale, result.experts.data_ptr(), result.gates.data_ptr(), _ptr(result.picked),
        grad_gates.data_ptr(), out.data_ptr(), out_stride, _obj._raw_stream(dev.index)), "iso_route_backward")
    return out


def iso_beam_choose(logits, scores, keep: int, done=None, *, end: int = 0, temperature: float = 1.0,
                    workspace=None, stream=None):
    """A step of beam search: the ``keep`` best continuations of each batch item's beams, by the
    beam's score and the token's log-probability.  ``logits``: ``[batch * beams, n]``; ``scores``:
    float32 ``[batch, beams]``, -inf for a beam that is not in use yet; ``done``: bool or uint8
    ``[batch, beams]``, a beam that offers the token ``end`` only, at its score.  Returns a
    :class:`BeamChoice`: ``scores`` (float32 ``[batch, keep]``, decreasing), ``beams`` (int32: the
    beam that each continues) and ``tokens`` (int64), both -1 where nothing is left, ``row_status``
    (int32 ``[batch * beams]``)."""
    code, rows, n, stride, dev = _scores(logits)
    torch = _torch()
    if not isinstance(scores, torch.Tensor) or scores.dim() != 2:
        raise ValueError("scores must be [batch, beams]")
    batch, beams = scores.shape
    _check(scores, "scores", torch.float32, scores.shape, dev)
    if logits.dim() != 2 or rows != batch * beams:
        raise ValueError("logits must be [batch * beams, n]")
    if not 1 <= beams <= MAX_BEAMS or not 1 <= keep <= MAX_KEEP:
        raise ValueError(f"1 to {MAX_BEAMS} beams, and 1 <= keep <= {MAX_KEEP}")
    if done is not None:
        _mask(done, "done", scores.shape, dev)
        if not 0 <= end < n:
            raise ValueError("end must be one of the tokens")
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_beam_choose(logits, scores, keep, done, end=end, temperature=temperature,
                                   workspace=workspace)
    need = _obj._abi.iso_beam_choose_workspace_bytes(batch, beams, n, code, keep)
    best = torch.empty((batch, keep), dtype=torch.float32, device=dev)
    parents = torch.empty((batch, keep), dtype=torch.int32, device=dev)
    tokens = torch.empty((batch, keep), dtype=torch.int64, device=dev)
    ahead = need if workspace is None else 0
    buf = torch.empty((ahead >> 2) + rows, dtype=torch.int32, device=dev)
    ws, ws_bytes = (buf.data_ptr(), need) if workspace is None else _own_workspace(workspace, dev)
    _done(_obj._abi.iso_beam_choose(
        logits.data_ptr(), code, batch, beams, n, stride, scores.data_ptr(), _ptr(done), end,
        temperature, keep, best.data_ptr(), parents.data_ptr(), tokens.data_ptr(), ws, ws_bytes,
        buf.data_ptr() + ahead, _obj._raw_stream(dev.index)), "iso_beam_choose")
    return BeamChoice(best, parents, tokens, buf, rows)


def _layout(shape, stride, rows, batch):
    """(row stride, runs, run stride, elements of a run) of a state, in elements; None where a row is
    not runs of equal length at equal distances (its dimensions may be in any order)."""
    if shape[0] != rows:   # [batch, beams, ...]: one dimension of rows
        if len(shape) < 2 or shape[0] != batch or shape[0] * shape[1] != rows:
            return None
        if shape[0] > 1 and shape[1] > 1 and stride[0] != shape[1] * stride[1]:
            return None
        row = stride[1] if shape[1] > 1 else stride[0]
        shape, stride = shape[2:], stride[2:]
    else:
        row = stride[0]
        shape, stride = shape[1:], stride[1:]
    inner, runs, apart = 1, 1, 0
    for step, size in sorted((step, size) for size, step in zip(shape, stride) if size > 1):
        if runs == 1 and step == inner:
            inner *= size
        elif runs == 1:
            runs, apart = size, step
        elif step == runs * apart:
            runs *= size
        else:
            return None
    return row, runs, apart, inner


def iso_beam_reorder(states, beams, *, stream=None):
    """Puts the states of beams, in place, where their continuations are: row ``item * beams + b`` of
    each state becomes what row ``item * beams + parents[item, b]`` was, ``parents`` being ``beams``
    (int32 ``[batch, beams]``, as :func:`iso_beam_choose` returns it).  ``states``: a CUDA tensor
    or a list of them, of any type, ``[batch * beams, ...]`` or ``[batch, beams, ...]``; a view of
    the part in use (``cache[:, :, :length]``) moves no more than that.  Beyond its rows a state may
    be contiguous but for one dimension.  States may not share memory.  Returns None."""
    torch = _obj._setup() if _obj._dtypes is None else _torch()
    if isinstance(states, torch.Tensor):
        states = [states]
    if not isinstance(beams, torch.Tensor) or not beams.is_cuda or beams.dim() != 2:
        raise ValueError("beams must be a CUDA tensor [batch, beams]")
    batch, width = beams.shape
    dev = beams.device
    _check(beams, "beams", torch.int32, beams.shape, dev)
    if not 1 <= width <= MAX_BEAMS:
        raise ValueError(f"1 to {MAX_BEAMS} beams")
    rows = batch * width
    if not all(issubclass(kind, torch.Tensor) for kind in set(map(type, states))):
        raise ValueError("states must be tensors")
    words, bases = [], set()
    layouts, last, got = {}, None, ()
    for x in states:
        kind = (x.shape, x.stride(), x.dtype, x.device, x.requires_grad)
        if kind != last:   # (states of one call mostly have one layout)
            got, last = layouts.get(kind), kind
            if got is None:
                if kind[3] != dev:
                    raise ValueError(f"states must be tensors on {dev}")
                if kind[4] and torch.is_grad_enabled():
                    raise ValueError("states are moved in place: they may not require a gradient")
                got = layouts[kind] = _described(x, rows, batch)
        if got:
            base = x.data_ptr()
            bases.add(base)
            words += (base,) + got
    if 5 * len(bases) != len(words):
        raise ValueError("states may not share memory")
    there = _elsewhere(torch, dev, stream)
    if there is None:
        _reorder(words, batch, width, beams)
    else:
        with there:
            _reorder(words, batch, width, beams)
    # a graph that has saved a state for its backward finds that it was changed
    torch.autograd.graph.increment_version(states)


def _described(x, rows, batch):
    """iso_state's numbers behind the base, in bytes; () for a state without elements."""
    shape = x.shape
    if x.dim() < 1 or (shape[0] != rows and shape[0] != batch):
        raise ValueError("states must be [batch * beams, ...] or [batch, beams, ...]")
    if 0 in shape:
        return ()
    got = _layout(shape, x.stride(), rows, batch)
    if got is None:
        raise ValueError("a state may be contiguous but for one dimension beyond its rows")
    size = x.element_size()
    row, runs, apart, inner = got
    return row * size, runs, apart * size, inner * size


def _reorder(words, batch, width, beams):
    # iso_state: five 64-bit numbers
    table = (ctypes.c_int64 * len(words))(*words)
    _done(_obj._abi.iso_beam_reorder(table, len(words) // 5, batch, width, beams.data_ptr(),
                                     _obj._raw_stream(beams.device.index)), "iso_beam_reorder")


def _make():
    torch = _torch()

    class _FirstOnly(torch.autograd.Function):
        @staticmethod
        def forward(ctx, d, logits):
            return d.detach()

        @staticmethod
        def backward(ctx, g):
            raise RuntimeError("the choices have first derivatives only")

    class _Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, top_k, mask, options):
            r = iso_route(logits, top_k, mask, want_grad=ctx.needs_input_grad[0], **options)
            ctx.save_for_backward(logits, r.gates, r.experts, r.counts, r.picked)
            ctx.how = (r.score, r.renormalize, r.scale)
            ctx.mark_non_differentiable(r.experts, r.counts)
            return r.gates, r.experts, r.counts

        @staticmethod
        def backward(ctx, g, *_):
            logits, gates, experts, counts, picked = ctx.saved_tensors
            d = iso_route_backward(g.contiguous(), logits, Route(gates, experts, counts, *ctx.how, picked))
            # (a kernel's output, without a graph of its own: its derivative is refused)
            if torch.is_grad_enabled() and logits.requires_grad:
                d = _FirstOnly.apply(d, logits)
            return d, None, None, None

    return _Route


_Fn = None


def route(logits, top_k: int, mask=None, *, score: str = "softmax", bias=None, groups: int = 1,
          top_groups: int = 1, group_best: int = 2, renormalize: bool = False, scale: float = 1.0):
    """Differentiable router: returns ``(gates, experts, counts)``, of which the gates carry a
    gradient to the logits (the bias has none)."""
    global _Fn
    if _Fn is None:
        _Fn = _make()
    options = {"score": score, "bias": bias, "groups": int(groups), "top_groups": int(top_groups),
               "group_best": int(group_best), "renormalize": bool(renormalize), "scale": float(scale)}
    return _Fn.apply(logits, int(top_k), mask, options)
