"""Training objectives over rows of scores, each with its gradient.

What a model trained on ranks and preferences needs beside the fit: rewards
calibrated by :func:`iso_fit`, or their :func:`soft_rank.soft_rank`, enter a
policy or preference loss over the log-probabilities of a model's tokens, and a
router of experts adds its balance loss.  With ``x`` a row's scores (logits),
``l`` its label and ``T`` the temperature,

    lp = x[l] / T - log sum_j exp(x[j] / T),   d lp / d x[j] = ([j == l] - p[j]) / T.

Explicit calls (same names and arguments as the C ABI of ``include/iso.h``,
which states the formulas, the masks and the errors in full):

* :func:`iso_token_logp`, :func:`iso_token_logp_backward`
* :func:`iso_policy_loss` -- loss and gradient in one call
* :func:`iso_preference_loss` -- loss and gradient in one call
* :func:`iso_balance_loss`, :func:`iso_balance_loss_backward`

Differentiable in the scores (autograd): :func:`token_logp`, :func:`policy_loss`,
:func:`preference_loss`, :func:`balance_loss` (first derivatives only).

Scores are float32, bfloat16 or float16 CUDA tensors, ``[rows, n]`` or ``[n]``,
contiguous within a row (rows may be strided); gradients have their type.
Labels are int64, and a negative one marks a row that takes no part.  Calls
run on ``stream`` (default: the current one); what they allocate belongs to it.
"""
from __future__ import annotations

from . import ISO_OK, IsoError, _torch, load_library

MAX_EXPERTS = 1024   # ISO_MAX_EXPERTS
MAX_TOP_K = 32       # ISO_MAX_TOP_K
ISO_ROW_BAD_LABEL = 8
KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}

class _Result:
    """Named outputs, some of them views of one buffer that are made when they are asked for."""
    _fields = ()
    __slots__ = ("_buf", "_rows", "_shape")

    def __iter__(self):
        return (getattr(self, name) for name in self._fields)

    def __len__(self):
        return len(self._fields)

    # the buffer's tail, in 4-byte words: norm [rows, 2], coef [rows], row_status [rows]
    def _tail(self, first, end):
        at = self._buf.numel() - 4 * self._rows
        return self._buf[at + first * self._rows:at + end * self._rows]

    @property
    def norm(self):
        return self._tail(0, 2).view(self._rows, 2)

    @property
    def coef(self):
        return self._tail(2, 3).view(self._shape)

    @property
    def row_status(self):
        return self._tail(3, 4).view(_torch().int32)


class PolicyLoss(_Result):
    """What :func:`iso_policy_loss` returns."""
    _fields = ("loss", "stats", "logp", "norm", "coef", "dlogits", "row_status")
    __slots__ = ("loss", "stats", "logp", "dlogits")


class PreferenceLoss(_Result):
    """What :func:`iso_preference_loss` returns."""
    _fields = ("loss", "margins", "seq_logp", "logp", "norm", "coef", "dlogits", "row_status", "pair_status")
    __slots__ = ("loss", "margins", "seq_logp", "logp", "dlogits")

    @property
    def pair_status(self):
        return self._buf[:self.margins.numel()].view(_torch().int32)


class BalanceLoss:
    """What :func:`iso_balance_loss` returns."""
    _fields = ("loss", "counts", "experts", "gates", "live", "mask", "renormalize")
    __slots__ = ("loss", "counts", "experts", "gates", "mask", "renormalize", "_buf")

    def __init__(self, loss, counts, experts, gates, buf, mask, renormalize):
        self.loss, self.counts, self.experts, self.gates = loss, counts, experts, gates
        self._buf, self.mask, self.renormalize = buf, mask, renormalize

    def __iter__(self):
        return (getattr(self, name) for name in self._fields)

    def __len__(self):
        return len(self._fields)

    @property
    def live(self):
        return self._buf[0]   # int64; the call's workspace follows


_abi = None      # the loaded library
_dtypes = None
_raw_stream = None


def _setup():
    global _abi, _dtypes, _raw_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _abi = load_library()
    _raw_stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
    # last: calls, of other threads too, take this one for all three
    _dtypes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    return torch


def _scores(t, name="logits"):
    """(dtype code, rows, n, row stride, device) of a tensor of scores."""
    torch = _setup() if _dtypes is None else _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _dtypes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    dim = t.dim()
    if dim == 2:
        rows, n = t.shape
        stride, inner = t.stride()
    elif dim == 1:
        rows, n, inner = 1, t.shape[0], t.stride(0)
        stride = n
    else:
        raise ValueError(f"{name} must be [n] or [rows, n]")
    if n < 1:
        raise ValueError(f"{name} must have at least one score a row")
    if inner != 1 and n > 1:
        raise ValueError(f"{name} must be contiguous within a row")
    return code, rows, n, stride, t.device


def _check(t, name, dtype, shape, device):
    if getattr(t, "dtype", None) == dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if not isinstance(t, _torch().Tensor) or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check_out(t, like):
    """A caller's gradient buffer: its row stride."""
    _, rows, n, stride, _ = _scores(t, "out")
    if t.dtype != like.dtype or t.shape != like.shape or t.device != like.device:
        raise ValueError("out must have the logits' shape, type and device")
    if rows > 1 and stride < n:
        raise ValueError("out's rows must not overlap")
    return stride


def _like(torch, t, rows, n, stride):
    """A gradient's buffer beside the scores t, with their row stride where rows are only
    padded: its rows are then aligned as theirs."""
    if n <= stride <= n + max(64, n >> 3) and t.dim() == 2:
        return torch.empty_strided((rows, n), (stride, 1), dtype=t.dtype, device=t.device), stride
    return torch.empty(t.shape, dtype=t.dtype, device=t.device), n


def _elsewhere(torch, device, stream):
    """None where the call belongs on the current device's current stream; otherwise the
    context that makes it so."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return None


def _done(status, name):
    if status != ISO_OK:
        raise IsoError(status, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _own_workspace(workspace, device):
    torch = _torch()
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or \
            workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace.data_ptr(), workspace.numel()


def iso_token_logp(logits, labels, *, temperature: float = 1.0, workspace=None, stream=None):
    """The labels' log-probabilities.  Returns ``(logp, norm, row_status)``: float32 of the
    labels' shape; the rows' softmax statistics ``[rows, 2]`` for the backward; int32 ``[rows]``."""
    code, rows, n, stride, dev = _scores(logits)
    torch = _torch()
    _check(labels, "labels", torch.int64, logits.shape[:-1], dev)
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_token_logp(logits, labels, temperature=temperature, workspace=workspace)
    logp = torch.empty(labels.shape, dtype=torch.float32, device=dev)
    norm = torch.empty((rows, 2), dtype=torch.float32, device=dev)
    status = torch.empty(rows, dtype=torch.int32, device=dev)
    need = _abi.iso_token_logp_workspace_bytes(rows)
    ws = None
    if workspace is not None:
        ws, need = _own_workspace(workspace, dev)
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws = workspace.data_ptr()
    _done(_abi.iso_token_logp(
        logits.data_ptr(), code, rows, n, stride, labels.data_ptr(), temperature, logp.data_ptr(),
        norm.data_ptr(), ws, need, status.data_ptr(), _raw_stream(dev.index)), "iso_token_logp")
    return logp, norm, status


def iso_token_logp_backward(grad_logp, logits, labels, norm, *, temperature: float = 1.0,
                            grad_scale: float = 1.0, grad_scale_dev=None,
                            changed_only: bool = False, out=None, stream=None):
    """The gradient of ``grad_scale * grad_scale_dev * sum(grad_logp * logp)`` in the logits.
    ``norm`` is the forward's.  With ``changed_only`` and ``out`` given, nothing is written
    when the device scalar ``grad_scale_dev`` is 1.  ``out`` may be the logits themselves."""
    code, rows, n, stride, dev = _scores(logits)
    torch = _torch()
    _check(labels, "labels", torch.int64, logits.shape[:-1], dev)
    _check(grad_logp, "grad_logp", torch.float32, labels.shape, dev)
    _check(norm, "norm", torch.float32, (rows, 2), dev)
    if grad_scale_dev is not None:
        _check(grad_scale_dev, "grad_scale_dev", torch.float32, (), dev)
    if changed_only and out is None:
        raise ValueError("changed_only needs out")
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_token_logp_backward(
                grad_logp, logits, labels, norm, temperature=temperature, grad_scale=grad_scale,
                grad_scale_dev=grad_scale_dev, changed_only=changed_only, out=out)
    if out is None:
        out, out_stride = _like(torch, logits, rows, n, stride)
    else:
        out_stride = _check_out(out, logits)
    _done(_abi.iso_token_logp_backward(
        logits.data_ptr(), code, rows, n, stride, labels.data_ptr(), temperature, norm.data_ptr(),
        grad_logp.data_ptr(), grad_scale, _ptr(grad_scale_dev), bool(changed_only), out.data_ptr(),
        out_stride, _raw_stream(dev.index)), "iso_token_logp_backward")
    return out


def iso_policy_loss(logits, labels, old_logp, advantages, ref_logp=None, weights=None, *,
                    clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                    temperature: float = 1.0, grad_scale: float = 1.0, want_grad: bool = True,
                    out=None, workspace=None, stream=None):
    """Clipped policy loss with a KL term, and its gradient in the logits, in one pass over
    them.  Returns a :class:`PolicyLoss`: ``loss`` (scalar), ``stats`` (``[3]``: policy term,
    KL term, share of clipped rows), ``logp``, ``norm``, ``coef`` (the loss's derivative in
    ``logp``), ``dlogits`` (None without ``want_grad``; times ``grad_scale``; written to ``out``
    when given, which may be the logits themselves), ``row_status``."""
    code, rows, n, stride, dev = _scores(logits)
    torch = _torch()
    f32 = torch.float32
    shape = logits.shape[:-1]
    _check(labels, "labels", torch.int64, shape, dev)
    _check(old_logp, "old_logp", f32, shape, dev)
    _check(advantages, "advantages", f32, shape, dev)
    if ref_logp is not None:
        _check(ref_logp, "ref_logp", f32, shape, dev)
    if weights is not None:
        _check(weights, "weights", f32, shape, dev)
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_policy_loss(
                logits, labels, old_logp, advantages, ref_logp, weights, clip_low=clip_low,
                clip_high=clip_high, kl_coef=kl_coef, temperature=temperature,
                grad_scale=grad_scale, want_grad=want_grad, out=out, workspace=workspace)
    need = _abi.iso_policy_loss_workspace_bytes(rows)
    r = PolicyLoss()
    r._rows, r._shape = rows, shape
    r.loss = loss = torch.empty((), dtype=f32, device=dev)
    r.stats = stats = torch.empty(3, dtype=f32, device=dev)
    r.logp = logp = torch.empty(shape, dtype=f32, device=dev)
    r._buf = buf = torch.empty((need >> 2) + 4 * rows, dtype=f32, device=dev)
    ws, ws_bytes = (buf.data_ptr(), need) if workspace is None else _own_workspace(workspace, dev)
    rest = buf.data_ptr() + need
    out_stride = n
    if out is not None:
        out_stride = _check_out(out, logits)
    elif want_grad:
        out, out_stride = _like(torch, logits, rows, n, stride)
    r.dlogits = out
    _done(_abi.iso_policy_loss(
        logits.data_ptr(), code, rows, n, stride, labels.data_ptr(), temperature,
        old_logp.data_ptr(), advantages.data_ptr(), _ptr(ref_logp), _ptr(weights), clip_low,
        clip_high, kl_coef, grad_scale, loss.data_ptr(), stats.data_ptr(), logp.data_ptr(), rest,
        rest + 8 * rows, _ptr(out), out_stride, ws, ws_bytes, rest + 12 * rows,
        _raw_stream(dev.index)), "iso_policy_loss")
    return r


def iso_preference_loss(logits, labels, offsets, ref_logp=None, *, kind: str = "sigmoid",
                        beta: float = 0.1, label_smoothing: float = 0.0, average: bool = False,
                        grad_scale: float = 1.0, want_grad: bool = True, out=None,
                        workspace=None, stream=None):
    """Preference loss over pairs of token sequences laid end to end, and its gradient in the
    logits.  ``offsets``: int64 CUDA tensor of ``2 * pairs + 1`` entries (not read by the
    host); sequence ``2q`` is pair q's chosen one, ``2q + 1`` its rejected one.  ``kind``:
    "sigmoid", "hinge" or "squared".  Returns a :class:`PreferenceLoss`."""
    code, rows, n, stride, dev = _scores(logits)
    torch = _torch()
    f32 = torch.float32
    shape = logits.shape[:-1]
    _check(labels, "labels", torch.int64, shape, dev)
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() % 2 != 1:
        raise ValueError("offsets must hold 2 * pairs + 1 entries")
    _check(offsets, "offsets", torch.int64, offsets.shape, dev)
    how = KINDS.get(kind)
    if how is None:
        raise ValueError(f"kind must be one of {sorted(KINDS)}")
    if ref_logp is not None:
        _check(ref_logp, "ref_logp", f32, shape, dev)
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_preference_loss(
                logits, labels, offsets, ref_logp, kind=kind, beta=beta,
                label_smoothing=label_smoothing, average=average, grad_scale=grad_scale,
                want_grad=want_grad, out=out, workspace=workspace)
    pairs = offsets.numel() // 2
    need = _abi.iso_preference_loss_workspace_bytes(rows, pairs)
    r = PreferenceLoss()
    r._rows, r._shape = rows, shape
    r.loss = loss = torch.empty((), dtype=f32, device=dev)
    r.margins = margins = torch.empty(pairs, dtype=f32, device=dev)
    r.seq_logp = seq_logp = torch.empty(2 * pairs, dtype=f32, device=dev)
    r.logp = logp = torch.empty(shape, dtype=f32, device=dev)
    head = (pairs + 63) // 64 * 256   # bytes of the pairs' statuses, the workspace behind them
    r._buf = buf = torch.empty((head + need >> 2) + 4 * rows, dtype=f32, device=dev)
    pair_status = buf.data_ptr()
    ws, ws_bytes = (pair_status + head, need) if workspace is None else _own_workspace(workspace, dev)
    rest = pair_status + head + need
    out_stride = n
    if out is not None:
        out_stride = _check_out(out, logits)
    elif want_grad:
        out, out_stride = _like(torch, logits, rows, n, stride)
    r.dlogits = out
    _done(_abi.iso_preference_loss(
        logits.data_ptr(), code, rows, n, stride, labels.data_ptr(), offsets.data_ptr(), pairs,
        _ptr(ref_logp), how, beta, label_smoothing, bool(average), grad_scale, loss.data_ptr(),
        margins.data_ptr(), seq_logp.data_ptr(), logp.data_ptr(), rest, rest + 8 * rows, _ptr(out),
        out_stride, ws, ws_bytes, rest + 12 * rows, pair_status,
        _raw_stream(dev.index)), "iso_preference_loss")
    return r


def _router(logits, top_k, mask):
    code, tokens, experts, stride, dev = _scores(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    if experts > MAX_EXPERTS or not 1 <= top_k <= min(experts, MAX_TOP_K):
        raise ValueError(f"at most {MAX_EXPERTS} experts, and 1 <= top_k <= min(experts, {MAX_TOP_K})")
    torch = _torch()
    if mask is not None:   # (a bool is a byte of 0 or 1)
        dtype = torch.bool if getattr(mask, "dtype", None) == torch.bool else torch.uint8
        _check(mask, "mask", dtype, logits.shape[:1], dev)
    return torch, code, tokens, experts, stride, dev


def iso_balance_loss(logits, top_k: int, mask=None, *, renormalize: bool = False, workspace=None,
                     stream=None):
    """A router's choice of ``top_k`` experts for each row of ``logits`` ``[tokens, experts]``,
    its balance loss and the tokens of each expert.  ``mask``: bool or uint8 ``[tokens]``, false
    where a token takes no part.  Returns a :class:`BalanceLoss`: ``loss`` (scalar), ``counts``
    (int64 ``[experts]``), ``experts`` (int32 ``[tokens, top_k]``, -1 where none), ``gates``
    (float32), ``live`` (int64 scalar: the tokens that take part), ``mask``, ``renormalize``."""
    torch, code, tokens, experts, stride, dev = _router(logits, top_k, mask)
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_balance_loss(logits, top_k, mask, renormalize=renormalize, workspace=workspace)
    need = _abi.iso_balance_loss_workspace_bytes(tokens, experts)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty(experts, dtype=torch.int64, device=dev)
    chosen = torch.empty((tokens, top_k), dtype=torch.int32, device=dev)
    gates = torch.empty((tokens, top_k), dtype=torch.float32, device=dev)
    buf = torch.empty(32 + (need >> 3 if workspace is None else 0), dtype=torch.int64, device=dev)
    live = buf.data_ptr()
    ws, ws_bytes = (live + 256, need) if workspace is None else _own_workspace(workspace, dev)
    renormalize = bool(renormalize)
    _done(_abi.iso_balance_loss(
        logits.data_ptr(), code, tokens, experts, stride, top_k, _ptr(mask), renormalize,
        loss.data_ptr(), counts.data_ptr(), chosen.data_ptr(), gates.data_ptr(), live, ws, ws_bytes,
        _raw_stream(dev.index)), "iso_balance_loss")
    return BalanceLoss(loss, counts, chosen, gates, buf, mask, renormalize)


def iso_balance_loss_backward(logits, result, *, grad_loss: float = 1.0, grad_loss_dev=None,
                              grad_gates=None, out=None, stream=None):
    """The gradient of ``grad_loss * grad_loss_dev * loss + sum(grad_gates * gates)`` in the
    logits, ``result`` being :func:`iso_balance_loss`'s for them."""
    if not isinstance(result, BalanceLoss):
        raise ValueError("result must be iso_balance_loss's")
    shape = result.experts.shape
    mask = result.mask
    torch, code, tokens, experts, stride, dev = _router(logits, shape[1], mask)
    if shape[0] != tokens or result.counts.numel() != experts or result.counts.device != dev:
        raise ValueError("logits must have the shape and device that result was made for")
    if grad_gates is not None:
        _check(grad_gates, "grad_gates", torch.float32, shape, dev)
    if grad_loss_dev is not None:
        _check(grad_loss_dev, "grad_loss_dev", torch.float32, (), dev)
    there = _elsewhere(torch, dev, stream)
    if there is not None:
        with there:
            return iso_balance_loss_backward(logits, result, grad_loss=grad_loss,
                                             grad_loss_dev=grad_loss_dev, grad_gates=grad_gates,
                                             out=out)
    if out is None:
        out, out_stride = _like(torch, logits, tokens, experts, stride)
    else:
        out_stride = _check_out(out, logits)
    _done(_abi.iso_balance_loss_backward(
        logits.data_ptr(), code, tokens, experts, stride, shape[1], _ptr(mask),
        result.renormalize, result.counts.data_ptr(), result.experts.data_ptr(),
        result.gates.data_ptr(), result._buf.data_ptr(), _ptr(grad_gates), grad_loss,
        _ptr(grad_loss_dev), out.data_ptr(), out_stride, _raw_stream(dev.index)),
        "iso_balance_loss_backward")
    return out


def _make():
    torch = _torch()

    class _FirstOnly(torch.autograd.Function):
        @staticmethod
        def forward(ctx, d, logits):
            return d.detach()

        @staticmethod
        def backward(ctx, g):
            raise RuntimeError("the objectives have first derivatives only")

    def first_only(d, logits):
        # A gradient is a kernel's output, without a graph of its own: where one is asked for
        # (create_graph), its derivative is refused and not taken for 0.
        return _FirstOnly.apply(d, logits) if torch.is_grad_enabled() and logits.requires_grad else d

    class _TokenLogp(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, labels, temperature):
            logp, norm, _ = iso_token_logp(logits, labels, temperature=temperature)
            ctx.save_for_backward(logits, labels, norm)
            ctx.temperature = temperature
            return logp

        @staticmethod
        def backward(ctx, g):
            logits, labels, norm = ctx.saved_tensors
            d = iso_token_logp_backward(g.contiguous(), logits, labels, norm, temperature=ctx.temperature)
            return first_only(d, logits), None, None

    def hand_over(ctx, g):
        # The forward left the gradient for an upstream gradient of 1.  It is handed out once
        # (rewritten when g is not 1); a further backward through the same graph forms it anew.
        logits, labels, norm, coef = ctx.saved_tensors
        held, ctx.dlogits = ctx.dlogits, None
        d = iso_token_logp_backward(coef, logits, labels, norm, temperature=ctx.temperature,
                                    grad_scale_dev=g.contiguous(), changed_only=held is not None, out=held)
        return first_only(d, logits)

    class _PolicyLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, labels, old_logp, advantages, ref_logp, weights, options):
            r = iso_policy_loss(logits, labels, old_logp, advantages, ref_logp, weights,
                                want_grad=ctx.needs_input_grad[0], **options)
            ctx.save_for_backward(logits, labels, r.norm, r.coef)
            ctx.temperature, ctx.dlogits = options["temperature"], r.dlogits
            ctx.mark_non_differentiable(r.stats, r.logp)
            return r.loss, r.stats, r.logp

        @staticmethod
        def backward(ctx, g, *_):
            return (hand_over(ctx, g),) + (None,) * 6

    class _PreferenceLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, labels, offsets, ref_logp, options):
            r = iso_preference_loss(logits, labels, offsets, ref_logp,
                                    want_grad=ctx.needs_input_grad[0], **options)
            ctx.save_for_backward(logits, labels, r.norm, r.coef)
            ctx.temperature, ctx.dlogits = 1.0, r.dlogits
            ctx.mark_non_differentiable(r.margins, r.seq_logp)
            return r.loss, r.margins, r.seq_logp

        @staticmethod
        def backward(ctx, g, *_):
            return (hand_over(ctx, g),) + (None,) * 4

    class _BalanceLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, top_k, mask, renormalize):
            ctx.set_materialize_grads(False)
            r = iso_balance_loss(logits, top_k, mask, renormalize=renormalize)
            ctx.save_for_backward(logits, r.counts, r.experts, r.gates, r._buf, r.mask)
            ctx.renormalize = renormalize
            ctx.mark_non_differentiable(r.counts, r.experts)
            return r.loss, r.gates, r.counts, r.experts

        @staticmethod
        def backward(ctx, g_loss, g_gates, *_):
            logits, counts, experts, gates, buf, mask = ctx.saved_tensors
            if g_loss is None and g_gates is None:
                return (None,) * 4
            r = BalanceLoss(None, counts, experts, gates, buf, mask, ctx.renormalize)
            d = iso_balance_loss_backward(
                logits, r, grad_loss=0.0 if g_loss is None else 1.0,
                grad_loss_dev=None if g_loss is None else g_loss.contiguous(),
                grad_gates=None if g_gates is None else g_gates.contiguous())
            return first_only(d, logits), None, None, None

    return {"token": _TokenLogp, "policy": _PolicyLoss, "preference": _PreferenceLoss,
            "balance": _BalanceLoss}


_Fn = None


def _fn(name):
    global _Fn
    if _Fn is None:
        _Fn = _make()
    return _Fn[name]


def token_logp(logits, labels, temperature: float = 1.0):
    """Differentiable log-probabilities of the labels (0 where a label is negative)."""
    return _fn("token").apply(logits, labels, float(temperature))


def policy_loss(logits, labels, old_logp, advantages, ref_logp=None, weights=None, *,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                temperature: float = 1.0):
    """Differentiable clipped policy loss; returns ``(loss, stats, logp)``, of which only the
    loss carries a gradient (to the logits)."""
    options = {"clip_low": float(clip_low), "clip_high": float(clip_high),
               "kl_coef": float(kl_coef), "temperature": float(temperature)}
    return _fn("policy").apply(logits, labels, old_logp, advantages, ref_logp, weights, options)


def preference_loss(logits, labels, offsets, ref_logp=None, *, kind: str = "sigmoid",
                    beta: float = 0.1, label_smoothing: float = 0.0, average: bool = False):
    """Differentiable preference loss over pairs of sequences; returns ``(loss, margins,
    seq_logp)``, of which only the loss carries a gradient (to the logits)."""
    options = {"kind": kind, "beta": float(beta), "label_smoothing": float(label_smoothing),
               "average": bool(average)}
    return _fn("preference").apply(logits, labels, offsets, ref_logp, options)


def balance_loss(logits, top_k: int, mask=None, renormalize: bool = False):
    """Differentiable router: returns ``(loss, gates, counts, experts)``; the loss and the
    gates carry gradients to the logits."""
    return _fn("balance").apply(logits, int(top_k), mask, bool(renormalize))
