"""Losses at the vocabulary, from hidden states and the head's weight, with
their gradients, without ever holding the logits.

``xent_*`` is softmax cross entropy; ``distill_*`` is distillation from a
teacher's top-K logits at a temperature, alone or mixed with the cross entropy;
``policy_*`` is the clipped policy loss of sampled tokens, kept near a reference;
``preference_*`` the loss of pairs of a preferred and a rejected sequence (the
definitions, and what an empty row is, stand in ``include/zero_gb300.h`` at
``zero_head_loss_t`` and ``zero_policy_t``). Each comes as

- ``*_forward``: the losses;
- ``*_backward``: the gradients, from the forward pass's result;
- ``*_step``: both in one call.

``hidden`` is a [T, D] (or [..., D]) and ``weight`` a [V, D] CUDA tensor, both
float32 or both bfloat16, with adjacent elements in a row and any row stride.
What goes with the rows -- labels, the teacher's entries, ``dloss``, ``lse``, what a
policy loss is given -- has hidden's leading dimensions or the rows in one dimension; beside a [T, D]
``hidden`` it may have any leading dimensions, the same for all.
``dhidden`` and ``dweight`` may be given as outputs -- for ``dweight`` typically
the head's view into a rank's flat gradient buffer, which the ZeRO step then
reads -- and are allocated otherwise; ``accumulate`` adds to ``dweight``.

``linear_cross_entropy``, ``linear_distillation``, ``linear_policy`` and
``linear_preference`` are the same losses as differentiable functions for
torch.autograd. Their gradients can be part of a
graph (``create_graph``), but to differentiate them again raises a RuntimeError.

Work is queued on ``stream``: a ``torch.cuda.Stream``, a raw handle, or None for
the current stream. The workspace and the results that are not given are taken
from PyTorch's allocator for each call, as that stream's, so what the current
stream still does with memory that it has given back is not run into. The
allocator is told that ``stream`` uses the inputs and that the current stream
uses the results; to order the two streams' work is left to the caller.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import abi

_REDUCE = {"none": abi.ZERO_REDUCE_NONE, "mean": abi.ZERO_REDUCE_MEAN, "sum": abi.ZERO_REDUCE_SUM}


class Losses(NamedTuple):
    """``loss`` [T] float32 (0 for an empty row); ``reduced``, its mean over the
    rows that are not empty, or its sum (None for reduction "none"); ``lse`` and
    ``lse_tau``, the rows' log-sum-exp for a backward pass; the gradients, where
    they were taken."""
    loss: torch.Tensor | None
    reduced: torch.Tensor | None
    lse: torch.Tensor | None
    lse_tau: torch.Tensor | None
    dhidden: torch.Tensor | None = None
    dweight: torch.Tensor | None = None


class LogpLosses(NamedTuple):
    """Of the losses that are functions of the labels' log-probabilities: ``loss``
    float32, of each row (policy; 0 for an empty row) or of each pair
    (preference); ``reduced`` as in Losses; ``logps`` the log-probabilities of
    the rows, or their sums over each sequence, and ``counts`` the sequences'
    labelled rows (int32); for a backward pass ``lse``, ``row_logps``, the rows'
    log-probabilities (policy: ``logps`` itself), and ``slopes``, the losses'
    derivatives by them, of each row or of a sequence's rows; the gradients, where
    they were taken."""
    loss: torch.Tensor | None
    reduced: torch.Tensor | None
    logps: torch.Tensor | None
    slopes: torch.Tensor | None
    lse: torch.Tensor | None
    row_logps: torch.Tensor | None
    counts: torch.Tensor | None = None
    dhidden: torch.Tensor | None = None
    dweight: torch.Tensor | None = None


_KINDS = {"sigmoid": abi.ZERO_PREFERENCE_SIGMOID, "squared": abi.ZERO_PREFERENCE_SQUARED}

_PRECISION = {torch.float32: abi.ZERO_FP32, torch.bfloat16: abi.ZERO_BF16_MIXED}


def _matrix(t, what: str, dtype=None, rows=None, cols=None, device=None):
    """``t`` as a matrix [rows, cols] without a copy; (tensor, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    own = t.dtype
    if own is not dtype and (dtype is not None or own not in _PRECISION):
        want = "float32 or bfloat16" if dtype is None else dtype
        raise TypeError(f"{what} has dtype {own}, expected {want}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.dim() != 2:
        if t.dim() < 2:
            raise ValueError(f"{what} must have at least 2 dimensions")
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{what}'s rows must lie one stride apart") from None
    n, d = t.shape
    if (rows is not None and n != rows) or (cols is not None and d != cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected ({rows}, {cols})")
    stride, unit = t.stride()
    if unit != 1 and d > 1 and n > 0:
        raise ValueError(f"the elements of {what}'s rows must be adjacent")
    return t, stride if n > 1 else max(d, 1)


def _vector(t, what: str, dtype, count: int, device) -> int:
    """The address of ``count`` contiguous elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dtype:
        raise TypeError(f"{what} must be a {dtype} CUDA tensor")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {count} elements")
    return t.data_ptr()


def _named(stream, device):
    """``stream`` as the allocator knows it: a handle's memory is given back behind
    its work only if the allocator is told of the stream."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)
    # 1 names the legacy default stream, PyTorch's own default, whose handle is 0.
    return torch.cuda.ExternalStream(0 if handle == 1 else handle, device=device)


class _Call:
    """One call's zero_head_loss_t and the tensors behind its pointers."""

    def __init__(self, hidden, weight, labels, reduction, ignore_index, stream, teacher=None):
        hidden2, hs = _matrix(hidden, "hidden")
        self.dtype, self.device = hidden2.dtype, hidden2.device
        T, D = hidden2.shape
        weight2, ws = _matrix(weight, "weight", self.dtype, cols=D, device=self.device)
        if reduction not in _REDUCE:
            raise ValueError('reduction must be "none", "mean" or "sum"')
        V = weight2.shape[0]
        self.T, self.V, self.D = T, V, D
        self.shape = hidden.shape
        self.lead = hidden.shape[:-1]            # the rows' dimensions
        self.order = None                        # those longer than one, where they are several
        if len(self.lead) > 1:
            self.agree(self.lead, "hidden")
        self.stream = _named(stream, self.device)
        self.distill = teacher is not None
        self.labels = labels is not None
        self.none = reduction == "none"
        self.extra = None                        # a policy's or a preference's part
        self.count = self.T                      # of losses, and of the entries of dloss
        self.loss_shape = self.lead
        self.keep = [hidden2, weight2, labels]   # the caller's tensors
        self.made = []                           # its results
        y = None
        if labels is not None:
            y = self.vector(labels, "labels", torch.int64)
        elif teacher is None:
            raise TypeError("labels must be a torch.int64 CUDA tensor")
        # the fields in order: up to ignore_index
        p = self.p = abi.HeadLoss(T, V, D, _PRECISION[self.dtype], _REDUCE[reduction],
                                  hidden2.data_ptr(), hs, weight2.data_ptr(), ws, y, ignore_index)
        p.grad_scale = 1.0
        if teacher is not None:
            ids, logits, temperature, alpha = teacher
            if not isinstance(ids, torch.Tensor) or ids.dim() < 2:
                raise ValueError("teacher_ids must have at least 2 dimensions")
            K = ids.shape[-1]
            p.teacher_ids = self.vector(ids, "teacher_ids", torch.int64, K)
            self.keep += [ids, logits]
            if isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dtype == torch.bfloat16:
                with torch.cuda.stream(self.stream):     # None: the current one
                    logits = logits.float()
            self.wide = logits               # held until the call is queued
            p.teacher_logits = self.vector(logits, "teacher_logits", torch.float32, K)
            p.teacher_k = K
            p.temperature, p.alpha = float(temperature), float(alpha)

    def agree(self, rows, what):
        """Checks that rows of dimensions ``rows`` come in the order of the others': one dimension
        (beside such of one element) agrees with every other form, several only with the same."""
        long = [n for n in rows if n != 1]
        if len(long) > 1:
            if self.order is not None and long != self.order:
                raise ValueError(f"{what}'s rows have the dimensions {tuple(rows)}, others' {tuple(self.order)}")
            self.order = long

    def vector(self, t, what: str, dtype, last: int | None = None) -> int:
        """The address of contiguous elements, one (or ``last``) for each row."""
        address = _vector(t, what, dtype, self.T if last is None else self.T * last, self.device)
        if last is None:
            if t.dim() > 1:
                self.agree(t.shape, what)
        elif t.dim() < 1 or t.shape[-1] != last:
            raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {last} entries for each row")
        elif t.dim() > 2:
            self.agree(t.shape[:-1], what)
        return address

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def new(self, shape, dtype=torch.float32):
        t = self.empty(shape, dtype)
        self.made.append(t)
        return t

    def statistics(self, lse, lse_tau):
        """The forward pass's, for a backward pass."""
        p = self.p
        if self.labels:
            p.lse = self.vector(lse, "lse", torch.float32)
        if self.distill:
            p.lse_tau = self.vector(lse_tau, "lse_tau", torch.float32)
        self.keep += [lse, lse_tau]

    def losses(self):
        """loss, reduced, lse, lse_tau, to be written."""
        p, T = self.p, self.T
        loss = self.new(self.loss_shape)
        p.loss = loss.data_ptr()
        reduced = lse = lse_tau = None
        if not self.none:
            reduced = self.new(())
            p.reduced = reduced.data_ptr()
        if self.labels:
            lse = self.new(T)
            p.lse = lse.data_ptr()
        if self.distill:
            lse_tau = self.new(T)
            p.lse_tau = lse_tau.data_ptr()
        return loss, reduced, lse, lse_tau

    def gradients(self, dloss, grad_scale, dhidden, dweight, accumulate):
        """dhidden / dweight: a tensor to write, None to allocate one, False to leave it out."""
        p = self.p
        p.grad_scale = grad_scale
        if accumulate:
            p.accumulate = 1
        if dloss is not None:
            p.dloss = (self.vector(dloss, "dloss", torch.float32) if self.none and self.loss_shape is self.lead else
                       _vector(dloss, "dloss", torch.float32, self.count if self.none else 1, self.device))
            self.keep.append(dloss)
        if dhidden is None:
            dhidden = self.new(self.shape, self.dtype)
            p.dhidden, p.dhidden_stride = dhidden.data_ptr(), self.D
        elif dhidden is False:
            dhidden = None
        else:
            m, stride = _matrix(dhidden, "dhidden", self.dtype, self.T, self.D, self.device)
            p.dhidden, p.dhidden_stride = m.data_ptr(), stride
            self.keep.append(m)
        if dweight is None:
            if accumulate:
                raise ValueError("accumulate adds to a dweight that is given")
            dweight = self.new((self.V, self.D), self.dtype)
            p.dweight, p.dweight_stride = dweight.data_ptr(), self.D
        elif dweight is False:
            dweight = None
        else:
            m, stride = _matrix(dweight, "dweight", self.dtype, self.V, self.D, self.device)
            p.dweight, p.dweight_stride = m.data_ptr(), stride
            self.keep.append(m)
        return dhidden, dweight

    def run(self, xent, distill):
        """Queues the call: ``xent`` or ``distill`` of abi, with its workspace."""
        index = self.device.index
        if index != torch.cuda.current_device():
            with torch.cuda.device(index):
                return self.run(xent, distill)
        p = self.p
        more = () if self.extra is None else (self.extra,)
        if self.distill:
            size, call = abi.zero_distill_workspace_bytes(p), distill
        elif not more:
            size, call = abi.zero_xent_workspace_bytes(p), xent
        elif isinstance(self.extra, abi.Policy):
            size, call = abi.zero_policy_workspace_bytes(p, *more), xent
        else:
            size, call = abi.zero_preference_workspace_bytes(p, *more), xent
        space = self.empty(size, torch.uint8)
        p.workspace, p.workspace_bytes = space.data_ptr(), size
        stream = self.stream
        if stream is not None:
            for t in self.keep:
                if t is not None:
                    t.record_stream(stream)
            current = torch.cuda.current_stream(self.device)
            for t in self.made:
                t.record_stream(current)
        # the current stream's handle, without the object around it
        call(p, *more, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream)

    def policy(self, old_logps=None, advantages=None, ref_logps=None, clip=0.0, kl_weight=0.0, forward=True):
        """Makes it a policy loss; ``forward``: with what a forward pass is given."""
        q = self.extra = abi.Policy()
        if not forward:
            return
        q.clip_low, q.clip_high = (clip, clip) if isinstance(clip, (int, float)) else clip
        q.kl_weight = kl_weight
        q.old_logps = self.vector(old_logps, "old_logps", torch.float32)
        q.advantages = self.vector(advantages, "advantages", torch.float32)
        self.keep += [old_logps, advantages]
        if ref_logps is not None:
            q.ref_logps = self.vector(ref_logps, "ref_logps", torch.float32)
            self.keep.append(ref_logps)
        elif kl_weight != 0.0:
            raise ValueError("kl_weight weighs the distance from ref_logps, which are not given")

    def preference(self, offsets, **options):
        """Makes it a preference loss; the options: a forward pass's."""
        q = self.extra = abi.Preference()
        if offsets is not None:
            if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] % 2 == 0:
                raise ValueError("offsets must have one dimension of 2 * pairs + 1 entries")
            q.pairs = offsets.shape[0] // 2
            q.offsets = _vector(offsets, "offsets", torch.int64, 2 * q.pairs + 1, self.device)
            self.keep.append(offsets)
        else:
            if len(self.lead) != 2 or self.lead[0] % 2:
                raise ValueError("without offsets hidden must be [2 * pairs, length, D]")
            q.pairs = self.lead[0] // 2
        self.count, self.loss_shape = q.pairs, (q.pairs,)
        if not options:
            return
        kind, ref_logps = options["kind"], options["ref_logps"]
        if kind not in _KINDS:
            raise ValueError('kind must be "sigmoid" or "squared"')
        q.kind, q.average = _KINDS[kind], 1 if options["average"] else 0
        q.beta, q.smoothing, q.margin = options["beta"], options["smoothing"], options["margin"]
        q.nll_weight = options["nll_weight"]
        if ref_logps is not None:
            q.ref_logps = _vector(ref_logps, "ref_logps", torch.float32, 2 * q.pairs, self.device)
            self.keep.append(ref_logps)

    def slopes(self, lse, row_logps, slopes):
        """The forward pass's, for a backward pass."""
        q = self.extra
        self.p.lse = self.vector(lse, "lse", torch.float32)
        rows = self.vector(row_logps, "row_logps", torch.float32)
        if isinstance(q, abi.Policy):
            q.logps, q.slopes = rows, self.vector(slopes, "slopes", torch.float32)
        else:
            q.row_logps = rows
            q.slopes = _vector(slopes, "slopes", torch.float32, 2 * self.count, self.device)
        self.keep += [lse, row_logps, slopes]

    def logp_losses(self):
        """The fields of a LogpLosses but for the gradients, to be written."""
        q = self.extra
        loss, reduced, lse, _ = self.losses()
        logps = rows = self.new(self.lead)
        counts = None
        if isinstance(q, abi.Policy):
            slopes = self.new(self.lead)
        else:
            q.row_logps = rows.data_ptr()
            logps, slopes = self.new(2 * q.pairs), self.new(2 * q.pairs)
            counts = self.new(2 * q.pairs, torch.int32)
            q.counts = counts.data_ptr()
        q.logps, q.slopes = logps.data_ptr(), slopes.data_ptr()
        return loss, reduced, logps, slopes, lse, rows, counts


def xent_forward(hidden, weight, labels, *, reduction: str = "mean", ignore_index: int = -100,
                 stream=None) -> Losses:
    """Cross entropy of every row against ``labels`` (int64 [T])."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    out = c.losses()
    c.run(abi.zero_xent_forward, None)
    return Losses(*out)


def xent_backward(hidden, weight, labels, lse, *, reduction: str = "mean",
                  ignore_index: int = -100, dloss=None, grad_scale: float = 1.0, dhidden=None,
                  dweight=None, accumulate: bool = False, stream=None) -> Losses:
    """The gradients, given ``lse`` of xent_forward on the same inputs.
    ``dloss`` (float32): the gradient of the total with respect to ``loss``
    (reduction "none") or to ``reduced``; ones when None."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    c.statistics(lse, None)
    dh, dw = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(abi.zero_xent_backward, None)
    return Losses(None, None, lse, None, dh, dw)


def xent_step(hidden, weight, labels, *, reduction: str = "mean", ignore_index: int = -100,
              dloss=None, grad_scale: float = 1.0, dhidden=None, dweight=None,
              accumulate: bool = False, stream=None) -> Losses:
    """xent_forward and xent_backward in one call."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    out = c.losses()
    grads = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(abi.zero_xent_step, None)
    return Losses(*out, *grads)


def distill_forward(hidden, weight, teacher_ids, teacher_logits, *, temperature: float = 1.0,
                    labels=None, alpha: float = 1.0, reduction: str = "mean",
                    ignore_index: int = -100, stream=None) -> Losses:
    """Distillation from the teacher's top logits (``teacher_ids`` int64 [T, K],
    ``teacher_logits`` float32 or bfloat16 [T, K]; an id outside [0, V) is an
    absent entry, and so is a logit of -inf), weighted ``alpha``, and with ``labels``
    the cross entropy, weighted ``1 - alpha``."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream,
              (teacher_ids, teacher_logits, temperature, alpha))
    out = c.losses()
    c.run(None, abi.zero_distill_forward)
    return Losses(*out)


def distill_backward(hidden, weight, teacher_ids, teacher_logits, lse, lse_tau, *,
                     temperature: float = 1.0, labels=None, alpha: float = 1.0,
                     reduction: str = "mean", ignore_index: int = -100, dloss=None,
                     grad_scale: float = 1.0, dhidden=None, dweight=None,
                     accumulate: bool = False, stream=None) -> Losses:
    """The gradients, given ``lse`` and ``lse_tau`` of distill_forward on the
    same inputs; ``dloss`` as in xent_backward."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream,
              (teacher_ids, teacher_logits, temperature, alpha))
    c.statistics(lse, lse_tau)
    dh, dw = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(None, abi.zero_distill_backward)
    return Losses(None, None, lse, lse_tau, dh, dw)


def distill_step(hidden, weight, teacher_ids, teacher_logits, *, temperature: float = 1.0,
                 labels=None, alpha: float = 1.0, reduction: str = "mean",
                 ignore_index: int = -100, dloss=None, grad_scale: float = 1.0, dhidden=None,
                 dweight=None, accumulate: bool = False, stream=None) -> Losses:
    """distill_forward and distill_backward in one call."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream,
              (teacher_ids, teacher_logits, temperature, alpha))
    out = c.losses()
    grads = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(None, abi.zero_distill_step)
    return Losses(*out, *grads)


def policy_forward(hidden, weight, labels, old_logps, advantages, *, ref_logps=None, clip=0.2,
                   kl_weight: float = 0.0, reduction: str = "mean", ignore_index: int = -100,
                   stream=None) -> LogpLosses:
    """The clipped policy loss of every labelled row: ``old_logps`` float32, the
    labels' log-probabilities when they were sampled, ``advantages`` float32,
    ``clip`` how far the ratio may move either way, or a pair for down and up,
    ``ref_logps`` float32, a reference's log-probabilities, from which
    ``kl_weight`` holds the policy. The mean is over the labelled rows."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    c.policy(old_logps, advantages, ref_logps, clip, kl_weight)
    out = c.logp_losses()
    c.run(abi.zero_policy_forward, None)
    return LogpLosses(*out)


def policy_backward(hidden, weight, labels, lse, row_logps, slopes, *, reduction: str = "mean",
                    ignore_index: int = -100, dloss=None, grad_scale: float = 1.0, dhidden=None, dweight=None,
                    accumulate: bool = False, stream=None) -> LogpLosses:
    """The gradients, given ``lse``, ``row_logps`` and ``slopes`` of policy_forward
    on the same inputs; ``dloss`` as in xent_backward."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    c.policy(forward=False)
    c.slopes(lse, row_logps, slopes)
    dh, dw = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(abi.zero_policy_backward, None)
    return LogpLosses(None, None, None, slopes, lse, row_logps, None, dh, dw)


def policy_step(hidden, weight, labels, old_logps, advantages, *, ref_logps=None, clip=0.2, kl_weight: float = 0.0,
                reduction: str = "mean", ignore_index: int = -100, dloss=None, grad_scale: float = 1.0, dhidden=None,
                dweight=None, accumulate: bool = False, stream=None) -> LogpLosses:
    """policy_forward and policy_backward in one call."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    c.policy(old_logps, advantages, ref_logps, clip, kl_weight)
    out = c.logp_losses()
    grads = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(abi.zero_policy_step, None)
    return LogpLosses(*out, *grads)


def preference_forward(hidden, weight, labels, offsets=None, *, ref_logps=None, kind: str = "sigmoid",
                       beta: float = 0.1, smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                       nll_weight: float = 0.0, reduction: str = "mean", ignore_index: int = -100,
                       stream=None) -> LogpLosses:
    """The loss of pairs of sequences, the preferred ones first, then the rejected
    in the same order: ``offsets`` int64 [2 * pairs + 1], the sequences' first
    rows and the end of the last, or None where ``hidden`` is [2 * pairs, length,
    D]. ``ref_logps`` float32 [2 * pairs]: a reference's sums of
    log-probabilities (a forward call's ``logps``), with ``average`` their means
    (``logps / counts``). ``kind`` "sigmoid" or "squared"; with beta = 1,
    average, and the margin 1 / (2 tau) the squared loss pulls the log-ratio of a
    pair toward that margin. The mean is over the pairs that have labelled rows."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    c.preference(offsets, ref_logps=ref_logps, kind=kind, beta=beta, smoothing=smoothing, margin=margin,
                 average=average, nll_weight=nll_weight)
    out = c.logp_losses()
    c.run(abi.zero_preference_forward, None)
    return LogpLosses(*out)


def preference_backward(hidden, weight, labels, lse, row_logps, slopes, offsets=None, *, reduction: str = "mean",
                        ignore_index: int = -100, dloss=None, grad_scale: float = 1.0, dhidden=None, dweight=None,
                        accumulate: bool = False, stream=None) -> LogpLosses:
    """The gradients, given ``lse``, ``row_logps`` and ``slopes`` of
    preference_forward on the same inputs. ``dloss`` (float32): the gradient of
    the total with respect to ``loss`` [pairs] (reduction "none") or to
    ``reduced``; ones when None."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    c.preference(offsets)
    c.slopes(lse, row_logps, slopes)
    dh, dw = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(abi.zero_preference_backward, None)
    return LogpLosses(None, None, None, slopes, lse, row_logps, None, dh, dw)


def preference_step(hidden, weight, labels, offsets=None, *, ref_logps=None, kind: str = "sigmoid",
                    beta: float = 0.1, smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                    nll_weight: float = 0.0, reduction: str = "mean", ignore_index: int = -100, dloss=None,
                    grad_scale: float = 1.0, dhidden=None, dweight=None, accumulate: bool = False,
                    stream=None) -> LogpLosses:
    """preference_forward and preference_backward in one call."""
    c = _Call(hidden, weight, labels, reduction, ignore_index, stream)
    c.preference(offsets, ref_logps=ref_logps, kind=kind, beta=beta, smoothing=smoothing, margin=margin,
                 average=average, nll_weight=nll_weight)
    out = c.logp_losses()
    grads = c.gradients(dloss, grad_scale, dhidden, dweight, accumulate)
    c.run(abi.zero_preference_step, None)
    return LogpLosses(*out, *grads)


# -------------------------------------------------------------- autograd --

class _Once(torch.autograd.Function):
    """Passes gradients on; to differentiate them again raises. ``inputs`` are what they
    depend on: without that tie autograd would take the gradients for constants, and a
    second derivative would lose their part without a word."""

    @staticmethod
    def forward(ctx, dhidden, dweight, *inputs):
        return dhidden, dweight

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the vocabulary losses have no second derivatives")


def _once(r, *inputs):
    """dhidden and dweight of ``r`` as a backward function returns them."""
    if torch.is_grad_enabled():      # create_graph
        return _Once.apply(r.dhidden, r.dweight, *inputs)
    return r.dhidden, r.dweight


class _Xent(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, labels, reduction, ignore_index):
        r = xent_forward(hidden, weight, labels, reduction=reduction, ignore_index=ignore_index)
        ctx.save_for_backward(hidden, weight, labels, r.lse)
        ctx.options = dict(reduction=reduction, ignore_index=ignore_index)
        return r.loss if reduction == "none" else r.reduced

    @staticmethod
    def backward(ctx, dloss):
        hidden, weight, labels, lse = ctx.saved_tensors
        if not any(ctx.needs_input_grad[:2]):
            return None, None, None, None, None
        with torch.no_grad():
            r = xent_backward(hidden, weight, labels, lse, dloss=dloss.contiguous(),
                              dhidden=None if ctx.needs_input_grad[0] else False,
                              dweight=None if ctx.needs_input_grad[1] else False, **ctx.options)
        return *_once(r, hidden, weight, dloss), None, None, None


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, ids, logits, labels, options):
        r = distill_forward(hidden, weight, ids, logits, labels=labels, **options)
        ctx.save_for_backward(hidden, weight, ids, logits, labels, r.lse, r.lse_tau)
        ctx.options = options
        return r.loss if options["reduction"] == "none" else r.reduced

    @staticmethod
    def backward(ctx, dloss):
        hidden, weight, ids, logits, labels, lse, lse_tau = ctx.saved_tensors
        if not any(ctx.needs_input_grad[:2]):
            return None, None, None, None, None, None
        with torch.no_grad():
            r = distill_backward(hidden, weight, ids, logits, lse, lse_tau, labels=labels,
                                 dloss=dloss.contiguous(),
                                 dhidden=None if ctx.needs_input_grad[0] else False,
                                 dweight=None if ctx.needs_input_grad[1] else False, **ctx.options)
        return *_once(r, hidden, weight, dloss), None, None, None, None


class _Policy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, labels, old_logps, advantages, ref_logps, options, reduction, ignore_index):
        r = policy_forward(hidden, weight, labels, old_logps, advantages, ref_logps=ref_logps,
                           reduction=reduction, ignore_index=ignore_index, **options)
        ctx.save_for_backward(hidden, weight, labels, r.lse, r.row_logps, r.slopes)
        ctx.options = dict(reduction=reduction, ignore_index=ignore_index)
        return r.loss if reduction == "none" else r.reduced

    @staticmethod
    def backward(ctx, dloss):
        hidden, weight, labels, lse, logps, slopes = ctx.saved_tensors
        none = (None,) * 7
        if not any(ctx.needs_input_grad[:2]):
            return None, None, *none
        with torch.no_grad():
            r = policy_backward(hidden, weight, labels, lse, logps, slopes, dloss=dloss.contiguous(),
                                dhidden=None if ctx.needs_input_grad[0] else False,
                                dweight=None if ctx.needs_input_grad[1] else False, **ctx.options)
        return *_once(r, hidden, weight, dloss), *none


class _Preference(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, labels, offsets, ref_logps, options, reduction, ignore_index):
        r = preference_forward(hidden, weight, labels, offsets, ref_logps=ref_logps, reduction=reduction,
                               ignore_index=ignore_index, **options)
        ctx.save_for_backward(hidden, weight, labels, offsets, r.lse, r.row_logps, r.slopes)
        ctx.options = dict(reduction=reduction, ignore_index=ignore_index)
        return r.loss if reduction == "none" else r.reduced

    @staticmethod
    def backward(ctx, dloss):
        hidden, weight, labels, offsets, lse, logps, slopes = ctx.saved_tensors
        none = (None,) * 6
        if not any(ctx.needs_input_grad[:2]):
            return None, None, *none
        with torch.no_grad():
            r = preference_backward(hidden, weight, labels, lse, logps, slopes, offsets, dloss=dloss.contiguous(),
                                    dhidden=None if ctx.needs_input_grad[0] else False,
                                    dweight=None if ctx.needs_input_grad[1] else False, **ctx.options)
        return *_once(r, hidden, weight, dloss), *none


def linear_cross_entropy(hidden, weight, labels, reduction: str = "mean",
                         ignore_index: int = -100):
    """Cross entropy of ``hidden @ weight.T``, differentiable in ``hidden`` and ``weight``."""
    return _Xent.apply(hidden, weight, labels, reduction, ignore_index)


def linear_distillation(hidden, weight, teacher_ids, teacher_logits, temperature: float = 1.0,
                        labels=None, alpha: float = 1.0, reduction: str = "mean",
                        ignore_index: int = -100):
    """The distillation loss, differentiable in ``hidden`` and ``weight`` (the
    teacher's logits are constants)."""
    options = dict(temperature=temperature, alpha=alpha, reduction=reduction,
                   ignore_index=ignore_index)
    return _Distill.apply(hidden, weight, teacher_ids, teacher_logits, labels, options)


def linear_policy(hidden, weight, labels, old_logps, advantages, ref_logps=None, clip=0.2, kl_weight: float = 0.0,
                  reduction: str = "mean", ignore_index: int = -100):
    """The clipped policy loss, differentiable in ``hidden`` and ``weight`` (all else is
    constant)."""
    return _Policy.apply(hidden, weight, labels, old_logps, advantages, ref_logps,
                         dict(clip=clip, kl_weight=kl_weight), reduction, ignore_index)


def linear_preference(hidden, weight, labels, offsets=None, ref_logps=None, kind: str = "sigmoid", beta: float = 0.1,
                      smoothing: float = 0.0, margin: float = 0.0, average: bool = False, nll_weight: float = 0.0,
                      reduction: str = "mean", ignore_index: int = -100):
    """The preference loss, differentiable in ``hidden`` and ``weight`` (all else is
    constant)."""
    options = dict(kind=kind, beta=beta, smoothing=smoothing, margin=margin, average=average, nll_weight=nll_weight)
    return _Preference.apply(hidden, weight, labels, offsets, ref_logps, options, reduction, ignore_index)
