"""The embedding: token ids to rows of a table, and the table's gradient.

``embedding_forward`` looks the rows up and scales them, ``embedding_backward``
adds up the gradient of the tokens of equal id (the definitions stand in
``include/zero_gb300.h`` at ``zero_embedding_forward``). In a model whose
embedding and head are one matrix, the head's gradient is written by the
vocabulary losses (``losses``) into a rank's flat gradient buffer, and the
embedding's is then added to the rows that have a token::

    losses.xent_step(hidden, wte, labels, dweight=dwte)
    embedding.embedding_backward(tokens, dx, dweight=dwte, accumulate=True)

``ids`` is an int64 CUDA tensor of any shape; of a view, as ``tokens[:, :-1]``, the
call makes a copy (one that is expanded is taken by ``embedding`` alone). ``weight`` is a [V, D]
CUDA tensor, float32 or bfloat16, with adjacent elements in a row and any row
stride; what belongs to the tokens has ids' shape and a last dimension D.

``embedding`` is the same as a differentiable function for torch.autograd, in
any order.

Work is queued on ``stream``: a ``torch.cuda.Stream``, a raw handle, or None for
the current stream. The workspace and a result that is not given are taken from
PyTorch's allocator as that stream's; the allocator is told that ``stream`` uses
the inputs and that the current stream uses the result. To order the two
streams' work is left to the caller.
"""

from __future__ import annotations

import torch

from . import abi
from .losses import _PRECISION, _matrix, _named


def _tokens(ids, device, stream):
    """The ids side by side: themselves, or a copy made on ``stream``."""
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda or ids.dtype is not torch.int64:
        raise TypeError("ids must be a torch.int64 CUDA tensor")
    if ids.device != device:
        raise ValueError(f"ids is on {ids.device}, expected {device}")
    if ids.is_contiguous():
        return ids
    if any(step == 0 and n > 1 for step, n in zip(ids.stride(), ids.shape)):
        raise ValueError("ids must not be expanded")
    if stream is not None:
        ids.record_stream(stream)
    with torch.cuda.stream(stream):     # None: the current one
        return ids.contiguous()


def _rows(t, what: str, ids, D=None, dtype=None, device=None):
    """``t``, of ids' shape and a last dimension, as a matrix of a row for each id."""
    if isinstance(t, torch.Tensor) and t.shape[:-1] != ids.shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected ids' {tuple(ids.shape)} and a last dimension")
    if isinstance(t, torch.Tensor) and t.dim() == 1:      # a single id
        t = t.unsqueeze(0)
    return _matrix(t, what, dtype, ids.numel(), D, device)


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _run(p, call, device, stream, used, made):
    """Queues ``call``; ``used``: the caller's tensors, ``made``: its result."""
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _run(p, call, device, stream, used, made)
    if call is abi.zero_embedding_backward:
        size = abi.zero_embedding_workspace_bytes(p)
        space = _empty(size, torch.uint8, device, stream)
        p.workspace, p.workspace_bytes = space.data_ptr() if size else None, size
    if stream is not None:
        for t in used:
            t.record_stream(stream)
        if made is not None:
            made.record_stream(torch.cuda.current_stream(device))
    # the current stream's handle, without the object around it
    call(p, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream)


def embedding_forward(ids, weight, *, scale: float = 1.0, out=None, stream=None):
    """``scale * weight[ids]``, zeros for an id outside the table; written to ``out`` where given."""
    w, stride = _matrix(weight, "weight")
    device, dtype = w.device, w.dtype
    V, D = w.shape
    stream = _named(stream, device)
    ids = _tokens(ids, device, stream)
    p = abi.Embedding(ids.numel(), V, D, _PRECISION[dtype], 0, ids.data_ptr(), -1, scale, w.data_ptr(), stride)
    made = None
    if out is None:
        out = made = _empty((*ids.shape, D), dtype, device, stream)
        p.out, p.out_stride = out.data_ptr(), D
    else:
        m, p.out_stride = _rows(out, "out", ids, D, dtype, device)
        p.out = m.data_ptr()
    _run(p, abi.zero_embedding_forward, device, stream, (ids, w) if made is not None else (ids, w, out), made)
    return out


def embedding_backward(ids, dout, vocabulary: int | None = None, *, scale: float = 1.0, padding_id: int = -1,
                       dweight=None, accumulate: bool = False, stream=None):
    """The gradient of the table, given that of embedding_forward's result: a new
    [vocabulary, D] tensor, or ``dweight``, overwritten or with ``accumulate`` added
    to. Tokens of ``padding_id`` or outside the table add nothing."""
    if isinstance(ids, torch.Tensor) and isinstance(dout, torch.Tensor) and dout.dim() > 0:
        m, stride = _rows(dout, "dout", ids)
    else:
        raise TypeError("ids and dout must be CUDA tensors")
    device, dtype, D = m.device, m.dtype, m.shape[1]
    stream = _named(stream, device)
    ids = _tokens(ids, device, stream)
    made = None
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate adds to a dweight that is given")
        if vocabulary is None:
            raise ValueError("the vocabulary's size or a dweight must be given")
        dweight = made = _empty((vocabulary, D), dtype, device, stream)
    w, ws = _matrix(dweight, "dweight", dtype, vocabulary, D, device)
    p = abi.Embedding(ids.numel(), w.shape[0], D, _PRECISION[dtype], 1 if accumulate else 0, ids.data_ptr(), padding_id, scale,
                      None, 0, None, 0, m.data_ptr(), stride, w.data_ptr(), ws)
    _run(p, abi.zero_embedding_backward, device, stream, (ids, m) if made is not None else (ids, m, w), made)
    return dweight


# -------------------------------------------------------------- autograd --

class _Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding_id):
        if isinstance(ids, torch.Tensor):
            ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.options = weight.shape[0], scale, padding_id
        return embedding_forward(ids, weight, scale=scale)

    @staticmethod
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        if not ctx.needs_input_grad[0]:
            return None, None, None, None
        return _Gradient.apply(dout, ids, *ctx.options), None, None, None


class _Gradient(torch.autograd.Function):
    """The gradient, which is linear in dout: its own is the lookup."""

    @staticmethod
    def forward(ctx, dout, ids, vocabulary, scale, padding_id):
        ctx.save_for_backward(ids)
        ctx.options = scale, padding_id
        return embedding_backward(ids, dout.contiguous(), vocabulary, scale=scale, padding_id=padding_id)

    @staticmethod
    def backward(ctx, dweight):
        ids, = ctx.saved_tensors
        scale, padding_id = ctx.options
        if not ctx.needs_input_grad[0]:
            return None, None, None, None, None
        if padding_id >= 0:
            ids = torch.where(ids == padding_id, -1, ids)
        return _Lookup.apply(dweight.contiguous(), ids, scale, -1), None, None, None, None


def embedding(ids, weight, scale: float = 1.0, padding_id: int = -1):
    """``scale * weight[ids]``, differentiable in ``weight``."""
    return _Lookup.apply(weight, ids, scale, padding_id)
