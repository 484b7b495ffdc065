"""The gradients an optimizer step consumes: their global norm and clipping, the
embedding and its gradient, the output layer's loss with its gradients.

Argument marshalling only, like the rest of the binding: the work is queued on
``stream`` (default: the current stream of the tensors' device) and never waits
for the device.  Outputs and scratch memory are torch allocations made for the
call on that stream, so calls on different streams share nothing and every
call can be captured into a graph.
"""
from __future__ import annotations

import contextlib

import torch

from . import (MUONH_BF16, MUONH_ENOMEM, MUONH_F32, MUONH_REDUCE_MEAN, MUONH_REDUCE_SUM, MuonhError,
               MuonhUnavailable, load)

try:
    from . import _tensors
except ImportError:  # not built
    _tensors = None

_CODE = {torch.float32: MUONH_F32, torch.bfloat16: MUONH_BF16}


@contextlib.contextmanager
def _switched(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream(dev).cuda_stream
        else:
            if stream.device.index != dev:
                raise ValueError("stream belongs to another device than the tensors")
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _on(dev, stream):
    """Context in which allocations and launches go to ``stream`` on device
    ``dev``; gives the raw stream."""
    if stream is None and dev == torch.cuda.current_device():
        return contextlib.nullcontext(torch._C._cuda_getCurrentRawStream(dev))
    return _switched(dev, stream)


def _check(rc, where):
    if rc:
        raise MuonhError(rc, where)


def _held(ts):
    """A list or tuple of the tensors: any other sequence may make them on access, and they
    have to last until the work that reads them is queued."""
    return ts if isinstance(ts, (list, tuple)) else list(ts)


def _table(ts, what):
    """(pointers, sizes, dtype codes, device) of a list of gradients, checked."""
    if _tensors is None:
        raise MuonhUnavailable("_tensors.so is not built; run `python -m matrix_orthogonalizing_optimizer_momentum_amd.build`")
    return _tensors.table(ts, what)


def grad_norm(grads, max_norm=None, stream=None):
    """2-norm of all gradients together.

    ``grads``: float32 / bfloat16 tensors of any shapes (contiguous, one
    device).  Returns ``(total, coef, norms)``, float32 on the device: the
    global norm, the clipping coefficient ``min(1, max_norm / (total + 1e-6))``
    (``None`` without ``max_norm``) and the norm of every tensor.  Pass ``coef``
    to ``muonh_step`` / ``adamh_step`` as ``grad_scale`` to step on the clipped
    gradients without another pass over them.
    """
    grads = _held(grads)
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients")
    ptrs, sizes, codes, dev = _table(grads, "grads")
    lib = load()
    with _on(dev, stream) as raw:
        ws_bytes = lib.muonh_grad_norm_workspace(n)
        where = grads[0].device
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=where)
        norms = torch.empty(n, dtype=torch.float32, device=where)
        total = torch.empty((), dtype=torch.float32, device=where)
        coef = None if max_norm is None else torch.empty((), dtype=torch.float32, device=where)
        rc = lib.muonh_grad_norm(ptrs, sizes, codes, n, 0.0 if coef is None else max_norm,
                                 total.data_ptr(), None if coef is None else coef.data_ptr(), norms.data_ptr(),
                                 ws.data_ptr(), ws_bytes, raw)
    _check(rc, "muonh_grad_norm")
    return total, coef, norms


def clip_grads(grads, max_norm, outputs=None, stream=None):
    """Scale the gradients so that their global norm is at most ``max_norm``.

    ``outputs[i] = coef * grads[i]`` with ``grad_norm``'s coefficient;
    ``outputs=None`` scales ``grads`` in place.  Returns ``(total, coef)``.
    """
    grads = _held(grads)
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients")
    ptrs, sizes, codes, dev = _table(grads, "grads")
    outs = ptrs
    if outputs is not None:
        outputs = _held(outputs)
        if len(outputs) != n:
            raise ValueError("outputs must have one tensor per gradient")
        outs, osizes, ocodes, odev = _table(outputs, "outputs")
        if osizes != sizes or ocodes != codes or odev != dev:
            raise ValueError("outputs must match grads in size, dtype and device")
    lib = load()
    with _on(dev, stream) as raw:
        ws_bytes = lib.muonh_grad_norm_workspace(n)
        where = grads[0].device
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=where)
        total = torch.empty((), dtype=torch.float32, device=where)
        coef = torch.empty((), dtype=torch.float32, device=where)
        rc = lib.muonh_clip_grads(ptrs, outs, sizes, codes, n, max_norm,
                                  total.data_ptr(), coef.data_ptr(), ws.data_ptr(), ws_bytes, raw)
    _check(rc, "muonh_clip_grads")
    return total, coef


def _plain(t, what, dev=None):
    """Checks one tensor: on the GPU (device ``dev`` if given), contiguous; returns its device."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{what} must be on the GPU")
    if dev is not None and d != dev:
        raise ValueError(f"{what} is on another device")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return d


def _code(t, what):
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")
    return code


def _id_bits(t, what):
    if t.dtype == torch.int64:
        return 64
    if t.dtype == torch.int32:
        return 32
    raise TypeError(f"{what}: unsupported dtype {t.dtype}: use torch.int64 or torch.int32")


def embedding(table, ids, scale=1.0, out=None, out_dtype=None, stream=None):
    """``out[i] = scale * table[ids[i]]``, zeros for an id outside the table.

    ``table``: rows x width, float32 or bfloat16; ``ids``: int64 / int32 of any
    shape; ``out``: ``ids.shape + (width,)`` in ``out_dtype`` (default: the
    table's), allocated unless given.  Returns ``out``.
    """
    if table.dim() != 2:
        raise ValueError("table must be a matrix (2-D)")
    dev = _plain(table, "table")
    _plain(ids, "ids", dev)
    bits, code = _id_bits(ids, "ids"), _code(table, "table")
    shape = (*ids.shape, table.shape[1])
    lib = load()
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty(shape, dtype=out_dtype or table.dtype, device=table.device)
        else:
            _plain(out, "out", dev)
            if tuple(out.shape) != shape or (out_dtype is not None and out.dtype != out_dtype):
                raise ValueError("out must have the shape of ids and the table's width, and out_dtype")
        rc = lib.muonh_embedding(table.data_ptr(), code, table.shape[0], table.shape[1], ids.data_ptr(), bits,
                                 ids.numel(), scale, out.data_ptr(), _code(out, "out"), raw)
    _check(rc, "muonh_embedding")
    return out


def embedding_grad(ids, dout, rows=None, scale=1.0, out=None, out_dtype=None, accumulate=False, stream=None):
    """Gradient of ``embedding``'s table: ``out[v] = scale * sum of dout[i] over ids[i] == v``.

    ``dout``: ``ids.shape + (width,)``, float32 or bfloat16; ``out``: ``rows`` x
    width in ``out_dtype`` (default: dout's), allocated unless given.  Rows
    without a token become zero; with ``accumulate`` the sums are added to
    ``out`` instead.  Tokens with ids outside the table are left out.  Returns
    ``out``.
    """
    dev = _plain(dout, "dout")
    _plain(ids, "ids", dev)
    bits, code = _id_bits(ids, "ids"), _code(dout, "dout")
    if tuple(dout.shape[:-1]) != tuple(ids.shape) or dout.dim() != ids.dim() + 1:
        raise ValueError("dout must have the shape of ids and one more axis, the table's width")
    if out is None:
        if rows is None:
            raise ValueError("embedding_grad needs rows or out")
        if accumulate:
            raise ValueError("accumulate needs out")
    else:
        _plain(out, "out", dev)
        rows = out.shape[0] if rows is None else rows
        if tuple(out.shape) != (rows, dout.shape[-1]) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must be rows x width, of out_dtype")
    width = dout.shape[-1]
    lib = load()
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty((rows, width), dtype=out_dtype or dout.dtype, device=dout.device)
        ws_bytes = lib.muonh_embedding_grad_workspace(ids.numel(), rows, width)
        ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dout.device)
        rc = lib.muonh_embedding_grad(ids.data_ptr(), bits, ids.numel(), dout.data_ptr(), code, scale,
                                      1 if accumulate else 0, out.data_ptr(), _code(out, "out"), rows, width,
                                      ws.data_ptr(), ws_bytes, raw)
    _check(rc, "muonh_embedding_grad")
    return out


_REDUCTION = {"mean": MUONH_REDUCE_MEAN, "sum": MUONH_REDUCE_SUM}


def cross_entropy(x, w, targets, reduction="mean", grad=True, grad_scale=1.0, ignore_index=-100, dx=None, dw=None,
                  dw_dtype=None, accumulate=False, workspace_limit=0, stream=None):
    """Softmax cross entropy of ``x @ w.T`` with its gradients, without the logits.

    ``x``: ``targets.shape + (width,)``, bfloat16; ``w``: rows x width, bfloat16;
    ``targets``: int64 / int32.  Tokens whose target is ``ignore_index`` or
    outside ``[0, rows)`` are not counted: they have no loss and no gradient.
    ``reduction``: "mean" over the counted tokens, or "sum".

    Returns ``(loss, token_loss, dx, dw)``: the loss and the loss of every token
    in float32, and the gradients times ``grad_scale`` (``None`` with
    ``grad=False``).  ``grad`` may also be "x" or "w" for one of the two.
    ``dx`` (bfloat16) and ``dw`` (bfloat16 or float32, ``dw_dtype``) are
    allocated unless given; ``accumulate`` adds to the given ``dw``.  Both are
    products of the softmax rounded to bfloat16 (2^-8 of each weight), summed in
    float32: a float32 ``dw`` saves the rounding of its sums, not that one.
    ``workspace_limit`` (bytes) bounds the scratch memory: the vocabulary is
    taken in pieces that fit it.
    """
    if reduction not in _REDUCTION:
        raise ValueError(f"reduction must be 'mean' or 'sum', got {reduction!r}")
    if grad not in (True, False, "x", "w"):
        raise ValueError("grad must be True, False, 'x' or 'w'")
    if w.dim() != 2:
        raise ValueError("w must be a matrix (2-D)")
    dev = _plain(x, "x")
    _plain(w, "w", dev)
    _plain(targets, "targets", dev)
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("x and w must be torch.bfloat16")
    bits = _id_bits(targets, "targets")
    rows, width = w.shape
    if tuple(x.shape) != (*targets.shape, width):
        raise ValueError("x must have the shape of targets and w's width")
    want_x, want_w = grad in (True, "x"), grad in (True, "w")
    if (dx is not None and not want_x) or (dw is not None and not want_w):
        raise ValueError("an output is given for a gradient that is not asked for")
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    if dx is not None:
        _plain(dx, "dx", dev)
        if dx.shape != x.shape or dx.dtype != torch.bfloat16:
            raise ValueError("dx must match x in shape and dtype")
    if dw is not None:
        _plain(dw, "dw", dev)
        if dw.shape != w.shape or (dw_dtype is not None and dw.dtype != dw_dtype):
            raise ValueError("dw must match w in shape, and dw_dtype")
    n = targets.numel()
    lib = load()
    with _on(dev, stream) as raw:
        if want_x and dx is None:
            dx = torch.empty_like(x)
        if want_w and dw is None:
            dw = torch.empty_like(w, dtype=dw_dtype or torch.bfloat16)
        code = MUONH_BF16 if dw is None else _code(dw, "dw")
        grads = (1 if want_x else 0) + (2 if want_w else 0)
        ws_bytes = lib.muonh_cross_entropy_workspace(w.data_ptr(), n, rows, width, grads, workspace_limit)
        if ws_bytes == 0 and workspace_limit and lib.muonh_cross_entropy_workspace(w.data_ptr(), n, rows, width, grads, 0):
            raise MuonhError(MUONH_ENOMEM, "muonh_cross_entropy")
        ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=x.device)
        loss = torch.empty((), dtype=torch.float32, device=x.device)
        token_loss = torch.empty(targets.shape, dtype=torch.float32, device=x.device)
        rc = lib.muonh_cross_entropy(x.data_ptr(), w.data_ptr(), targets.data_ptr(), bits, n, rows, width, ignore_index,
                                     _REDUCTION[reduction], grad_scale, loss.data_ptr(),
                                     token_loss.data_ptr() if n else None, dx.data_ptr() if want_x else None,
                                     dw.data_ptr() if want_w else None, code, 1 if accumulate else 0, ws.data_ptr(),
                                     ws_bytes, raw)
    _check(rc, "muonh_cross_entropy")
    return loss, token_loss, dx, dw
