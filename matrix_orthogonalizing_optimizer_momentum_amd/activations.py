"""Between the embedding and the output layer: the root-mean-square norm with its
gradient, activations kept in 8 bits, and the gradient of a weight from them.

Argument marshalling only, as in ``gradients.py``: the work is queued on
``stream`` (default: the current stream of the tensors' device) and never waits
for the device; outputs and scratch memory are torch allocations made for the
call on that stream.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import MUONH_BF16, MUONH_PACK_NORMALIZED, MUONH_PACK_OUTPUT, load
from .gradients import _check, _code, _on, _plain

BLOCK = 32  # values that share one scale


class Packed(NamedTuple):
    """A matrix in 8 bits: ``q[..., j] * scales[..., j // 32]``.

    ``q``: ``torch.float8_e4m3fn`` of the matrix's shape; ``scales``:
    ``torch.float8_e8m0fnu`` (powers of two), one for each 32 values of a row.
    """
    q: torch.Tensor
    scales: torch.Tensor


class Normed(NamedTuple):
    """What ``rms_norm`` computed; ``None`` for what was not asked for."""
    y: Optional[torch.Tensor]
    h: Optional[torch.Tensor]
    rstd: torch.Tensor
    packed: Optional[Packed]


def _rows(t):
    """(rows, width) of a tensor whose last axis is a row."""
    if t.dim() < 1 or t.shape[-1] == 0:
        raise ValueError("the last axis must hold at least one value")
    return t.numel() // t.shape[-1], t.shape[-1]


def _new_packed(like):
    width = like.shape[-1]
    return Packed(torch.empty(like.shape, dtype=torch.float8_e4m3fn, device=like.device),
                  torch.empty((*like.shape[:-1], -(-width // BLOCK)), dtype=torch.float8_e8m0fnu, device=like.device))


def _packed(p, what, dev=None):
    """(q, scales) of a Packed or a pair like it, checked."""
    q, scales = p
    if q.dtype != torch.float8_e4m3fn or scales.dtype != torch.float8_e8m0fnu:
        raise TypeError(f"{what} must hold torch.float8_e4m3fn values and torch.float8_e8m0fnu scales")
    dev = _plain(q, what, dev)
    _plain(scales, f"{what}'s scales", dev)
    _rows(q)
    if tuple(scales.shape) != (*q.shape[:-1], -(-q.shape[-1] // BLOCK)):
        raise ValueError(f"{what} must have one scale for each {BLOCK} values of a row")
    return q, scales


def _like(t, ref, what, dev, dtype=None):
    """Checks a tensor against another's shape."""
    _plain(t, what, dev)
    if t.shape != ref.shape:
        raise ValueError(f"{what} must have the shape of the other tensors")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")


def _gain(gain, width, dev):
    if gain is None:
        return None
    _plain(gain, "gain", dev)
    if gain.dtype != torch.float32:
        raise TypeError("gain must be torch.float32")
    if tuple(gain.shape) != (width,):
        raise ValueError("gain must have one value for each of the last axis")
    return gain.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


_PACK = {"normalized": MUONH_PACK_NORMALIZED, "output": MUONH_PACK_OUTPUT}


def rms_norm(x, gain=None, residual=None, eps=1e-6, pack=None, output=True, out=None, out_dtype=None, h=None, stream=None):
    """Root-mean-square norm over the last axis, with the residual's addition.

    ``h = x + residual`` (rounded to ``residual``'s dtype; ``h = x`` without
    one), ``rstd = (mean(h^2) + eps)^-1/2``, ``y = gain * rstd * h``.  ``x`` and
    ``residual``: float32 or bfloat16, each its own; ``gain``: float32, or ``None``.

    Returns ``Normed(y, h, rstd, packed)``: ``y`` in ``out_dtype`` (default:
    x's; ``None`` with ``output=False``), ``h`` (``None`` without a residual; a
    given ``h`` may be ``residual`` itself), ``rstd`` in float32, and with
    ``pack`` a matrix in 8 bits: "normalized" for ``rstd * h``, which
    ``rms_norm_grad`` and, with the gain, ``weight_grad`` take in place of the
    activations, or "output" for ``y``.
    """
    if pack is not None and pack not in _PACK:
        raise ValueError(f"pack must be None, 'normalized' or 'output', got {pack!r}")
    n, width = _rows(x)
    dev = _plain(x, "x")
    code = _code(x, "x")
    if residual is not None:
        _like(residual, x, "residual", dev)
        _code(residual, "residual")
    if h is not None:
        if residual is None:
            raise ValueError("h needs a residual")
        _like(h, x, "h", dev, residual.dtype)
    if out is not None:
        if not output:
            raise ValueError("out is given, but output is False")
        _like(out, x, "out", dev, out_dtype)
    gain_ptr = _gain(gain, width, dev)
    lib = load()
    with _on(dev, stream) as raw:
        if out is None and output:
            out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
        if h is None and residual is not None:
            h = torch.empty_like(residual)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        packed = None if pack is None else _new_packed(x)
        rc = lib.muonh_rms_norm(x.data_ptr(), code, _ptr(residual) if n else None,
                                MUONH_BF16 if h is None else _code(h, "h"), gain_ptr, eps, n, width,
                                _ptr(h) if n else None, _ptr(out), MUONH_BF16 if out is None else _code(out, "out"),
                                rstd.data_ptr(), None if packed is None or not n else packed.q.data_ptr(),
                                None if packed is None or not n else packed.scales.data_ptr(),
                                _PACK[pack] if pack else MUONH_PACK_NORMALIZED, raw)
    _check(rc, "muonh_rms_norm")
    return Normed(out, h, rstd, packed)


def rms_norm_grad(dy, x, rstd, gain=None, dres=None, out=None, out_dtype=None, dgain=None, accumulate=False,
                  gain_grad=None, stream=None):
    """Gradients of ``rms_norm``'s input and gain.

    ``dy``: float32 or bfloat16; ``x``: the norm's input (``h``, or ``x`` without a
    residual) in the dtype of the result, or what ``pack="normalized"`` kept;
    ``rstd``: as ``rms_norm`` returned it; ``dres``: a gradient that reaches ``h``
    on the residual's path, of the result's dtype, added to the result.

    Returns ``(dx, dgain)``: the gradient of ``h``, and so of ``x`` and of the
    residual, in ``out_dtype`` (default: that of ``out``, ``x`` as a tensor,
    ``dres`` or ``dy``, the first there is; ``out`` may be ``dres``), and the gain's
    in float32, allocated unless ``dgain`` is given (``accumulate`` adds to it), or
    ``None`` without a gain (``gain_grad`` asks for it or not all the same).
    """
    n, width = _rows(dy)
    dev = _plain(dy, "dy")
    code = _code(dy, "dy")
    tensor = isinstance(x, torch.Tensor)
    if out_dtype is None:
        out_dtype = next((t for t in (out, x if tensor else None, dres) if t is not None), dy).dtype
    if tensor:
        _like(x, dy, "x", dev, out_dtype)
        q = scales = None
    else:
        q, scales = _packed(x, "x", dev)
        if q.shape != dy.shape:
            raise ValueError("x must have the shape of dy")
    _plain(rstd, "rstd", dev)
    if rstd.dtype != torch.float32:
        raise TypeError("rstd must be torch.float32")
    if rstd.shape != dy.shape[:-1]:
        raise ValueError("rstd must have one value for each row of dy")
    if dres is not None:
        _like(dres, dy, "dres", dev, out_dtype)
    if out is not None:
        _like(out, dy, "out", dev, out_dtype)
    gain_ptr = _gain(gain, width, dev)
    if gain_grad is None:
        gain_grad = gain is not None or dgain is not None
    if dgain is not None:
        if not gain_grad:
            raise ValueError("dgain is given, but gain_grad is False")
        _gain(dgain, width, dev)
    elif accumulate:
        raise ValueError("accumulate needs dgain")
    lib = load()
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty(dy.shape, dtype=out_dtype, device=dy.device)
        if gain_grad and dgain is None:
            dgain = torch.empty(width, dtype=torch.float32, device=dy.device)
        ws_bytes = lib.muonh_rms_norm_grad_workspace(n, width) if gain_grad else 0
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dy.device) if ws_bytes else None
        rc = lib.muonh_rms_norm_grad(dy.data_ptr(), code, x.data_ptr() if tensor and n else None,
                                     _ptr(q) if n else None, _ptr(scales) if n else None, rstd.data_ptr(), gain_ptr,
                                     _ptr(dres), _code(out, "out"), n, width, out.data_ptr(), _ptr(dgain),
                                     1 if accumulate else 0, _ptr(ws), ws_bytes, raw)
    _check(rc, "muonh_rms_norm_grad")
    return out, dgain


def mx_pack(x, stream=None):
    """``x`` (float32 or bfloat16) in 8 bits: ``Packed(q, scales)``.

    Blocks of 32 along the last axis, each with the least power of two that no
    finite value of it exceeds 448 times (at least 2^-117); values are rounded to
    e4m3, to nearest even, at most 2^-4 of themselves off unless they are below
    2^-6 of the scale.  Infinities and NaN become NaN and reach no other value.
    """
    n, width = _rows(x)
    dev = _plain(x, "x")
    code = _code(x, "x")
    lib = load()
    with _on(dev, stream) as raw:
        packed = _new_packed(x)
        rc = lib.muonh_mx_pack(x.data_ptr(), code, n, width, packed.q.data_ptr(), packed.scales.data_ptr(), raw)
    _check(rc, "muonh_mx_pack")
    return packed


def mx_unpack(packed, out=None, out_dtype=None, stream=None):
    """What a matrix in 8 bits stands for, in ``out_dtype`` (float32 or bfloat16, the
    default, exact for what ``mx_pack`` and ``rms_norm`` write).  Returns ``out``."""
    q, scales = _packed(packed, "packed")
    n, width = _rows(q)
    dev = q.get_device()
    if out is not None:
        _like(out, q, "out", dev, out_dtype)
    lib = load()
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype or torch.bfloat16, device=q.device)
        rc = lib.muonh_mx_unpack(q.data_ptr(), scales.data_ptr(), n, width, out.data_ptr(), _code(out, "out"), raw)
    _check(rc, "muonh_mx_unpack")
    return out


def weight_grad(dz, packed, gain=None, scale=1.0, out=None, out_dtype=None, accumulate=False, stream=None):
    """Gradient of a weight of rows x width behind ``z = (gain * x) @ W.T``, from ``x``
    in 8 bits: ``scale * gain * (dz.T @ x)`` over all leading axes.

    ``dz``: ``(..., rows)``, bfloat16; ``packed``: ``(..., width)`` from ``mx_pack``
    or ``rms_norm`` (with ``pack="normalized"`` give the norm's ``gain``); ``out``:
    rows x width in ``out_dtype`` (float32 or bfloat16, the default), allocated unless
    given; ``accumulate`` adds to it.  Sums are float32.  Returns ``out``.
    """
    n, rows = _rows(dz)
    dev = _plain(dz, "dz")
    if dz.dtype != torch.bfloat16:
        raise TypeError("dz must be torch.bfloat16")
    q, scales = _packed(packed, "packed", dev)
    if q.shape[:-1] != dz.shape[:-1]:
        raise ValueError("dz and packed must have the same leading axes")
    width = q.shape[-1]
    gain_ptr = _gain(gain, width, dev)
    if out is not None:
        _plain(out, "out", dev)
        if tuple(out.shape) != (rows, width) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must be rows x width, of out_dtype")
    elif accumulate:
        raise ValueError("accumulate needs out")
    lib = load()
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty((rows, width), dtype=out_dtype or torch.bfloat16, device=dz.device)
        code = _code(out, "out")
        ws_bytes = lib.muonh_weight_grad_workspace(dz.data_ptr(), n, rows, width)
        ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dz.device)
        rc = lib.muonh_weight_grad(dz.data_ptr(), q.data_ptr(), scales.data_ptr(), gain_ptr, scale, n, rows, width,
                                   out.data_ptr(), code, 1 if accumulate else 0, ws.data_ptr(), ws_bytes, raw)
    _check(rc, "muonh_weight_grad")
    return out
