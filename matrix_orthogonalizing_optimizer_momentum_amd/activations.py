"""Between the embedding and the output layer: the root-mean-square norm with its
gradient, activations kept in 8 bits, and the gradient of a weight from them.

Arguments are checked and outputs allocated by ``_tensors.so`` (a call of one token
would wait for Python otherwise), the rest is the library's.  As in
``gradients.py`` the work is queued on ``stream`` (default: the current stream of
the tensors' device) and never waits for the device; outputs and scratch memory
are torch allocations made for the call on that stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import MUONH_PACK_NORMALIZED, MUONH_PACK_OUTPUT, MuonhError, MuonhUnavailable, load
from .gradients import _switched

try:
    from . import _tensors
except ImportError:  # not built
    _tensors = None


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


_ENTRIES = ("muonh_rms_norm", "muonh_rms_norm_grad_workspace", "muonh_rms_norm_grad", "muonh_mx_pack", "muonh_mx_unpack",
            "muonh_weight_grad_workspace", "muonh_weight_grad")
_bound = False


def _bind():
    global _bound
    lib = load()
    if _tensors is None:
        raise MuonhUnavailable("_tensors.so is not built; run `python -m matrix_orthogonalizing_optimizer_momentum_amd.build`")
    _tensors.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _ENTRIES))
    _bound = True


def _call(name, first, stream, *args):
    """The extension's function `name` on the device of the tensor `first`."""
    if not _bound:
        _bind()
    fn = getattr(_tensors, name)
    dev = first.get_device() if isinstance(first, torch.Tensor) else -1
    if dev < 0:
        r = fn(0, *args)  # which refuses it
    elif stream is None and dev == torch._C._cuda_getDevice():
        r = fn(torch._C._cuda_getCurrentRawStream(dev), *args)
    else:
        with _switched(dev, stream) as raw:
            r = fn(raw, *args)
    if type(r) is int:
        raise MuonhError(r, "muonh_" + name)
    return r


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
    y, h, rstd, q, scales = _call("rms_norm", x, stream, x, gain, residual, eps, -1 if pack is None else _PACK[pack], output, out,
                                  out_dtype, h)
    return Normed(y, h, rstd, None if q is None else Packed(q, scales))


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
    return _call("rms_norm_grad", dy, stream, dy, x, rstd, gain, dres, out, out_dtype, dgain, accumulate, gain_grad)


def mx_pack(x, stream=None):
    """``x`` (float32 or bfloat16) in 8 bits: ``Packed(q, scales)``.

    Blocks of 32 along the last axis, each with the least power of two that no
    finite value of it exceeds 448 times (at least 2^-117); values are rounded to
    e4m3, to nearest even, at most 2^-4 of themselves off unless they are below
    2^-6 of the scale.  Infinities and NaN become NaN and reach no other value.
    """
    return Packed(*_call("mx_pack", x, stream, x))


def mx_unpack(packed, out=None, out_dtype=None, stream=None):
    """What a matrix in 8 bits stands for, in ``out_dtype`` (float32 or bfloat16, the
    default, exact for what ``mx_pack`` and ``rms_norm`` write).  Returns ``out``."""
    return _call("mx_unpack", packed[0], stream, packed, out, out_dtype)


def weight_grad(dz, packed, gain=None, scale=1.0, out=None, out_dtype=None, accumulate=False, stream=None):
    """Gradient of a weight of rows x width behind ``z = (gain * x) @ W.T``, from ``x``
    in 8 bits: ``scale * gain * (dz.T @ x)`` over all leading axes.

    ``dz``: ``(..., rows)``, bfloat16; ``packed``: ``(..., width)`` from ``mx_pack``
    or ``rms_norm`` (with ``pack="normalized"`` give the norm's ``gain``); ``out``:
    rows x width in ``out_dtype`` (float32 or bfloat16, the default), allocated unless
    given; ``accumulate`` adds to it.  Sums are float32.  Returns ``out``.
    """
    return _call("weight_grad", dz, stream, dz, packed, gain, scale, out, out_dtype, accumulate)
