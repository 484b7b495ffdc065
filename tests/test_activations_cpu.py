"""Refusals and sizes of the entry points between the embedding and the output layer,
without a GPU: every refused call here is rejected by host validation, before any HIP
call."""
import os

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = [pytest.mark.skipif(not os.path.exists(mm.LIB_PATH), reason="libmuonh.so not built"),
              pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that are never followed")]

NAN, INF = float("nan"), float("inf")
MB = 1 << 20
A, B, C, D, E, F, G, H, WS = (MB * k for k in range(1, 10))  # a megabyte apart
FAILS = (mm.MUONH_EINVAL, mm.MUONH_ENOTIMPL, mm.MUONH_ENOMEM)


def norm(x=A, xdt=1, res=B, hdt=0, gain=C, eps=1e-6, n=4, width=40, h=D, y=E, ydt=1, rstd=F, q=G, scales=H, packs=0):
    return mm.load().muonh_rms_norm(x, xdt, res, hdt, gain, eps, n, width, h, y, ydt, rstd, q, scales, packs, None)


def grad(dy=A, ydt=1, x=None, q=B, scales=C, rstd=D, gain=E, dres=F, xdt=0, n=4, width=40, dx=G, dgain=H, acc=0, ws=WS,
         ws_bytes=MB):
    return mm.load().muonh_rms_norm_grad(dy, ydt, x, q, scales, rstd, gain, dres, xdt, n, width, dx, dgain, acc, ws, ws_bytes,
                                         None)


def pack(x=A, xdt=1, n=4, width=40, q=B, scales=C):
    return mm.load().muonh_mx_pack(x, xdt, n, width, q, scales, None)


def unpack(q=A, scales=B, n=4, width=40, out=C, odt=1):
    return mm.load().muonh_mx_unpack(q, scales, n, width, out, odt, None)


def weight(dz=A, q=B, scales=C, gain=D, scale=1.0, n=4, rows=24, width=40, dw=E, wdt=1, acc=0, ws=WS, ws_bytes=MB):
    return mm.load().muonh_weight_grad(dz, q, scales, gain, scale, n, rows, width, dw, wdt, acc, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=A + 1), dict(x=A + 2, xdt=0), dict(xdt=2), dict(res=None), dict(h=None), dict(res=B + 2),
    dict(h=D + 1), dict(hdt=3), dict(gain=C + 2), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(n=-1),
    dict(width=0), dict(y=E + 1), dict(ydt=2), dict(rstd=F + 1), dict(q=None), dict(scales=None), dict(packs=2),
    # overlaps: 4 x 40 of bf16 x and y, fp32 h and residual, 160 bytes of gain and of q, 8 scales
    dict(h=A), dict(h=A + 316), dict(h=B + 4), dict(h=B - 4), dict(h=B, hdt=1, res=B + 2), dict(y=A), dict(y=A + 318),
    dict(y=B + 638), dict(y=C + 158), dict(y=D + 2), dict(rstd=D + 636), dict(rstd=E), dict(rstd=C + 156), dict(q=A + 319),
    dict(q=E - 159), dict(scales=G + 159), dict(scales=G - 7), dict(scales=F + 15), dict(q=D, scales=G),
])
def test_norm_refuses(kw):
    assert norm(**kw) == mm.MUONH_EINVAL


@pytest.mark.parametrize("kw", [
    dict(), dict(h=B), dict(res=None, h=None), dict(gain=None), dict(y=None), dict(rstd=None), dict(q=None, scales=None),
    dict(packs=1), dict(q=G + 1, scales=H + 3), dict(scales=G + 160), dict(h=B + 640), dict(y=A + 320), dict(x=A + 2),
    dict(width=16384, x=A, res=None, h=None, y=None, gain=None, q=None, scales=None, n=1),
])
def test_norm_takes(kw):
    # without a GPU the first launch fails: the checks were passed
    assert norm(**kw) == mm.MUONH_EHIP


def test_norm_limits():
    assert norm(width=16385) == norm(n=(1 << 26) + 1) == norm(n=1 << 26, width=16385) == mm.MUONH_ENOTIMPL
    assert norm(n=0, x=None) == mm.MUONH_OK  # nothing to do, nothing queued


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(dy=A + 1), dict(dy=A + 2, ydt=0), dict(ydt=5), dict(x=B, q=B), dict(x=None, q=None, scales=None),
    dict(x=None, q=None), dict(scales=None), dict(x=B + 2, q=None, scales=None), dict(x=B, q=None), dict(rstd=None),
    dict(rstd=D + 2), dict(gain=E + 1), dict(dres=F + 2), dict(xdt=2), dict(n=-1), dict(width=0), dict(dx=None),
    dict(dx=G + 2), dict(dgain=H + 2), dict(acc=2), dict(ws=None), dict(ws=WS + 128),
    dict(dx=A), dict(dx=B + 156), dict(dx=B - 636), dict(dx=C + 4), dict(dx=D + 12), dict(dx=E + 156), dict(dx=F + 4),
    dict(dx=F - 4), dict(dx=H + 156), dict(dgain=A + 316), dict(dgain=D), dict(dgain=E), dict(dgain=F + 636),
])
def test_grad_refuses(kw):
    assert grad(**kw) == mm.MUONH_EINVAL


@pytest.mark.parametrize("kw", [
    dict(), dict(x=B, q=None, scales=None), dict(gain=None), dict(dres=None), dict(dx=F), dict(dgain=None, ws=None),
    dict(acc=1), dict(dx=A + 320), dict(q=B + 3, scales=C + 1),
])
def test_grad_takes(kw):
    assert grad(**kw) == mm.MUONH_EHIP


def test_grad_limits_and_workspace():
    size = mm.load().muonh_rms_norm_grad_workspace
    assert size(-1, 40) == size(4, 0) == size(4, 16385) == size(1 << 27, 40) == 0
    for n, width in ((0, 40), (1, 1), (4, 40), (10 ** 6, 768), (100, 16384)):
        assert 4 * width <= size(n, width) <= 4 * width * min(max(n, 1), 1024) + 256
    assert grad(ws_bytes=size(4, 40) - 1) == mm.MUONH_ENOMEM
    assert grad(width=16385) == mm.MUONH_ENOTIMPL
    assert grad(n=0, dy=None, q=None, scales=None, rstd=None, dx=None, dgain=None) == mm.MUONH_OK
    assert grad(n=0, dy=None, q=None, scales=None, rstd=None, dx=None, acc=1) == mm.MUONH_OK


@pytest.mark.parametrize("call,kw", [
    (pack, dict(x=None)), (pack, dict(x=A + 1)), (pack, dict(x=A + 2, xdt=0)), (pack, dict(xdt=2)), (pack, dict(n=-1)),
    (pack, dict(width=0)), (pack, dict(q=None)), (pack, dict(scales=None)), (pack, dict(q=A + 319)), (pack, dict(q=A)),
    (pack, dict(scales=A + 1)), (pack, dict(scales=B + 159)), (pack, dict(scales=B - 7)),
    (unpack, dict(q=None)), (unpack, dict(scales=None)), (unpack, dict(out=None)), (unpack, dict(out=C + 1)),
    (unpack, dict(out=C + 2, odt=0)), (unpack, dict(odt=-1)), (unpack, dict(n=-2)), (unpack, dict(width=-1)),
    (unpack, dict(out=A)), (unpack, dict(out=A + 158)), (unpack, dict(out=B + 6)), (unpack, dict(out=B - 318)),
    (weight, dict(dz=None)), (weight, dict(dz=A + 1)), (weight, dict(q=None)), (weight, dict(scales=None)),
    (weight, dict(gain=D + 2)), (weight, dict(scale=NAN)), (weight, dict(scale=INF)), (weight, dict(n=-1)),
    (weight, dict(rows=0)), (weight, dict(width=0)), (weight, dict(dw=None)), (weight, dict(dw=E + 1)),
    (weight, dict(dw=E + 2, wdt=0)), (weight, dict(wdt=2)), (weight, dict(acc=2)), (weight, dict(ws=None)),
    (weight, dict(ws=WS + 16)), (weight, dict(dw=A)), (weight, dict(dw=A + 190)), (weight, dict(dw=B + 158)),
    (weight, dict(dw=C + 6)), (weight, dict(dw=D + 158)), (weight, dict(dw=A - 1918)),
])
def test_others_refuse(call, kw):
    assert call(**kw) == mm.MUONH_EINVAL


@pytest.mark.parametrize("call,kw", [
    (pack, dict()), (pack, dict(q=B + 1, scales=C + 1)), (pack, dict(x=A + 2)), (pack, dict(q=A + 320)),
    (unpack, dict()), (unpack, dict(q=A + 1, scales=B + 1)), (unpack, dict(out=A + 160)),
    (weight, dict()), (weight, dict(dz=A + 2)), (weight, dict(gain=None)), (weight, dict(dw=A + 192)),
    (weight, dict(acc=1, wdt=0)), (weight, dict(q=B + 5, scales=C + 3)), (weight, dict(n=0, dz=None, q=None, scales=None)),
])
def test_others_take(call, kw):
    assert call(**kw) == mm.MUONH_EHIP


def test_limits_and_workspace():
    assert pack(n=0, x=None, q=None, scales=None) == unpack(n=0, q=None, scales=None, out=None) == mm.MUONH_OK
    assert pack(width=(1 << 20) + 1) == unpack(width=(1 << 20) + 1) == pack(n=(1 << 26) + 1) == mm.MUONH_ENOTIMPL
    assert pack(n=1 << 26, width=1 << 15) == mm.MUONH_ENOTIMPL
    for kw in (dict(n=(1 << 22) + 1), dict(rows=(1 << 20) + 1), dict(width=(1 << 20) + 1), dict(rows=1 << 20, width=1 << 18),
               dict(n=1 << 22, rows=1 << 14), dict(n=1 << 22, width=1 << 14)):
        assert weight(**kw) == mm.MUONH_ENOTIMPL
    size = mm.load().muonh_weight_grad_workspace
    assert size(0, -1, 8, 8) == size(0, 8, 0, 8) == size(0, 8, 8, 0) == size(0, (1 << 22) + 1, 8, 8) == size(1, 8, 8, 8) == 0
    assert weight(ws_bytes=size(A, 4, 24, 40) - 1) == mm.MUONH_ENOMEM
    assert weight(n=0, acc=1, dz=None, q=None, scales=None) == mm.MUONH_OK
    # x in bf16, once; dz again where its rows are off the grid; never a share that grows with more than the sizes.
    # 56 x 16 tiles of 256 are 3 rounds of 256 and 128 tiles, these in two parts of 4 bytes a value
    n, rows, width = 8192, 14336, 4096
    assert size(0, n, rows, width) <= 2 * width * (n + 192) + 2 * 128 * 4 * 256 * 256 + 4096
    assert size(0, n, 16 * 256, width) <= 2 * width * (n + 192) + 4096
    assert size(2, n, rows, width) >= 2 * n * (rows + width)
    assert size(0, n, rows + 1, width) >= 2 * n * (rows + width)


def test_python_checks():
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    a, g = torch.zeros(4, 40), torch.zeros(40)
    with pytest.raises(ValueError, match="pack must"):
        mm.rms_norm(a, pack="both")
    with pytest.raises(ValueError, match="last axis"):
        mm.rms_norm(torch.zeros(4, 0))
    with pytest.raises(ValueError, match="last axis"):
        mm.mx_pack(torch.zeros(()))
    with pytest.raises(ValueError, match="GPU"):
        mm.rms_norm(a, g)
    with pytest.raises(ValueError, match="GPU"):
        mm.rms_norm_grad(a, a, g[:4])
    with pytest.raises(ValueError, match="GPU"):
        mm.mx_pack(a)
    with pytest.raises(TypeError, match="e4m3"):
        mm.mx_unpack((a, a))
    with pytest.raises(TypeError, match="e4m3"):
        mm.mx_unpack((a.to(f8), a))
    with pytest.raises(ValueError, match="GPU"):
        mm.mx_unpack((a.to(f8), torch.zeros(4, 2, dtype=torch.uint8).view(e8)))
    with pytest.raises(ValueError, match="GPU"):
        mm.weight_grad(a.bfloat16(), (a.to(f8), torch.zeros(4, 2, dtype=torch.uint8).view(e8)))
