"""Outputs that overlap what a call still reads, or another output, are refused on
the host: nothing is queued, no pointer is followed."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = [pytest.mark.skipif(not os.path.exists(mm.LIB_PATH), reason="libmuonh.so not built"),
              pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that are never followed")]

MB = 1 << 20
A, B, C, D, E, F, WS = (MB * k for k in range(1, 8))  # a megabyte apart


def arr(t, v):
    return (t * len(v))(*v)


def emb(out, table=A, ids=B):
    # 100 x 8 fp32 table, 10 int64 ids, bf16 out
    return mm.load().muonh_embedding(table, 0, 100, 8, ids, 64, 10, 1.0, out, 1, None)


def emb_grad(dtable, dout=A, ids=B):
    return mm.load().muonh_embedding_grad(ids, 64, 10, dout, 1, 1.0, 0, dtable, 0, 100, 8, WS, MB, None)


def xent(x=A, w=B, t=C, loss=D, tok=D + 256, dx=E, dw=F):
    # 10 tokens, 100 x 8 bf16, fp32 dw
    return mm.load().muonh_cross_entropy(x, w, t, 64, 10, 100, 8, -100, 0, 1.0, loss, tok, dx, dw, 0, 0, WS, 1 << 30, None)


def clip(total=C, coef=C + 4, outs=(A, A + 256)):
    return mm.load().muonh_clip_grads(arr(ctypes.c_uint64, (A, A + 256)), arr(ctypes.c_uint64, outs),
                                      arr(ctypes.c_int64, (8, 8)), arr(ctypes.c_int, (0, 1)), 2, 1.0, total, coef, WS,
                                      MB, None)


@pytest.mark.parametrize("call,kw", [
    (emb, dict(out=A)), (emb, dict(out=A + 3198)), (emb, dict(out=A - 158)), (emb, dict(out=B + 78)), (emb, dict(out=B - 2)),
    (emb_grad, dict(dtable=A)), (emb_grad, dict(dtable=A + 156)), (emb_grad, dict(dtable=A - 3196)),
    (emb_grad, dict(dtable=B + 76)),
    (xent, dict(dw=B)), (xent, dict(dw=B + 1596)), (xent, dict(dw=C + 76)), (xent, dict(dw=E + 156)),
    (xent, dict(dx=B)), (xent, dict(dx=C)), (xent, dict(dx=F + 3198)),
    (xent, dict(tok=A + 156)), (xent, dict(loss=B + 1596)), (xent, dict(loss=E)), (xent, dict(loss=F + 3196)),
    (xent, dict(tok=C + 76)), (xent, dict(tok=D)), (xent, dict(tok=E + 156)), (xent, dict(loss=C)),
    (clip, dict(total=A)), (clip, dict(coef=A + 28)), (clip, dict(coef=A + 268)), (clip, dict(total=B, outs=(B, D))),
    (clip, dict(coef=C)), (clip, dict(coef=D + 12, outs=(B, D))),
])
def test_refused(call, kw):
    assert call(**kw) == mm.MUONH_EINVAL


@pytest.mark.parametrize("call,kw", [
    # side by side; the gradients and the loss over x, which is copied first; nothing asked for
    (emb, dict(out=A + 3200)), (emb, dict(out=A - 160)), (emb, dict(out=B + 80)),
    (emb_grad, dict(dtable=A + 160)), (emb_grad, dict(dtable=A - 3200)),
    (xent, dict()), (xent, dict(dx=A)), (xent, dict(dx=A + 2)), (xent, dict(dw=A)), (xent, dict(loss=A)),
    (xent, dict(tok=A + 160)), (xent, dict(dx=A + 160)), (xent, dict(dw=B + 1600)), (xent, dict(tok=None)),
    (xent, dict(dx=None, dw=None)), (xent, dict(dx=None)), (xent, dict(loss=A + 160)),
    (clip, dict()), (clip, dict(total=A + 32)), (clip, dict(total=A + 272)),
])
def test_taken(call, kw):
    # without a GPU the first launch fails: the checks were passed
    assert call(**kw) == mm.MUONH_EHIP
