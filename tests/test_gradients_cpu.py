"""Refusals and sizes of the entry points around the step, without a GPU: every
call here is rejected by host validation, before any HIP call."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(mm.LIB_PATH), reason="libmuonh.so not built")

P = 0x100000  # a pointer that is never followed
NAN, INF = float("nan"), float("inf")


def arr(t, v):
    return (t * len(v))(*v)


def norm(clip=False, n=2, numel=(8, 8), dtypes=(0, 1), ptrs=(P, P + 256), outs=(P + 512, P + 768), max_norm=1.0, total=P,
         coef=P + 4, ws=P, ws_bytes=1 << 20, null=None):
    lib = mm.load()
    a = dict(g=arr(ctypes.c_uint64, ptrs), n=arr(ctypes.c_int64, numel), d=arr(ctypes.c_int, dtypes),
             o=arr(ctypes.c_uint64, outs))
    g, nu, d, o = (None if null == k else a[k] for k in "gndo")
    if clip:
        return lib.muonh_clip_grads(g, o, nu, d, n, max_norm, total, coef, ws, ws_bytes, None)
    return lib.muonh_grad_norm(g, nu, d, n, max_norm, total, coef, None, ws, ws_bytes, None)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=-1), dict(null="g"), dict(null="n"), dict(null="d"), dict(numel=(-1, 8)), dict(numel=(1 << 60, 8)),
    dict(dtypes=(2, 0)), dict(dtypes=(0, -1)), dict(ptrs=(0, P)), dict(ptrs=(P + 2, P)), dict(ptrs=(P, P + 1)),
    dict(max_norm=-1.0), dict(max_norm=NAN), dict(max_norm=INF), dict(total=None), dict(ws=None), dict(ws=P + 16),
])
def test_norm_and_clip_refuse(clip, kw):
    assert norm(clip, **kw) == mm.MUONH_EINVAL


@pytest.mark.parametrize("kw", [dict(null="o"), dict(outs=(0, P)), dict(outs=(P, P + 1)), dict(coef=None), dict(outs=(P, P))])
def test_clip_refuses(kw):
    assert norm(True, **kw) == mm.MUONH_EINVAL


def test_norm_workspace():
    lib = mm.load()
    assert lib.muonh_grad_norm_workspace(0) == 0 and lib.muonh_grad_norm_workspace(-3) == 0
    sizes = [lib.muonh_grad_norm_workspace(n) for n in (1, 2, 100, 5000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    for clip in (False, True):
        assert norm(clip, ws_bytes=lib.muonh_grad_norm_workspace(2) - 1) == mm.MUONH_ENOMEM
    assert norm(n=1 << 25) == mm.MUONH_ENOTIMPL


def emb(table=P, tdt=0, rows=10, width=8, ids=P, bits=64, n=4, scale=1.0, out=P, odt=1):
    return mm.load().muonh_embedding(table, tdt, rows, width, ids, bits, n, scale, out, odt, None)


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(table=P + 2), dict(tdt=2), dict(odt=5), dict(rows=0), dict(rows=1 << 31), dict(width=0),
    dict(ids=None), dict(ids=P + 4), dict(bits=16), dict(n=-1), dict(scale=NAN), dict(scale=INF), dict(out=None),
    dict(out=P + 1),
])
def test_embedding_refuses(kw):
    assert emb(**kw) == mm.MUONH_EINVAL


def test_embedding_limits():
    assert emb(n=0, ids=None, out=None) == mm.MUONH_OK  # nothing to do, nothing queued
    assert emb(width=(1 << 18) + 1) == mm.MUONH_ENOTIMPL
    assert emb(n=(1 << 26) + 1) == mm.MUONH_ENOTIMPL
    assert emb(n=1 << 26, width=2048) == mm.MUONH_ENOTIMPL


def emb_grad(ids=P, bits=64, n=4, dout=P, ddt=1, scale=1.0, acc=0, dtable=P, tdt=0, rows=10, width=8, ws=P, ws_bytes=1 << 20):
    return mm.load().muonh_embedding_grad(ids, bits, n, dout, ddt, scale, acc, dtable, tdt, rows, width, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(ids=None), dict(ids=P + 4), dict(bits=8), dict(n=-1), dict(dout=None), dict(dout=P + 1), dict(ddt=2),
    dict(scale=NAN), dict(acc=2), dict(acc=-1), dict(dtable=None), dict(dtable=P + 2), dict(tdt=3), dict(rows=0),
    dict(width=0), dict(ws=None), dict(ws=P + 8),
])
def test_embedding_grad_refuses(kw):
    assert emb_grad(**kw) == mm.MUONH_EINVAL


def test_embedding_grad_workspace():
    lib = mm.load()
    assert lib.muonh_embedding_grad_workspace(-1, 10, 8) == 0
    assert lib.muonh_embedding_grad_workspace(4, 0, 8) == 0
    assert lib.muonh_embedding_grad_workspace(1 << 27, 10, 8) == 0
    need = lib.muonh_embedding_grad_workspace(4, 10, 8)
    assert need >= 4 * 4 * 4
    assert emb_grad(ws_bytes=need - 1) == mm.MUONH_ENOMEM
    assert emb_grad(n=(1 << 26) + 1) == mm.MUONH_ENOTIMPL
    # a share of dout (partial rows), whatever the table's rows but for the digits' counts (2^11 x 64 blocks at most)
    small, large = (lib.muonh_embedding_grad_workspace(65536, rows, 2048) for rows in (1000, 10 ** 9))
    assert small <= large <= small + 4 * 64 * 2 ** 11 and large < 65536 * 2048 * 2


def xent(x=P, w=P, t=P, bits=64, n=4, rows=10, width=8, ign=-100, red=0, gs=1.0, loss=P, tok=P, dx=P, dw=P, wdt=1, acc=0,
         ws=P, ws_bytes=1 << 30):
    return mm.load().muonh_cross_entropy(x, w, t, bits, n, rows, width, ign, red, gs, loss, tok, dx, dw, wdt, acc, ws,
                                         ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=P + 1), dict(w=None), dict(w=P + 1), dict(t=None), dict(t=P + 4), dict(bits=16), dict(n=-1),
    dict(rows=0), dict(width=0), dict(red=2), dict(red=-1), dict(gs=NAN), dict(gs=INF), dict(loss=None), dict(loss=P + 2),
    dict(tok=P + 2), dict(dx=P + 1), dict(dw=P + 1), dict(dw=P + 2, wdt=0), dict(wdt=2), dict(acc=3), dict(ws=None),
    dict(ws=P + 128),
])
def test_cross_entropy_refuses(kw):
    assert xent(**kw) == mm.MUONH_EINVAL


def test_cross_entropy_limits_and_workspace():
    lib = mm.load()
    for kw in (dict(n=(1 << 22) + 1), dict(rows=(1 << 23) + 1), dict(width=65537), dict(n=1 << 22, width=8192)):
        assert xent(**kw) == mm.MUONH_ENOTIMPL
    size = lib.muonh_cross_entropy_workspace
    assert size(0, -1, 10, 8, 3, 0) == 0 and size(0, 4, 10, 8, 4, 0) == 0 and size(0, 4, 10, 8, -1, 0) == 0
    loss_only, both = size(0, 4096, 50257, 768, 0, 0), size(0, 4096, 50257, 768, 3, 0)
    assert 0 < loss_only < size(0, 4096, 50257, 768, 2, 0) <= both
    # never the logits: less than their bf16 size with every gradient, at any size of vocabulary
    assert both - loss_only < 2 * 4096 * 200000 and size(0, 4096, 10 ** 6, 768, 3, 0) < 2 * 4096 * 10 ** 6 / 4
    assert xent(n=4096, rows=50257, width=768, ws_bytes=loss_only) == mm.MUONH_ENOMEM
    # a limit gives a layout within it, and none below the smallest
    for limit in (both, both // 2, both // 4):
        got = size(0, 4096, 50257, 768, 3, limit)
        assert 0 < got <= limit
    assert size(0, 4096, 50257, 768, 3, 1 << 20) == 0
    # an address off the 16-byte grid needs the copy of w
    assert size(2, 4096, 50257, 768, 0, 0) > loss_only + 2 * 50257 * 768 - (1 << 20)


def test_python_checks():
    a, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="no gradients"):
        mm.grad_norm([])
    with pytest.raises(ValueError, match="no gradients"):
        mm.clip_grads([], 1.0)
    with pytest.raises(ValueError, match="GPU"):
        mm.grad_norm([a])
    with pytest.raises(ValueError, match="GPU"):
        mm.clip_grads([a], 1.0)
    with pytest.raises(TypeError, match="dtype"):
        mm.grad_norm([a.double()])
    with pytest.raises(ValueError, match="GPU"):
        mm.embedding(a, i)
    with pytest.raises(ValueError, match="2-D"):
        mm.embedding(a[0], i)
    with pytest.raises(ValueError, match="GPU"):
        mm.embedding_grad(i, a, 10)
    with pytest.raises(ValueError, match="GPU"):
        mm.cross_entropy(a.bfloat16(), a.bfloat16(), i)
    with pytest.raises(ValueError, match="reduction"):
        mm.cross_entropy(a.bfloat16(), a.bfloat16(), i, reduction="none")
    with pytest.raises(ValueError, match="grad must be"):
        mm.cross_entropy(a.bfloat16(), a.bfloat16(), i, grad="both")
    with pytest.raises(ValueError, match="grad_scale"):
        mm.make_opts(grad_scale=torch.ones(1), stream=0)


def test_tensor_lists():
    from matrix_orthogonalizing_optimizer_momentum_amd import _tensors
    assert _tensors.table([], "x") == (b"", b"", b"", -1)
    a = torch.zeros(4)
    for bad, err in ((3, TypeError), ([a, 3], ValueError), ([3], TypeError), ([None], TypeError), ([a], ValueError),
                     ([a.half()], TypeError), ([a.to_sparse()], ValueError)):
        with pytest.raises(err):
            _tensors.table(bad, "x")


def test_options_carry_the_scale():
    o = mm.Opts()
    mm.load().muonh_default_opts(ctypes.byref(o))
    assert o.grad_scale is None
    assert ctypes.sizeof(mm.Opts) % 8 == 0 and mm.Opts.grad_scale.offset == ctypes.sizeof(mm.Opts) - 8


@pytest.mark.parametrize("ptrs,outs", [
    ((P, P + 256), (P + 256, P)),           # each the other's
    ((P, P + 256), (P + 512, P + 528)),     # outs overlap: 8 float32 and 8 bfloat16
    ((P, P + 256), (P + 16, P + 768)),      # its own gradient, not in place
    ((P, P + 256), (P + 240, P + 768)),     # the next one's first values
    ((P, P + 256), (P, P + 16)),            # in place, and inside the first
])
def test_clip_refuses_overlapping_buffers(ptrs, outs):
    assert norm(True, ptrs=ptrs, outs=outs) == mm.MUONH_EINVAL
    # behind the check of the workspace when they are apart
    assert norm(True, ptrs=ptrs, outs=(P + 1024, P + 1056), ws_bytes=1) == mm.MUONH_ENOMEM
    assert norm(True, ptrs=(P, P), outs=(P + 32, P + 64), ws_bytes=1) == mm.MUONH_ENOMEM
    assert norm(True, ptrs=(P, P + 32), outs=(P, P + 32), ws_bytes=1) == mm.MUONH_ENOMEM
    assert norm(True, ptrs=(P, P + 32), outs=(P, P + 64), numel=(8, 0), ws_bytes=1) == mm.MUONH_ENOMEM


def test_grad_scale_of_another_device():
    from types import SimpleNamespace
    scale = SimpleNamespace(is_cuda=True, dtype=torch.float32, numel=lambda: 1, data_ptr=lambda: P,
                            device=torch.device("cuda:1"))
    stream = lambda i: SimpleNamespace(cuda_stream=0, device=torch.device("cuda", i))  # noqa: E731
    with pytest.raises(ValueError, match="another device"):
        mm.make_opts(grad_scale=scale, stream=stream(0))
    assert mm.make_opts(grad_scale=scale, stream=stream(1))[0].grad_scale == P
