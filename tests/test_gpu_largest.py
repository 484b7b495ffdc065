"""The largest tokens, rows and widths that the calls take, against fp64 on the GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402
from test_gpu_cross_entropy import BF16, ULP32, reference  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _inputs(n, rows, width, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(n, width, generator=g, device=DEV).bfloat16()
    w = (torch.randn(rows, width, generator=g, device=DEV) * (3.0 / math.sqrt(width))).bfloat16()
    t = torch.randint(0, rows, (n,), generator=g, device=DEV)
    t[1::7] = -100
    return x, w, t


@pytest.mark.parametrize("n,rows,width", [(100, 1 << 23, 8), (300, 700, 65536), (1 << 22, 300, 8)])
def test_cross_entropy(n, rows, width):
    print(f"[case] xent {n} tokens, {rows} x {width}", flush=True)
    x, w, t = _inputs(n, rows, width, 51)
    ok = t >= 0
    c = 1.0 / int(ok.sum())
    got, tok, gx, gw = mm.cross_entropy(x, w, t, dw_dtype=torch.float32)
    total, slack = 0.0, 0.0
    want = torch.zeros(rows, width, dtype=torch.float64, device=DEV)
    room, mag = torch.zeros_like(want), torch.zeros_like(want)
    for b in range(0, n, 1 << 19):  # fp64 logits of a block of tokens at a time
        s = slice(b, b + (1 << 19))
        clean = torch.where(ok[s, None], x[s], torch.zeros((), dtype=BF16, device=DEV))
        loss, tol, dx, tol_dx, dw, tol_dw = reference(clean, w, t[s], c, ok[s])
        assert bool(((tok[s].double() - loss).abs() <= tol).all())
        assert bool(((gx[s].double() - dx).abs() <= tol_dx).all())
        total, slack = total + float(loss.sum()), slack + float(tol.sum())
        want += dw
        room += tol_dw
        soft = (clean.double() @ w.double().t()).softmax(1)
        soft[torch.arange(len(loss), device=DEV), torch.where(ok[s], t[s], 0)] -= 1.0
        mag += (soft.abs() * ok[s, None] * c).t() @ clean.double().abs()
        del clean, loss, tol, dx, tol_dx, dw, tol_dw, soft
    assert abs(float(got) - total * c) <= slack * c + ULP32 * abs(total * c)
    # each block's tolerance counts the additions of its own tokens; all of them stand in one sum
    room += n * ULP32 * mag
    assert bool(((gw.double() - want).abs() <= room + ULP32 * (want.abs() + room)).all())
    only = mm.cross_entropy(x, w, t, grad=False)
    assert bool(((only[1] - tok).abs() <= 64 * ULP32 * (1 + tok.abs())).all())


def test_embedding_of_2_26_tokens():
    print("[case] embedding of 2^26 tokens", flush=True)
    n, rows, width = 1 << 26, 1000, 3
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    ids = torch.randint(-1, rows, (n,), generator=g, device=DEV, dtype=torch.int32)
    table = torch.randn(rows, width, generator=g, device=DEV)
    out = mm.embedding(table, ids)
    for b in range(0, n, n // 8):
        part = ids[b: b + n // 8].long()
        want = torch.where((part >= 0)[:, None], table[part.clamp(min=0)], torch.zeros((), device=DEV))
        assert torch.equal(out[b: b + n // 8], want)
    del out
    # whole numbers: about 67 thousand of them a row, every partial sum exact in fp32
    dout = torch.randint(-8, 9, (n, width), generator=g, device=DEV, dtype=torch.int32).to(torch.bfloat16)
    got = mm.embedding_grad(ids, dout, rows, out_dtype=torch.float32)
    ok = ids >= 0
    want = torch.zeros(rows, width, dtype=torch.float64, device=DEV)
    want.index_add_(0, torch.where(ok, ids, 0).long(), torch.where(ok[:, None], dout, torch.zeros((), dtype=BF16, device=DEV)).double())
    assert torch.equal(got.double(), want)
