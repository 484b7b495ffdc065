"""Cross entropy where a workgroup of the logits kernels takes several tiles one
after the other, and where the vocabulary falls into pieces by its size."""
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402
from test_gpu_cross_entropy import BF16, DEV, RB, ULP32, check, make, reference  # noqa: E402

pytestmark = pytest.mark.gpu


# 9 x 36 tiles of 256: up to two for each of the 256 workgroups, 17 x 36: three;
# rows of 1, 3 and 4 stages of 64, and of a padded copy of w
@pytest.mark.parametrize("n,rows,width", [(2900, 9000, 64), (2900, 9000, 192), (2900, 9000, 256), (2900, 9000, 130),
                                          (5400, 9000, 128)])
def test_more_tiles_than_workgroups(n, rows, width):
    # of the tokens that `make` gives, about 3 in 11 are not counted
    print(f"[case] xent tiles {n} {rows} {width}", flush=True)
    x, w, t = make(n, rows, width, 41)
    full = check(x, w, t)
    xd, wd, td = x.to(DEV), w.to(DEV), t.to(DEV)
    only = mm.cross_entropy(xd, wd, td, grad=False)
    assert torch.equal(only[0], full[0]) and torch.equal(only[1], full[1])
    again = mm.cross_entropy(xd, wd, td)
    for a, b in zip(again, full):
        assert torch.equal(a, b)


def test_pieces_of_a_large_call():
    # P of 65536 tokens by 4400 words takes more than one piece holds; the
    # tokens are 16 copies of 4096, so that fp64 sees those alone
    print("[case] xent pieces without a limit", flush=True)
    copies, rows = 16, 4400
    x, w, t = make(4096, rows, 64, 42)
    ok = (t >= 0) & (t < rows)
    c = 1.0 / int(ok.sum())
    clean = torch.where(ok[:, None], x, torch.zeros((), dtype=BF16))
    loss, tol_loss, dx, tol_dx, dw, tol_dw = reference(clean, w, t, c, ok)
    got, tok, gx, gw = mm.cross_entropy(x.repeat(copies, 1).to(DEV), w.to(DEV), t.repeat(copies).to(DEV))
    assert abs(float(got) - float(loss.sum()) * c) <= float(tol_loss.sum()) * c + ULP32 * abs(float(got))
    # the copies stand in other tiles, with the same products in the same order
    tok, gx = tok.cpu().view(copies, -1), gx.cpu().view(copies, *x.shape)
    for k in range(1, copies):
        assert torch.equal(tok[k], tok[0]) and torch.equal(gx[k], gx[0])
    assert bool(((tok[0].double() - loss).abs() <= tol_loss).all())
    # dx: the mean is over 16 times the tokens, a power of two
    assert bool(((gx[0].double() * copies - dx).abs() <= tol_dx).all())
    # dw: a sum over 16 times the terms, each a 16th
    soft = (clean.double() @ w.double().t()).softmax(1)
    soft[torch.arange(len(t)), torch.where(ok, t, 0)] -= 1.0
    mag = (soft.abs() * ok[:, None] * c).t() @ clean.double().abs()
    tol = tol_dw + len(t) * (copies - 1) * ULP32 * mag
    assert bool(((gw.double().cpu() - dw).abs() <= tol + RB * (dw.abs() + tol)).all())
