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


@pytest.mark.parametrize("n", [3, 40])
def test_loss_of_few_tokens_over_many_rounds(n):
    """Every workgroup's largest logit stands in its first round of words, and
    64 rounds follow that do not change the maximum: its weight stays 1.

    x has one entry (1, 1/2, 1/4 or -1) and w one column (29.0 or 0), so the logits
    are exact in fp32.  What the arithmetic may lose: the exponent's argument is
    the difference of two fp32 values of log2(e) times at most 29.0, below 64,
    each rounded by at most 2^-19 (a relative 2^-19 ln 2 of the sum; allowed
    three times: in a lane, between lanes, between workgroups); 2^-24 for each of
    the additions that a term goes through (32 words of a tile, 64 rounds, two
    lanes, 32 workgroups of a lane) and 2^-22 for v_exp_f32, together below 64 *
    2^-22; and log, the sum with the maximum and the difference with the target's
    logit, each half a unit of a value below 64, 2^-19."""
    print(f"[case] xent rounds {n}", flush=True)
    rows, first = 1 << 23, 2048 * 64
    w = torch.zeros(rows, 8, dtype=BF16)
    w[:first:4, 0] = 29.0
    x = torch.zeros(n, 8, dtype=BF16)
    x[:, 0] = torch.tensor([1.0, 0.5, 0.25, -1.0])[torch.arange(n) % 4]
    t = torch.tensor([0, 1, rows - 1])[torch.arange(n) % 3]
    high, low = first // 4, rows - first // 4
    lx = x[:, 0].double() * 29.0
    top = lx.clamp(min=0.0)
    lse = top + (high * (lx - top).exp() + low * (-top).exp()).log()
    want = lse - x[:, 0].double() * w[t, 0].double()
    got, tok, _, _ = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), grad=False)
    tol = 6 * 2.0 ** -19 + 64 * 2.0 ** -22
    err = (tok.double().cpu() - want).abs()
    print(f"  off by at most {float(err.max()):.2e} of {tol:.2e}", flush=True)
    assert bool((err <= tol).all())
    assert abs(float(got) - float(want.mean())) <= tol + ULP32 * float(want.mean())
