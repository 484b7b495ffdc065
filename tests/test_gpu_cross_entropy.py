"""The output layer's cross entropy and its gradients against fp64."""
import math

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
ULP32 = 2.0 ** -23   # one unit of an fp32 value, relative: twice its rounding
RB = 2.0 ** -8       # one rounding to bf16, relative


def make(n, rows, width, seed, spread=3.0, pad=True):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    x = torch.randn(n, width, generator=g).bfloat16()
    w = (torch.randn(rows, width, generator=g) * (spread / math.sqrt(width))).bfloat16()
    t = torch.randint(0, rows, (n,), generator=g)
    if pad and n > 2:
        t[1::5] = -100
        t[2::11] = rows
    return x, w, t


def reference(x, w, t, c, ok):
    """fp64 values and the tolerances that the arithmetic allows, on the CPU.

    A logit is a sum of `width` exact products, each fp32 addition off by at
    most one unit of the sum of magnitudes so far: dl = width * ULP32 * sum|x w|.
    The exponent's argument is rounded a few times more (l and lse in units of
    log2(e) are at most 1.5 |l|: 8 units of the largest logit cover both).  The
    sum of exponents is a tree whose longest path is 32 values in a lane, the
    wave's halves and rows, and one of 8 chains over the tiles."""
    X, W = x.double(), w.double()
    n, rows = X.shape[0], W.shape[0]
    L = X @ W.t()
    lse = torch.logsumexp(L, 1)
    at = torch.where(ok, t, 0)
    loss = torch.where(ok, lse - L.gather(1, at[:, None])[:, 0], 0.0)
    dl = X.shape[1] * ULP32 * (X.abs() @ W.abs().t()) + 8 * ULP32 * L.abs().amax(1, keepdim=True)
    path = 32 + 4 + 8 + 8 + (rows / 256) / 8
    dlse = dl.amax(1) + path * ULP32
    tol_loss = torch.where(ok, dlse + dl.gather(1, at[:, None])[:, 0] + 2 * ULP32 * lse.abs(), 0.0)
    soft = (L - lse[:, None]).exp()
    P = soft.clone()
    P[torch.arange(n), at] -= 1.0
    P = P * ok[:, None] * c
    # P is off by the exponent's error and one rounding to bf16
    dP = (soft * ok[:, None] * c) * (dl + dlse[:, None]) * 1.1 + RB * P.abs() * 1.01 + 2 * ULP32 * c
    dx = P @ W
    tol_dx = dP @ W.abs() + (rows + 64) * ULP32 * (P.abs() @ W.abs())
    tol_dx = tol_dx + RB * (dx.abs() + tol_dx)
    dw = P.t() @ X
    tol_dw = dP.t() @ X.abs() + (n + 64) * ULP32 * (P.abs().t() @ X.abs())
    return loss, tol_loss, dx, tol_dx, dw, tol_dw


def check(x, w, t, reduction="mean", ignore_index=-100, grad_scale=1.0, dw_dtype=BF16, **kw):
    rows = w.shape[0]
    ok = (t >= 0) & (t < rows) & (t != ignore_index)
    count = int(ok.sum())
    c = (1.0 / max(1, count) if reduction == "mean" else 1.0)
    clean = torch.where(ok[:, None], x, torch.zeros((), dtype=BF16))
    loss, tol_loss, dx, tol_dx, dw, tol_dw = reference(clean, w, t, c * grad_scale, ok)
    got, tok, gx, gw = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), reduction=reduction, ignore_index=ignore_index,
                                        grad_scale=grad_scale, dw_dtype=dw_dtype, **kw)
    assert gx.dtype == BF16 and gw.dtype == dw_dtype and got.dtype == F32 and tok.dtype == F32
    e = (tok.double().cpu() - loss).abs()
    assert bool((e <= tol_loss).all()), float((e - tol_loss).max())
    assert abs(float(got) - float(loss.sum()) * c) <= float(tol_loss.sum()) * c + ULP32 * abs(float(got))
    e = (gx.double().cpu() - dx).abs()
    assert bool((e <= tol_dx).all()), float((e - tol_dx).max())
    assert bool((gx.cpu()[~ok] == 0).all())
    r = RB if dw_dtype == BF16 else ULP32
    tol_dw = tol_dw + r * (dw.abs() + tol_dw)
    e = (gw.double().cpu() - dw).abs()
    assert bool((e <= tol_dw).all()), float((e - tol_dw).max())
    return got, tok, gx, gw


SHAPES = [  # tokens, rows, width
    (1, 1, 1), (1, 2, 64), (3, 5, 7), (17, 255, 64), (256, 256, 64), (257, 513, 128), (300, 1000, 100), (64, 5000, 72),
    (1000, 3001, 320), (700, 777, 1024), (255, 2049, 576),
]


@pytest.mark.parametrize("n,rows,width", SHAPES)
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_values(n, rows, width, reduction):
    print(f"[case] xent {n} tokens, {rows} x {width}, {reduction}", flush=True)
    x, w, t = make(n, rows, width, 7)
    check(x, w, t, reduction)


@pytest.mark.parametrize("n,rows,width", [(257, 513, 128), (300, 2000, 100), (520, 5001, 192)])
def test_pieces(n, rows, width):
    # a limit that leaves room for one 256-row piece of the vocabulary
    print(f"[case] xent pieces {n} {rows} {width}", flush=True)
    x, w, t = make(n, rows, width, 8)
    lib = mm.load()
    lo, hi = 1, 1 << 32
    while lo < hi:  # the smallest limit that is enough
        mid = (lo + hi) // 2
        if lib.muonh_cross_entropy_workspace(0, n, rows, width, 3, mid):
            hi = mid
        else:
            lo = mid + 1
    got, tok, gx, gw = check(x, w, t, workspace_limit=lo)
    one = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV))
    assert torch.equal(one[0], got) and torch.equal(one[1], tok)  # the loss does not see the pieces
    assert torch.equal(one[3], gw)                                # nor does a row of dw
    with pytest.raises(mm.MuonhError) as e:
        mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), workspace_limit=lo - 1)
    assert e.value.code == mm.MUONH_ENOMEM


def test_bitwise_reproducible():
    print("[case] xent twice", flush=True)
    x, w, t = (a.to(DEV) for a in make(1000, 3001, 320, 9))
    a, b = mm.cross_entropy(x, w, t), mm.cross_entropy(x, w, t)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_parts_and_types():
    print("[case] xent parts", flush=True)
    x, w, t = make(300, 1000, 192, 10)
    full = check(x, w, t, "sum", grad_scale=0.25, dw_dtype=F32)
    xd, wd, td = x.to(DEV), w.to(DEV), t.to(DEV)
    only = mm.cross_entropy(xd, wd, td, reduction="sum", grad=False)
    assert only[2] is None and only[3] is None and torch.equal(only[0], full[0]) and torch.equal(only[1], full[1])
    gx = mm.cross_entropy(xd, wd, td, reduction="sum", grad="x", grad_scale=0.25)
    assert gx[3] is None and torch.equal(gx[2], full[2])
    gw = mm.cross_entropy(xd, wd, td, reduction="sum", grad="w", grad_scale=0.25, dw_dtype=F32)
    assert gw[2] is None and torch.equal(gw[3], full[3])
    i32 = mm.cross_entropy(xd.view(3, 100, 192), wd, td.int().view(3, 100), reduction="sum", grad_scale=0.25,
                           dw_dtype=F32)
    assert i32[1].shape == (3, 100) and i32[2].shape == (3, 100, 192)
    for p, q in zip(i32, full):
        assert torch.equal(p.flatten(), q.flatten())


def test_accumulates():
    print("[case] xent accumulate", flush=True)
    x, w, t = make(300, 1000, 192, 11)
    xd, wd, td = x.to(DEV), w.to(DEV), t.to(DEV)
    for dt in (F32, BF16):
        add = mm.cross_entropy(xd, wd, td, dw_dtype=F32)[3]
        start = torch.randn(1000, 192, device=DEV).to(dt)
        out = start.clone()
        got = mm.cross_entropy(xd, wd, td, dw=out, accumulate=True)[3]
        assert got.data_ptr() == out.data_ptr()
        assert torch.equal(got, (start.float() + add).to(dt))


def test_tokens_that_are_not_counted():
    print("[case] xent masks", flush=True)
    x, w, t = make(300, 700, 128, 12)
    bad = (t < 0) | (t >= 700)
    dirty = x.clone()
    dirty[bad] = float("nan")
    dirty[torch.nonzero(bad)[::2, 0]] = float("inf")
    a = check(dirty, w, t)
    b = check(x, w, t)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    # an ignored id inside the table
    check(x, w, t, ignore_index=int(t[0]))
    # none counted
    got = mm.cross_entropy(dirty.to(DEV), w.to(DEV), torch.full((300,), -1, device=DEV))
    assert float(got[0]) == 0
    for p in got[1:]:
        assert bool((p == 0).all())
    keep = torch.randn(700, 128, device=DEV)
    got = mm.cross_entropy(dirty.to(DEV), w.to(DEV), torch.full((300,), -1, device=DEV), dw=keep.clone(), accumulate=True)
    assert torch.equal(got[3], keep)
    empty = mm.cross_entropy(x[:0].to(DEV), w.to(DEV), t[:0].to(DEV))
    assert float(empty[0]) == 0 and empty[2].shape == (0, 128) and bool((empty[3] == 0).all())


def test_one_counted_token_at_the_end():
    print("[case] xent last token", flush=True)
    x, w, t = make(1025, 300, 64, 13, pad=False)
    t[:-1] = -100
    check(x, w, t)


@pytest.mark.parametrize("spread", [1e-3, 100.0, 1e4])
def test_flat_and_peaked(spread):
    # logits up to tens of thousands: the softmax is one word, no exponent may
    # overflow
    print(f"[case] xent spread {spread}", flush=True)
    x, w, t = make(200, 600, 64, 14, spread=spread)
    got = check(x, w, t, "sum")
    assert all(bool(torch.isfinite(p).all()) for p in got)


def test_non_finite_rows_stay_in_their_token():
    print("[case] xent non-finite", flush=True)
    x, w, t = (a.to(DEV) for a in make(300, 700, 128, 15, pad=False))
    clean = mm.cross_entropy(x, w, t)
    x[5, 3] = float("nan")
    got = mm.cross_entropy(x, w, t)
    assert torch.isnan(got[0]) and torch.isnan(got[1][5]) and torch.isnan(got[2][5]).all()
    keep = torch.arange(300, device=DEV) != 5
    assert torch.equal(got[1][keep], clean[1][keep]) and torch.equal(got[2][keep], clean[2][keep])
    assert torch.isnan(got[3]).all()  # every word's gradient sums over every counted token


def _offset(t, k):
    buf = torch.empty(t.numel() + k, dtype=t.dtype, device=t.device)
    v = buf[k:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("k", [1, 4])
def test_unaligned_buffers(k):
    print(f"[case] xent offset {k}", flush=True)
    x, w, t = make(300, 700, 128, 16)
    xd, wd, td = x.to(DEV), w.to(DEV), t.to(DEV)
    want = mm.cross_entropy(xd, wd, td)
    dx, dw = _offset(torch.zeros_like(xd), k), _offset(torch.zeros_like(wd), k)
    got = mm.cross_entropy(_offset(xd, k), _offset(wd, k), _offset(td, k), dx=dx, dw=dw)
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_gradients_against_differences():
    # the loss itself, in fp32 at inputs that bf16 holds: a central difference
    # of the fp64 loss along random directions
    print("[case] xent differences", flush=True)
    x, w, t = make(40, 300, 64, 17)
    ok = (t >= 0) & (t < 300)
    _, _, dx, dw = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), dw_dtype=F32)

    def loss(X, W):
        L = X[ok] @ W.t()
        return (torch.logsumexp(L, 1) - L[torch.arange(len(L)), t[ok]]).mean()

    g = torch.Generator().manual_seed(3)
    h = 1e-4
    for name, base, other, grad in (("x", x, w, dx), ("w", w, x, dw)):
        for _ in range(4):
            v = torch.randn(base.shape, generator=g, dtype=torch.float64)
            a, b, o = base.double() + h * v, base.double() - h * v, other.double()
            d = (loss(a, o) - loss(b, o)) / (2 * h) if name == "x" else (loss(o, a) - loss(o, b)) / (2 * h)
            got = (grad.double().cpu() * v).sum()
            # P and the result are each within 2^-8 of their values; the directions' signs do not favour any
            slack = 2 * RB * (grad.double().cpu() * v).norm() + 1e-6
            assert abs(float(d - got)) <= float(slack) * 4


@pytest.mark.parametrize("n,rows,width", [(1024, 259, 64), (1025, 259, 64), (1365, 3070, 64), (1366, 3070, 72), (5000, 1500, 64)])
def test_both_sides_of_the_size_rules(n, rows, width):
    # tokens listed by the gathering blocks (up to 1024) or by a launch of their
    # own; loss by one workgroup (tokens x tiles up to 16384) or by many
    print(f"[case] xent sizes {n} {rows} {width}", flush=True)
    x, w, t = make(n, rows, width, 18)
    check(x, w, t)
    ok = (t >= 0) & (t < rows)
    only = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), grad=False)
    assert bool((only[1].cpu()[~ok] == 0).all())


@pytest.mark.parametrize("n", [1, 37, 300, 1100])
def test_words_shut_out_by_an_infinite_weight(n):
    """A word whose logits are all -inf has weight 0 everywhere: the loss and
    the other words' gradients are those without it, and its own is zero, whatever
    stands behind the last token."""
    print(f"[case] xent infinite weight, {n} tokens", flush=True)
    x, w, t = make(n, 600, 128, 21)
    x[:, 5] = 1.0
    shut = [17, 300, 599]
    t[torch.isin(t, torch.tensor(shut))] = 0
    ok = (t >= 0) & (t < 600)
    c = 1.0 / max(1, int(ok.sum()))
    keep = torch.ones(600, dtype=torch.bool)
    keep[shut] = False
    place = torch.cumsum(keep, 0) - 1
    small = torch.where(ok, place[t.clamp(0, 599)], 0)
    loss, tol_loss, _, _, dw, tol_dw = reference(torch.where(ok[:, None], x, torch.zeros((), dtype=BF16)), w[keep],
                                                 small, c, ok)
    w[shut, 5] = -math.inf
    got, tok, gx, gw = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), grad="w", dw_dtype=F32)
    assert gx is None
    assert bool(((tok.double().cpu() - loss).abs() <= tol_loss).all())
    assert abs(float(got) - float(loss.sum()) * c) <= float(tol_loss.sum()) * c + ULP32 * abs(float(got))
    assert bool((gw.cpu()[~keep] == 0).all())
    e = (gw.double().cpu()[keep] - dw).abs()
    assert bool((e <= tol_dw + ULP32 * dw.abs()).all()), float((e - tol_dw).max())


def check_loss(x, w, t, reduction="mean"):
    """The loss alone, with the tolerance of `reference`."""
    ok = (t >= 0) & (t < w.shape[0])
    c = 1.0 / max(1, int(ok.sum())) if reduction == "mean" else 1.0
    clean = torch.where(ok[:, None], x, torch.zeros((), dtype=BF16))
    loss, tol, *_ = reference(clean, w, t, c, ok)
    got, tok, gx, gw = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), reduction=reduction, grad=False)
    assert gx is None and gw is None
    e = (tok.double().cpu() - loss).abs()
    assert bool((e <= tol).all()), float((e - tol).max())
    assert bool((tok.cpu()[~ok] == 0).all())
    assert abs(float(got) - float(loss.sum()) * c) <= float(tol.sum()) * c + ULP32 * abs(float(got))
    return got, tok


@pytest.mark.parametrize("n", [1, 5, 31, 32, 33, 64, 65])
@pytest.mark.parametrize("rows,width", [(1, 1), (63, 7), (64, 64), (65, 63), (1000, 65), (5001, 320), (70000, 100)])
def test_loss_of_few_tokens(n, rows, width):
    print(f"[case] xent loss, {n} tokens, {rows} x {width}", flush=True)
    x, w, t = make(n, rows, width, 31)
    if n > 4:
        t[4] = rows - 1
        x[1] = math.inf  # not counted
    check_loss(x, w, t, "sum" if n % 2 else "mean")


@pytest.mark.parametrize("n", [3, 40])
def test_loss_of_few_tokens_off_the_grid(n):
    print(f"[case] xent loss off the grid, {n}", flush=True)
    x, w, t = make(n, 900, 130, 32)
    want = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), grad=False)
    got = mm.cross_entropy(_offset(x.to(DEV), 1), _offset(w.to(DEV), 3), _offset(t.to(DEV), 1), grad=False)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # and as int32, on another stream, captured
    s = torch.cuda.Stream()
    X, W, T = x.to(DEV), w.to(DEV), t.to(DEV).int()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = mm.cross_entropy(X, W, T, grad=False)
    for _ in range(3):
        out[0].zero_(), out[1].fill_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])


def test_loss_of_few_tokens_none_counted_and_not_finite():
    print("[case] xent loss, none counted / not finite", flush=True)
    x, w, t = make(6, 300, 96, 33, pad=False)
    got = mm.cross_entropy(x.to(DEV), w.to(DEV), torch.full((6,), -100, device=DEV), grad=False)
    assert float(got[0]) == 0 and bool((got[1] == 0).all())
    got = mm.cross_entropy(x[:0].to(DEV), w.to(DEV), t[:0].to(DEV), grad=False)
    assert float(got[0]) == 0 and got[1].numel() == 0
    x[2, 7] = math.nan  # stays in its token
    got = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), grad=False)
    assert bool(got[1][2].isnan()) and bool(got[0].isnan())
    assert bool(got[1].isfinite()[[0, 1, 3, 4, 5]].all())
    # words shut out by an infinite weight
    x, w, t = make(6, 300, 96, 34, pad=False)
    x[:, 5] = 1.0
    t[:] = torch.tensor([0, 1, 2, 3, 4, 5])
    want = mm.cross_entropy(x.to(DEV), w[:100].contiguous().to(DEV), t.to(DEV), grad=False)
    w[100:, 5] = -math.inf
    got = mm.cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV), grad=False)
    # both are one sum of the same exponents, in two groupings
    assert bool(((got[1] - want[1]).abs() <= 64 * ULP32 * (1 + want[1].abs())).all())
