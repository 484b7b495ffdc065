"""The root-mean-square norm with the residual's addition, and its gradient, against fp64."""
import math

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative
HALF = {BF16: 2.0 ** -8, F32: U}
TINY = {BF16: 2.0 ** -133, F32: 2.0 ** -149}  # and below the normal range


def rnd(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def within(got, want, bound, what):
    d = (got.double().cpu() - want).abs()
    bad = ~(d <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(d[bad].max()), float((d / bound.clamp(min=1e-300)).max()))


def values(packed):
    q, s = packed
    f = s.cpu().view(torch.uint8).double().sub(127).exp2().repeat_interleave(32, -1)[..., :q.shape[-1]]
    return q.cpu().to(F32).double() * f, f


def check_packed(packed, want, rel):
    """8-bit rows against `want`, whose own values are known to `rel`."""
    got, f = values(packed)
    n, d = want.shape
    pad = torch.zeros(n, -(-d // 32) * 32, dtype=torch.float64)
    pad[:, :d] = want.abs()
    top = pad.view(n, -1, 32).amax(2)
    s = packed.scales.cpu().view(torch.uint8).double().sub(127).exp2()
    assert bool((top <= 448 * s * (1 + rel)).all())                          # holds the block
    assert bool(((top >= 224 * s * (1 - rel)) | (s == 2.0 ** -117)).all())   # and is the least to
    within(got, want, 2.0 ** -4 * want.abs() * (1 + 16 * rel) + 2.0 ** -10 * f + rel * want.abs(), "packed")


WIDTHS = [1, 7, 8, 31, 33, 64, 511, 513, 768, 1024, 1999, 2048, 2049, 4096, 5001, 8192, 8200, 16384]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("xt,rt,yt", [(BF16, None, BF16), (F32, None, F32), (BF16, F32, BF16), (BF16, BF16, F32), (F32, BF16, BF16),
                                      (F32, F32, F32)])
def test_norm(width, xt, rt, yt):
    print(f"[case] norm {width} {xt} {rt} {yt}", flush=True)
    for n, pack in ((1, "normalized"), (13, "output")):
        x = rnd(width, n, width, dtype=xt)
        res = None if rt is None else rnd(width + 1, n, width, dtype=rt, scale=3.0)
        gain = 1 + rnd(width + 2, width, scale=0.3)
        h = x if rt is None else (x.float() + res.float()).to(rt)
        r = mm.rms_norm(x.to(DEV), gain.to(DEV), residual=None if rt is None else res.to(DEV), eps=1e-5, pack=pack, out_dtype=yt)
        if rt is not None:
            assert torch.equal(r.h.cpu(), h)
        else:
            assert r.h is None
        v = h.double()
        rstd = (v.square().mean(1) + float(torch.tensor(1e-5))) ** -0.5
        within(r.rstd, rstd, rstd * U * 1.001, "rstd")
        xn = v * rstd[:, None]
        y = xn * gain.double()
        # rstd, its product and the gain's are rounded to fp32, then the result
        within(r.y, y, y.abs() * (HALF[yt] + 3.01 * U) + TINY[yt], "y")
        check_packed(r.packed, xn if pack == "normalized" else y, 3.01 * U)


def test_norm_parts():
    print("[case] parts of the norm", flush=True)
    x, res = rnd(1, 5, 3, 200, dtype=BF16).to(DEV), rnd(2, 5, 3, 200).to(DEV)
    whole = mm.rms_norm(x, residual=res, pack="output")
    assert whole.y.shape == x.shape and whole.rstd.shape == (5, 3) and whole.packed.scales.shape == (5, 3, 7)
    few = mm.rms_norm(x, residual=res, output=False)
    assert few.y is None and few.packed is None and torch.equal(few.h, whole.h) and torch.equal(few.rstd, whole.rstd)
    # without a gain the output is the normalised row
    assert torch.equal(mm.rms_norm(x, residual=res, pack="normalized").packed.q.view(torch.uint8), whole.packed.q.view(torch.uint8))
    # into given buffers, the residual's own among them
    out, stream = torch.full_like(x, 7), res.clone()
    got = mm.rms_norm(x, residual=stream, h=stream, out=out)
    assert got.h is stream and got.y is out and torch.equal(stream, whole.h) and torch.equal(out, whole.y)
    assert torch.equal(mm.rms_norm(whole.h, out_dtype=BF16).y, whole.y)


@pytest.mark.parametrize("width", [96, 1500, 6000])
def test_norm_extremes(width):
    print(f"[case] norm extremes {width}", flush=True)
    x = rnd(3, 12, width)
    x[1] = 0.0
    x[2] *= 1e30            # squares beyond fp32
    x[3] *= 1e-30           # and below it: eps decides
    x[4, width // 2] = math.nan
    x[5, 3] = math.inf
    x[6, 3] = -1e38         # one value far above its row
    x[7] = 1e-45            # fp32's least
    x[8] = 3e38
    gain = 1 + rnd(4, width, scale=0.3)
    r = mm.rms_norm(x.to(DEV), gain.to(DEV), eps=1e-6, pack="normalized")
    v = x.double()
    rstd = (v.square().mean(1) + float(torch.tensor(1e-6))) ** -0.5
    ok = [k for k in range(12) if k not in (4, 5)]
    within(r.rstd[ok], rstd[ok], rstd[ok] * U * 1.001 + TINY[F32], "rstd")
    xn = v * rstd[:, None]
    # rstd below fp32's normal range has an absolute error
    low = TINY[F32] * v.abs() * (1 + gain.double().abs()) + TINY[F32]
    within(r.y[ok], (xn * gain.double())[ok], (xn * gain.double()).abs()[ok] * 4.01 * U + low[ok], "y")
    assert bool(r.y[4].isnan().all()) and float(r.rstd[5]) == 0.0
    want5 = torch.zeros(width)
    want5[3] = math.nan
    assert torch.equal(r.y[5].cpu().nan_to_num(nan=9.0), want5.nan_to_num(nan=9.0))
    got, _ = values(r.packed)
    assert bool(got[4].isnan().all()) and bool(got[5, 3].isnan()) and float(got[5].nan_to_num(nan=0.0).abs().max()) == 0.0
    assert bool(got[ok].isfinite().all())


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("yt,rt,kept,res", [(BF16, F32, "packed", True), (BF16, BF16, "packed", False), (F32, F32, "input", True),
                                            (BF16, BF16, "input", True), (F32, BF16, "packed", True), (F32, F32, "packed", False),
                                            (BF16, F32, "input", False), (F32, BF16, "input", False)])
def test_grad(width, yt, rt, kept, res):
    print(f"[case] norm gradient {width} {yt} {rt} {kept} {res}", flush=True)
    for n in (1, 37):
        h = rnd(width, n, width, dtype=rt, scale=2.0).to(DEV)
        dy = rnd(width + 1, n, width, dtype=yt, scale=1e-3)
        gain = 1 + rnd(width + 2, width, scale=0.3)
        dres = rnd(width + 3, n, width, dtype=rt, scale=1e-3) if res else None
        r = mm.rms_norm(h, pack="normalized" if kept == "packed" else None)
        dx, dg = mm.rms_norm_grad(dy.to(DEV), r.packed if kept == "packed" else h, r.rstd, gain.to(DEV),
                                  dres=None if dres is None else dres.to(DEV), out_dtype=rt)
        assert dx.dtype == rt and dg.dtype == F32
        s = r.rstd.double().cpu()[:, None]
        xn = values(r.packed)[0] if kept == "packed" else h.double().cpu() * s
        u = dy.double() * gain.double()
        c = (u * xn).mean(1, keepdim=True)
        d = 0.0 if dres is None else dres.double()
        want = d + s * (u - xn * c)
        # c: u and xn rounded, sums of 16 and 6 in a lane and over lanes, 16 waves, the mean; then
        # the difference, the last step and the result
        dc = 46 * U * (u * xn).abs().mean(1, keepdim=True)
        bound = s * (3 * U * u.abs() + 4 * U * (xn * c).abs() + xn.abs() * dc) + (HALF[rt] + U) * want.abs() + TINY[rt]
        within(dx, want, bound, "dx")
        prod = dy.double() * xn
        within(dg, prod.sum(0), (n + 40) * U * prod.abs().sum(0) + TINY[F32], "dgain")


def test_grad_against_differences():
    print("[case] norm gradient against differences", flush=True)
    n, d = 3, 50
    h, w, gain = rnd(1, n, d), rnd(2, n, d), 1 + rnd(3, d, scale=0.2)
    f = lambda v, g: float(((v * (v.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * g) * w.double()).sum())  # noqa: E731
    r = mm.rms_norm(h.to(DEV), gain.to(DEV))
    dx, dg = mm.rms_norm_grad(w.to(DEV), h.to(DEV), r.rstd, gain.to(DEV))
    step = 1e-5
    for t, got, at in ((h, dx, [(0, 0), (1, 17), (2, 49)]), (gain, dg, [(0,), (31,), (49,)])):
        for i in at:
            a, b = t.double().clone(), t.double().clone()
            a[i] += step
            b[i] -= step
            pair = ((a, gain.double()), (b, gain.double())) if t is h else ((h.double(), a), (h.double(), b))
            diff = (f(*pair[0]) - f(*pair[1])) / (2 * step)
            # second-order terms step^2 of values around 1, and fp32 sums of 50 terms
            assert abs(float(got[i]) - diff) <= 1e-5 * max(1.0, abs(diff)), (i, float(got[i]), diff)


def test_grad_parts():
    print("[case] parts of the norm gradient", flush=True)
    n, d = 300, 1100
    h, dy, gain = rnd(1, n, d).to(DEV), rnd(2, n, d, dtype=BF16).to(DEV), (1 + rnd(3, d, scale=0.2)).to(DEV)
    dres = rnd(4, n, d).to(DEV)
    r = mm.rms_norm(h, gain, pack="normalized")
    dx, dg = mm.rms_norm_grad(dy, r.packed, r.rstd, gain, dres=dres)
    assert dx.dtype == F32
    # in place over the residual's gradient, without the gain's, into a sum
    buf = dres.clone()
    got, none = mm.rms_norm_grad(dy, r.packed, r.rstd, gain, dres=buf, out=buf, gain_grad=False)
    assert got is buf and none is None and torch.equal(buf, dx)
    total = torch.full((d,), 2.0, device=DEV)
    mm.rms_norm_grad(dy, r.packed, r.rstd, gain, dres=dres, dgain=total, accumulate=True)
    assert torch.equal(total, 2.0 + dg)
    one, dg1 = mm.rms_norm_grad(dy, r.packed, r.rstd, dres=dres, gain_grad=True)
    assert torch.equal(dg1, dg)
    same, none = mm.rms_norm_grad(dy, r.packed, r.rstd, torch.ones_like(gain), dres=dres, gain_grad=False)
    assert torch.equal(same, one)
    assert mm.rms_norm_grad(dy, h, r.rstd)[1] is None
    # bitwise the same again, and rows do not reach each other
    again, dg2 = mm.rms_norm_grad(dy, r.packed, r.rstd, gain, dres=dres)
    assert torch.equal(again, dx) and torch.equal(dg2, dg)
    bad = dy.clone()
    bad[7] = math.nan
    spoilt, _ = mm.rms_norm_grad(bad, r.packed, r.rstd, gain, dres=dres)
    keep = [k for k in range(n) if k != 7]
    assert bool(spoilt[7].isnan().all()) and torch.equal(spoilt[keep], dx[keep])


@pytest.mark.parametrize("n,d", [(20000, 96), (9000, 1000), (5000, 2500), (3000, 8192), (1500, 16000)])
def test_many_rows(n, d):
    """More rows than the launch has workgroups."""
    print(f"[case] many rows {n} {d}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    h = torch.randn(n, d, generator=g, device=DEV, dtype=F32).bfloat16()
    dy = torch.randn(n, d, generator=g, device=DEV, dtype=F32).bfloat16()
    gain = torch.rand(d, generator=g, device=DEV) + 0.5
    r = mm.rms_norm(h, gain, pack="normalized")
    rstd = (h.double().square().mean(1) + float(torch.tensor(1e-6))) ** -0.5
    assert bool(((r.rstd.double() - rstd).abs() <= 1.001 * U * rstd).all())
    y = h.double() * rstd[:, None] * gain.double()
    assert bool(((r.y.double() - y).abs() <= (2.0 ** -8 + 4 * U) * y.abs()).all())
    dx, dg = mm.rms_norm_grad(dy, h, r.rstd, gain)
    xn, u = h.double() * r.rstd.double()[:, None], dy.double() * gain.double()
    c = (u * xn).mean(1, keepdim=True)
    want = r.rstd.double()[:, None] * (u - xn * c)
    bound = r.rstd.double()[:, None] * (3 * U * u.abs() + 4 * U * (xn * c).abs() + xn.abs() * 46 * U * (u * xn).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - want).abs() <= bound + (2.0 ** -8 + U) * want.abs() + TINY[BF16]).all())
    prod = dy.double() * xn
    # a lane's rows (n over 256 workgroups at least), the workgroup's lanes, the join's 32 + 32
    assert bool(((dg.double() - prod.sum(0)).abs() <= (n / 256 + 80) * U * prod.abs().sum(0)).all())


def test_smallest_eps_and_widths():
    print("[case] norm, smallest eps", flush=True)
    for width in (1, 8, 700):
        x = torch.zeros(3, width)
        x[1], x[2] = 1e-30, -5.0
        r = mm.rms_norm(x.to(DEV), eps=1e-45, pack="output")
        eps = float(torch.tensor(1e-45))
        rstd = (x.double().square().mean(1) + eps) ** -0.5
        within(r.rstd, rstd, rstd * U * 1.001, "rstd")
        within(r.y, x.double() * rstd[:, None], (x.double() * rstd[:, None]).abs() * 3.01 * U, "y")
        dx, _ = mm.rms_norm_grad(torch.zeros(3, width, device=DEV), r.packed, r.rstd)
        assert bool((dx == 0).all())


def test_empty_and_refused():
    print("[case] norm, empty and refused", flush=True)
    e = torch.zeros(0, 64, device=DEV, dtype=BF16)
    r = mm.rms_norm(e, residual=torch.zeros(0, 64, device=DEV), pack="output")
    assert r.y.shape == (0, 64) and r.h.shape == (0, 64) and r.rstd.shape == (0,) and r.packed.scales.shape == (0, 2)
    dg = torch.ones(64, device=DEV)
    dx, got = mm.rms_norm_grad(e, e, r.rstd, dg, dgain=dg.clone())
    assert dx.shape == (0, 64) and bool((got == 0).all())
    assert bool((mm.rms_norm_grad(e, r.packed, r.rstd, dg, dgain=got, accumulate=True)[1] == 0).all())
    x, gain, rs = torch.zeros(4, 64, device=DEV), torch.zeros(64, device=DEV), torch.zeros(4, device=DEV)
    p = mm.mx_pack(x)
    for kw in (dict(gain=gain[:5]), dict(gain=gain.bfloat16()), dict(residual=x[:2]), dict(residual=x.double()), dict(h=x),
               dict(residual=x, h=x.bfloat16()), dict(out=x[:1]), dict(out=x.clone(), output=False), dict(residual=x.t().t()[:, :32]),
               dict(out=x.clone(), out_dtype=BF16), dict(gain=torch.zeros(64)), dict(out=x)):
        with pytest.raises((ValueError, TypeError, mm.MuonhError)):
            mm.rms_norm(x, **kw)
    with pytest.raises(ValueError):
        mm.rms_norm(x.t())
    with pytest.raises(TypeError):
        mm.rms_norm(x.half())
    with pytest.raises(mm.MuonhError):
        mm.rms_norm(x, eps=0.0)
    for args, kw in (((x, x.bfloat16(), rs), dict(out_dtype=F32)), ((x, x, rs[:3]), {}), ((x, x, rs.double()), {}),
                     ((x, x[:2], rs), {}), ((x, mm.mx_pack(x[:2]), rs), {}), ((x, p, rs), dict(dres=x.bfloat16(), out_dtype=F32)),
                     ((x, p, rs), dict(accumulate=True)), ((x, p, rs), dict(dgain=gain[:3])),
                     ((x, p, rs), dict(dgain=gain, gain_grad=False)), ((x, (p.q, p.scales[:, :1]), rs), {}),
                     ((x, p, rs), dict(out=x)), ((x.half(), p, rs), {})):
        with pytest.raises((ValueError, TypeError, mm.MuonhError)):
            mm.rms_norm_grad(*args, **kw)


@pytest.mark.parametrize("pack", ["normalized", "output"])
def test_packed_rows_are_rounded_once(pack):
    """8-bit rows are those of the row in 64 bits: with some 10^7 values, whose fp32 value
    lies on a border of e4m3 or on its other side ten times."""
    print(f"[case] packed rows rounded once, {pack}", flush=True)
    n, d = 10000, 1024
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    x = torch.randn(n, d, generator=g, device=DEV)
    gain = torch.rand(d, generator=g, device=DEV) + 0.5
    r = mm.rms_norm(x, gain, pack=pack, output=False)
    v = x.double() * (x.double().square().mean(1, keepdim=True) + float(torch.tensor(1e-6))) ** -0.5
    if pack == "output":
        v = v * gain.double()
    b = v.view(n, -1, 32)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    assert torch.equal((e[..., 0] + 127).to(torch.uint8), r.packed.scales.view(torch.uint8))
    t = torch.ldexp(b, -e)
    unit = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    want = (torch.round(t / unit) * unit).view(n, d)
    assert torch.equal(r.packed.q.double(), want)


@pytest.mark.parametrize("n,d", [(5001, 8), (4999, 50), (30000, 64), (7000, 65), (3001, 100), (50001, 128), (2500, 175), (2049, 256),
                                 (1500, 257)])
def test_narrow_rows(n, d):
    """Rows that share a wave (heads of an attention), in every direction."""
    print(f"[case] narrow rows {n} {d}", flush=True)
    test_many_rows(n, d)
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    x = torch.randn(n, d, generator=g, device=DEV)
    gain = torch.rand(d, generator=g, device=DEV) + 0.5
    # each row by itself, whatever its neighbours in the wave hold
    r = mm.rms_norm(x, gain, pack="normalized")
    y = x.clone()
    y[1::3] = math.nan
    s = mm.rms_norm(y, gain, pack="normalized")
    keep = [k for k in range(n) if k % 3 != 1]
    assert torch.equal(s.y[keep], r.y[keep]) and torch.equal(s.rstd[keep], r.rstd[keep])
    assert torch.equal(s.packed.q.view(torch.uint8)[keep], r.packed.q.view(torch.uint8)[keep])
    assert bool(s.y[1::3].isnan().all())
    for kept in (r.packed, x):
        dx, dg = mm.rms_norm_grad(x, kept, r.rstd, gain)
        xn = mm.mx_unpack(kept, out_dtype=F32).double() if kept is not x else x.double() * r.rstd.double()[:, None]
        prod = x.double() * xn
        assert bool(((dg.double() - prod.sum(0)).abs() <= (n / 256 + 80) * U * prod.abs().sum(0)).all())
        few, dg2 = mm.rms_norm_grad(x[:300], kept[:300] if kept is x else type(kept)(kept.q[:300], kept.scales[:300]), r.rstd[:300], gain)
        assert torch.equal(few, dx[:300])
        assert bool(((dg2.double() - prod[:300].sum(0)).abs() <= 340 * U * prod[:300].abs().sum(0)).all())
