"""Gradient norm, clipping and the embedding against plain fp64 computations."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}  # one rounding, relative


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def _offset(t, k):
    """A copy of t that starts k elements into its buffer."""
    buf = torch.empty(t.numel() + k, dtype=t.dtype, device=t.device)
    v = buf[k:].view(t.shape)
    v.copy_(t)
    return v


LISTS = {
    "one-element": [((1,), F32)],
    "scalar-and-empty": [((), F32), ((0,), BF16), ((0, 5), F32), ((3,), BF16)],
    "odd-sizes": [((7, 13), BF16), ((8191,), F32), ((8192,), BF16), ((8193,), BF16), ((255, 257), F32)],
    "many": [((1 + 37 * i % 501,), (F32, BF16)[i % 2]) for i in range(300)],
    "large-and-small": [((4099, 1031), BF16), ((3,), F32), ((2048, 2050), F32)],
}


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_norm(name, shift):
    print(f"[case] norm {name} shift {shift}", flush=True)
    ts = [_offset(_rand(s, d, 10 + i, 1e-3), shift) for i, (s, d) in enumerate(LISTS[name])]
    sq = [float((t.double() ** 2).sum()) for t in ts]
    total, coef, norms = mm.grad_norm(ts, max_norm=0.01)
    want = math.sqrt(sum(sq))
    # fp64 sums: what is left is the rounding of the result to fp32
    assert abs(float(total) - want) <= 1.01 * U[F32] * want
    assert norms.shape == (len(ts),)
    for a, b in zip(norms.tolist(), sq):
        assert abs(a - math.sqrt(b)) <= 1.01 * U[F32] * math.sqrt(b)
    c = min(1.0, float(np.float32(0.01)) / (want + 1e-6))
    assert abs(float(coef) - c) <= 1.01 * U[F32] * c
    again = mm.grad_norm(ts, max_norm=0.01)
    assert torch.equal(again[0], total) and torch.equal(again[2], norms)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [3e38, 1e-38])
def test_norm_of_extreme_values(dtype, value):
    print(f"[case] extreme {dtype} {value}", flush=True)
    t = torch.full((1000,), value, dtype=dtype, device=DEV)
    want = float(t[0].double()) * math.sqrt(1000.0)
    got = float(mm.grad_norm([t])[0])
    if want > float(np.finfo(np.float32).max):
        assert math.isinf(got)
    else:
        assert abs(got - want) <= 1.01 * U[F32] * want


def test_norm_of_non_finite_values():
    print("[case] non-finite", flush=True)
    for bad in (float("inf"), -float("inf"), float("nan")):
        a, b = _rand((100, 10), BF16, 1), _rand((77,), F32, 2)
        b[5] = bad
        total, coef, norms = mm.grad_norm([a, b], max_norm=1.0)
        if math.isnan(bad):
            assert torch.isnan(total) and torch.isnan(coef) and torch.isnan(norms[1])
        else:
            assert torch.isinf(total) and float(coef) == 0.0 and torch.isinf(norms[1])
        assert torch.isfinite(norms[0])


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("shift,oshift", [(0, 0), (1, 1), (2, 5)])
@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 1e9])
def test_clip_into_buffers(name, shift, oshift, max_norm):
    print(f"[case] clip {name} shift {shift} {oshift} max {max_norm}", flush=True)
    ts = [_offset(_rand(s, d, 40 + i, 1e-2), shift) for i, (s, d) in enumerate(LISTS[name])]
    keep = [t.clone() for t in ts]
    outs = [_offset(torch.full_like(t, 7.0), oshift) for t in ts]
    total, coef = mm.clip_grads(ts, max_norm, outputs=outs)
    c = float(coef)
    assert c <= 1.0 and (max_norm < 1e9 or c == 1.0)
    for t, k, o in zip(ts, keep, outs):
        assert torch.equal(t, k)
        # coef is an fp32 number: the product is rounded once to fp32 and once to the output
        want = (k.float() * coef).to(k.dtype)
        assert torch.equal(o, want)
    if 0 < max_norm < 1e9 and float(total) > max_norm:
        n2 = math.sqrt(sum(float((o.double() ** 2).sum()) for o in outs))
        assert n2 <= max_norm * (1 + 2 * U[BF16])


@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
def test_clip_in_place(max_norm):
    print(f"[case] clip in place {max_norm}", flush=True)
    ts = [_rand(s, d, 60 + i, 1e-2) for i, (s, d) in enumerate(LISTS["many"])]
    keep = [t.clone() for t in ts]
    total, coef = mm.clip_grads(ts, max_norm)
    for t, k in zip(ts, keep):
        assert torch.equal(t, (k.float() * coef).to(k.dtype))


def test_clipped_steps_equal_steps_on_scaled_gradients():
    # fp32 state: s * G formed by the caller and s * G formed in the step round
    # the same way up to the product's own rounding (2^-24 of a term).
    print("[case] grad_scale in the steps", flush=True)
    shapes = [(96, 64), (130, 257)]
    rho = [1.0, 1.0]
    for kw in (dict(), dict(tile_T=64), dict(hook="radial_brake", momentum="ema", nesterov=True)):
        w = [_rand(s, F32, 5 + i, 0.02) for i, s in enumerate(shapes)]
        m = [_rand(s, F32, 15 + i, 1e-3) for i, s in enumerate(shapes)]
        g = [_rand(s, F32, 25 + i, 1e-3) for i, s in enumerate(shapes)]
        _, coef, _ = mm.grad_norm(g, max_norm=0.01)
        assert 0 < float(coef) < 1
        w2, m2 = [t.clone() for t in w], [t.clone() for t in m]
        mm.muonh_step(w, g, m, 0.02, 0.95, 5, rho=rho, ns_dtype="f32", grad_scale=coef, **kw)
        mm.muonh_step(w2, [t * coef for t in g], m2, 0.02, 0.95, 5, rho=rho, ns_dtype="f32", **kw)
        for a, b in zip(m, m2):
            assert float((a - b).abs().max()) <= 4 * U[F32] * float(b.abs().max())
        for a, b in zip(w, w2):
            # the Newton-Schulz map amplifies small singular values by up to 3.4445^5 = 485
            assert float((a - b).norm()) <= 1e-4 * float(b.norm())


@pytest.mark.parametrize("tile", [0, 64, 256])
@pytest.mark.parametrize("noalloc", [False, True])
def test_step_with_power_of_two_scale_is_the_scaled_step(tile, noalloc):
    # A power of two scales bf16 gradients exactly: the two calls form the
    # same momentum, bit for bit.
    print(f"[case] power-of-two scale, tile {tile} noalloc {noalloc}", flush=True)
    shapes = [(256, 384), (300, 200)]
    w = [_rand(s, F32, 5 + i, 0.02) for i, s in enumerate(shapes)]
    m = [_rand(s, BF16, 15 + i, 1e-3) for i, s in enumerate(shapes)]
    g = [_rand(s, BF16, 25 + i, 1e-3) for i, s in enumerate(shapes)]
    w2, m2 = [t.clone() for t in w], [t.clone() for t in m]
    coef = torch.tensor([0.25], device=DEV)
    mm.muonh_step(w, g, m, 0.02, 0.95, 5, rho=[1.0, 2.0], tile_T=tile, noalloc=noalloc, grad_scale=coef)
    mm.muonh_step(w2, [t * 0.25 for t in g], m2, 0.02, 0.95, 5, rho=[1.0, 2.0], tile_T=tile, noalloc=noalloc)
    for a, b in zip(w + m, w2 + m2):
        assert torch.equal(a, b)


@pytest.mark.parametrize("hook", ["none", "hyperball"])
def test_adam_step_with_scale(hook):
    print(f"[case] adam scale {hook}", flush=True)
    shapes = [(1, 768), (257, 130)]
    w = [_rand(s, F32, 5 + i, 0.02) for i, s in enumerate(shapes)]
    g = [_rand(s, BF16, 25 + i, 1e-3) for i, s in enumerate(shapes)]
    m, v = [torch.zeros_like(t) for t in w], [torch.zeros_like(t) for t in w]
    w2, m2, v2 = ([t.clone() for t in x] for x in (w, m, v))
    kw = dict(eta=1e-3, step=1, rho=[1.0, 1.0], hook=hook)
    mm.adamh_step(w, g, m, v, grad_scale=torch.tensor(0.5, device=DEV), **kw)
    mm.adamh_step(w2, [t * 0.5 for t in g], m2, v2, **kw)
    for a, b in zip(w + m + v, w2 + m2 + v2):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ embedding

def _ids(n, rows, kind, dtype, seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    if kind == "uniform":
        v = torch.randint(0, rows, (n,), generator=g)
    elif kind == "one":
        v = torch.full((n,), rows // 2)
    elif kind == "skewed":
        v = (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * math.log(rows + 1.0)) - 1).long().clamp(0, rows - 1)
    else:  # every third token is padding of some kind
        v = torch.randint(0, rows, (n,), generator=g)
        v[::3] = torch.tensor([-100, -1, rows, 2 ** 31 - 1])[torch.arange(len(v[::3])) % 4]
    return v.to(dtype).to(DEV)


EMB = [  # rows, width, n
    (1, 1, 1), (5, 3, 7), (257, 8, 64), (1000, 100, 333), (50257, 768, 17), (2049, 1030, 129), (70000, 64, 5000),
]


@pytest.mark.parametrize("rows,width,n", EMB)
@pytest.mark.parametrize("tt,ot", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
def test_embedding(rows, width, n, tt, ot):
    print(f"[case] embedding {rows} x {width}, {n} tokens, {tt} {ot}", flush=True)
    table = _rand((rows, width), tt, 1)
    for kind, idt in (("uniform", torch.int64), ("padded", torch.int32), ("padded", torch.int64)):
        ids = _ids(n, rows, kind, idt, 2)
        out = mm.embedding(table, ids, scale=1.7, out_dtype=ot)
        ok = (ids >= 0) & (ids < rows)
        want = table[torch.where(ok, ids, 0).long()].float() * torch.tensor(1.7, device=DEV)
        want = torch.where(ok[:, None], want, torch.zeros((), device=DEV)).to(ot)
        assert torch.equal(out, want)


def test_embedding_shapes_and_non_finite_rows():
    print("[case] embedding shapes", flush=True)
    table = _rand((11, 16), BF16, 1)
    table[3] = float("nan")
    ids = torch.tensor([[0, 1, -1], [2, 10, 11]], device=DEV)
    out = mm.embedding(table, ids)
    assert out.shape == (2, 3, 16) and out.dtype == BF16
    assert torch.equal(out[0, 0], table[0]) and float(out[0, 2].abs().sum()) == 0 and float(out[1, 2].abs().sum()) == 0
    assert torch.isnan(mm.embedding(table, torch.tensor([3], device=DEV))).all()
    assert mm.embedding(table, torch.empty(0, dtype=torch.int64, device=DEV)).shape == (0, 16)
    odd = _offset(table, 1)  # not on a 16-byte grid
    assert torch.equal(mm.embedding(odd, ids), out)


def _grad_ref(ids, dout, rows, scale):
    ok = (ids >= 0) & (ids < rows)
    w = dout.double().cpu().numpy()
    want, mag = np.zeros((rows, dout.shape[1])), np.zeros((rows, dout.shape[1]))
    at = ids[ok].long().cpu().numpy()
    np.add.at(want, at, w[ok.cpu().numpy()])
    np.add.at(mag, at, np.abs(w[ok.cpu().numpy()]))
    return want * scale, mag * abs(scale), np.bincount(at, minlength=rows)


EGRAD = [  # rows, width, n, kind
    (1, 1, 1, "uniform"), (5, 3, 7, "uniform"), (7, 8, 200, "uniform"), (1000, 100, 333, "padded"),
    (300, 64, 32, "one"), (300, 64, 33, "one"), (300, 72, 5000, "one"), (4097, 130, 1024, "skewed"),
    (4097, 136, 1025, "skewed"), (50257, 64, 9000, "skewed"), (2 ** 22 + 5, 1, 3000, "uniform"),
    (200, 16, 70000, "padded"),
]


@pytest.mark.parametrize("rows,width,n,kind", EGRAD)
@pytest.mark.parametrize("gt,ot", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_embedding_grad(rows, width, n, kind, gt, ot):
    print(f"[case] embedding grad {rows} x {width}, {n} tokens {kind}, {gt} {ot}", flush=True)
    ids = _ids(n, rows, kind, torch.int32 if n % 2 else torch.int64, 3)
    dout = _rand((n, width), gt, 4)
    scale = 0.5
    got = mm.embedding_grad(ids, dout, rows, scale=scale, out_dtype=ot)
    assert got.shape == (rows, width) and got.dtype == ot
    want, mag, cnt = _grad_ref(ids, dout, rows, scale)
    # k terms: at most k fp32 additions, each off by 2^-24 of a partial sum that
    # the sum of magnitudes bounds; then the output's rounding
    tol = cnt[:, None] * U[F32] * mag + U[ot] * (np.abs(want) + cnt[:, None] * U[F32] * mag)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol + 1e-300).all(), float((err - tol).max())
    again = mm.embedding_grad(ids, dout, rows, scale=scale, out_dtype=ot)
    assert torch.equal(got, again)
    # accumulate: what was there, plus the sum
    start = _rand((rows, width), ot, 5)
    acc = mm.embedding_grad(ids, dout, scale=scale, out=start.clone(), accumulate=True)
    s = start.double().cpu().numpy()
    tol = (cnt[:, None] + 1) * U[F32] * (mag + np.abs(s)) + U[ot] * np.abs(s + want) * (1 + 1e-3)
    err = np.abs(acc.double().cpu().numpy() - (s + want))
    assert (err[cnt > 0] <= tol[cnt > 0] + 1e-300).all()
    absent = torch.from_numpy(cnt == 0).to(DEV)
    assert torch.equal(acc[absent], start[absent])


def test_embedding_grad_ignores_what_padding_holds():
    print("[case] padding with NaN rows", flush=True)
    ids = torch.tensor([3, -1, 3, 99, 5], device=DEV)
    dout = _rand((5, 24), BF16, 1)
    dout[1] = float("nan")
    dout[3] = float("inf")
    got = mm.embedding_grad(ids, dout, 99)
    assert torch.isfinite(got).all()
    assert torch.equal(got[5], dout[4])
    assert int((got.float().abs().sum(1) > 0).sum()) == 2
    none = mm.embedding_grad(torch.full((5,), -1, device=DEV), dout, 99)
    assert float(none.float().abs().sum()) == 0
    empty = mm.embedding_grad(torch.empty(0, dtype=torch.int64, device=DEV), dout[:0], 99)
    assert empty.shape == (99, 24) and float(empty.float().abs().sum()) == 0
