"""The gradient of a weight from activations in 8 bits, against fp64."""
import math

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: U}


def inputs(n, rows, width, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 7 * n + 11 * rows + width)
    dz = torch.randn(n, rows, generator=g, device=DEV).bfloat16()
    x = torch.randn(n, width, generator=g, device=DEV) * torch.exp(torch.randn(width, generator=g, device=DEV))
    return dz, mm.mx_pack(x), 1 + 0.3 * torch.randn(width, generator=g, device=DEV)


def check(dw, dz, p, gain=None, scale=1.0, base=None):
    x = mm.mx_unpack(p, out_dtype=F32).double()
    d = dz.double()
    f = 1.0 if gain is None else gain.double()
    want = scale * f * (d.t() @ x)
    size = abs(scale) * (1.0 if gain is None else f.abs()) * (d.abs().t() @ x.abs())
    n = dz.shape[0]
    # products are exact; each addition in the matrix cores at most a whole step of fp32
    # (n of them and the parts'), the factor's two roundings, then the result
    bound = 2 * U * (n + 64) * size + 3 * U * want.abs()
    if base is not None:
        want = want + base.double()
    bound = bound + (HALF[dw.dtype] + U) * want.abs() + 2.0 ** -133
    off = (dw.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    # and on the whole far below it: rounding errors do not add up in one direction
    rel = float((dw.double() - want).norm() / want.norm().clamp(min=1e-300))
    assert rel <= (2.0 ** -8 if dw.dtype == BF16 else 2 * U * math.sqrt(n + 64) * 8), rel


SIZES = [(1, 1, 1), (1, 8, 32), (2, 3, 5), (17, 64, 64), (63, 40, 33), (64, 128, 256), (65, 257, 255), (100, 300, 72),
         (128, 8, 1000), (500, 1003, 517), (777, 256, 2048), (1024, 768, 768), (1, 1000, 2000), (3000, 64, 96), (4096, 2304, 768)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("n,rows,width", SIZES)
def test_weight_grad(n, rows, width, out):
    print(f"[case] weight gradient {n} {rows} {width} {out}", flush=True)
    dz, p, gain = inputs(n, rows, width)
    dw = mm.weight_grad(dz, p, gain=gain, scale=0.5, out_dtype=out)
    assert dw.shape == (rows, width) and dw.dtype == out
    check(dw, dz, p, gain, 0.5)
    check(mm.weight_grad(dz, p, out_dtype=out), dz, p)
    base = torch.randn(rows, width, device=DEV).to(out)
    acc = base.clone()
    assert mm.weight_grad(dz, p, gain=gain, out=acc, accumulate=True) is acc
    check(acc, dz, p, gain, 1.0, base)
    assert torch.equal(mm.weight_grad(dz, p, gain=gain, scale=0.5, out_dtype=out), dw)


def test_larger():
    print("[case] weight gradient, several rounds", flush=True)
    for n, rows, width in ((2000, 5000, 4100), (8192, 1024, 4096)):
        dz, p, gain = inputs(n, rows, width)
        check(mm.weight_grad(dz, p, gain=gain, out_dtype=F32), dz, p, gain)


@pytest.mark.parametrize("n,rows,off", [(4100, 4093, 0), (4100, 4096, 1), (4096, 4096, 0)])
def test_large_tiles_and_copies(n, rows, off):
    """Sizes that 256 x 256 tiles take, with dz off the 16-byte grid (copied whole), and with
    its last stage alone."""
    print(f"[case] weight gradient, 256 tiles {n} {rows} {off}", flush=True)
    width = 4096
    dz, p, gain = inputs(n, rows, width)
    z = torch.zeros(n * rows + 8, dtype=BF16, device=DEV)
    z[off:off + n * rows] = dz.view(-1)
    dz = z[off:off + n * rows].view(n, rows)
    size = mm.load().muonh_weight_grad_workspace(dz.data_ptr(), n, rows, width)
    copied = n if rows % 8 or off else n % 64
    assert 2 * width * n + 2 * copied * rows <= size <= 2 * width * (n + 192) + 2 * (copied + 64) * (rows + 8) + 1024
    check(mm.weight_grad(dz, p, gain=gain, out_dtype=F32), dz, p, gain)
    base = torch.randn(rows, width, device=DEV).bfloat16()
    acc = base.clone()
    check(mm.weight_grad(dz, p, out=acc, accumulate=True, scale=-2.0), dz, p, None, -2.0, base)


@pytest.mark.parametrize("n,rows,width,off", [(2100, 4096, 8192, 0), (2049, 4001, 8192, 0), (2176, 4041, 16377, 1)])
def test_wide(n, rows, width, off):
    """Sizes whose dz is brought along the tokens as well."""
    print(f"[case] weight gradient, wide {n} {rows} {width} {off}", flush=True)
    dz, p, gain = inputs(n, rows, width)
    z = torch.zeros(n * rows + 8, dtype=BF16, device=DEV)
    z[off:off + n * rows] = dz.view(-1)
    dz = z[off:off + n * rows].view(n, rows)
    size = mm.load().muonh_weight_grad_workspace(dz.data_ptr(), n, rows, width)
    assert size >= 2 * n * (rows + width)
    check(mm.weight_grad(dz, p, gain=gain, out_dtype=F32), dz, p, gain)
    base = torch.randn(rows, width, device=DEV).bfloat16()
    acc = base.clone()
    check(mm.weight_grad(dz, p, out=acc, accumulate=True, scale=-2.0), dz, p, None, -2.0, base)


@pytest.mark.parametrize("n,rows,width", [(4099, 4107, 4090), (4160, 4104, 4096), (6150, 2100, 8440)])
def test_tiles_left_over(n, rows, width):
    """Sizes of 272 or 297 tiles: those behind the first 256 are cut into parts."""
    print(f"[case] weight gradient, tiles left over {n} {rows} {width}", flush=True)
    dz, p, gain = inputs(n, rows, width)
    left = (rows + 255) // 256 * ((width + 255) // 256) - 256
    parts = mm.load().muonh_weight_grad_workspace(dz.data_ptr(), n, rows, width) - 2 * width * n
    parts -= 2 * n * rows if rows % 8 or width >= 8192 else 2 * (n % 64) * rows
    assert 0 < left <= 41 and parts >= 2 * left * 4 * 65536
    check(mm.weight_grad(dz, p, gain=gain, out_dtype=F32), dz, p, gain)
    base = torch.randn(rows, width, device=DEV).bfloat16()
    acc = base.clone()
    check(mm.weight_grad(dz, p, out=acc, accumulate=True, scale=-2.0), dz, p, None, -2.0, base)


def test_of_the_norm():
    """From what the norm kept: the gradient behind its output."""
    print("[case] weight gradient behind the norm", flush=True)
    g = torch.Generator(device="cpu")
    g.manual_seed(4)
    x, gain = torch.randn(3, 50, 200, generator=g).to(DEV), (1 + 0.2 * torch.randn(200, generator=g)).to(DEV)
    dz = torch.randn(3, 50, 96, generator=g).bfloat16().to(DEV)
    r = mm.rms_norm(x, gain, pack="normalized")
    dw = mm.weight_grad(dz, r.packed, gain=gain, out_dtype=F32)
    want = dz.view(150, 96).double().t() @ r.y.view(150, 200).double()
    # 2^-4 of each value at most, in any direction: on the whole about 2^-4 / sqrt(3) of half of them
    assert float((dw.double() - want).norm() / want.norm()) <= 2.0 ** -4
    kept = mm.mx_unpack(r.packed, out_dtype=F32).double() * gain.double()
    got = (dw.double() - dz.view(150, 96).double().t() @ kept.view(150, 200)).abs()
    assert bool((got <= 2 * U * 220 * (dz.view(150, 96).double().abs().t() @ kept.view(150, 200).abs())).all())


def test_what_is_not_finite_stays_where_it_is():
    print("[case] weight gradient, not finite", flush=True)
    for n, rows, width in ((70, 40, 64), (70, 41, 64), (200, 300, 300)):
        dz, p, _ = inputs(n, rows, width)
        want = mm.weight_grad(dz, p, out_dtype=F32)
        bad, q = dz.clone(), p.q.clone()
        bad[n - 1, 5], bad[0, 8] = math.inf, math.nan
        q.view(torch.uint8)[n - 1, 9] = 0x7f
        got = mm.weight_grad(bad, (q, p.scales), out_dtype=F32)
        rows_bad, cols_bad = [5, 8], [9]
        keep_r = [k for k in range(rows) if k not in rows_bad]
        keep_c = [k for k in range(width) if k not in cols_bad]
        assert torch.equal(got[keep_r][:, keep_c], want[keep_r][:, keep_c])
        assert bool(got[8].isnan().all()) and bool(got[:, 9].isnan().all())
        assert not bool(got[5].isfinite().any())


def test_buffers_off_the_grid():
    print("[case] weight gradient, off the grid", flush=True)
    lib = mm.load()
    n, rows, width = 90, 72, 80
    dz, p, gain = inputs(n, rows, width)
    want = mm.weight_grad(dz, p, gain=gain)
    for off in (1, 2, 5):
        z = torch.zeros(n * rows + 8, dtype=BF16, device=DEV)
        z[off:off + n * rows] = dz.view(-1)
        q, s = (torch.zeros(t.numel() + 8, dtype=torch.uint8, device=DEV) for t in p)
        q[off:off + n * width] = p.q.view(torch.uint8).view(-1)
        s[off:off + 3 * n] = p.scales.view(torch.uint8).view(-1)
        o = torch.full((rows * width + 16,), 3.0, dtype=BF16, device=DEV)
        size = lib.muonh_weight_grad_workspace(z.data_ptr() + 2 * off, n, rows, width)
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)  # NaN, whatever it is read as
        assert lib.muonh_weight_grad(z.data_ptr() + 2 * off, q.data_ptr() + off, s.data_ptr() + off, gain.data_ptr(), 1.0, n,
                                     rows, width, o.data_ptr() + 2 * off, 1, 0, ws.data_ptr(), size,
                                     torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(o[off:off + rows * width].view(rows, width), want)
        assert bool((o[:off] == 3).all()) and bool((o[off + rows * width:] == 3).all())


def test_empty_and_refused():
    print("[case] weight gradient, empty and refused", flush=True)
    dz, p, gain = inputs(6, 16, 64)
    e = (p.q[:0], p.scales[:0])
    assert bool((mm.weight_grad(dz[:0], e, gain=gain) == 0).all())
    base = torch.ones(16, 64, device=DEV)
    assert bool((mm.weight_grad(dz[:0], e, out=base, accumulate=True) == 1).all())
    assert bool((mm.weight_grad(dz[:0], e, out=base) == 0).all())
    for args, kw in (((dz.float(), p), {}), ((dz[:5], p), {}), ((dz, p), dict(gain=gain[:3])), ((dz, p), dict(accumulate=True)),
                     ((dz, p), dict(out=base[:4])), ((dz, p), dict(out=base, out_dtype=BF16)), ((dz, p), dict(out_dtype=torch.float16)),
                     ((dz, (p.q, p.scales[:, :1])), {}), ((dz, (p.q.cpu(), p.scales)), {}), ((dz.t(), p), {}),
                     ((dz, p), dict(scale=math.nan))):
        with pytest.raises((ValueError, TypeError, mm.MuonhError)):
            mm.weight_grad(*args, **kw)


def test_large_offsets():
    """More than 2^31 values of dz."""
    print("[case] weight gradient, more than 2^31 values", flush=True)
    n, rows, width = 150000, 14400, 40
    dz = torch.zeros(n, rows, dtype=BF16, device=DEV)
    x = torch.randn(n, width, device=DEV)
    dz[-70:] = torch.randn(70, rows, device=DEV).bfloat16()
    dz[:3] = 1.0
    p = mm.mx_pack(x)
    dw = mm.weight_grad(dz, p, out_dtype=F32)
    rowsel = list(range(3)) + list(range(n - 70, n))
    v = mm.mx_unpack(p, out_dtype=F32)[rowsel].double()
    d = dz[rowsel].double()
    want, size = d.t() @ v, d.abs().t() @ v.abs()
    assert bool(((dw.double() - want).abs() <= 2 * U * 200 * size + U * want.abs()).all())


@pytest.mark.parametrize("n", [256, 300])
def test_every_code_and_scale(n):
    """dz of ones at (t, t): dw is x, for every code under every scale byte."""
    print(f"[case] weight gradient, every code and scale {n}", flush=True)
    q = torch.zeros(n, 256, dtype=torch.uint8)
    q[:256] = torch.arange(256, dtype=torch.uint8)
    s = torch.full((n, 8), 127, dtype=torch.uint8)
    s[:256] = torch.arange(256, dtype=torch.uint8)[:, None]
    p = (q.to(DEV).view(torch.float8_e4m3fn), s.to(DEV).view(torch.float8_e8m0fnu))
    want = mm.mx_unpack(p).float()  # rounded to bf16
    for t in range(0, 256, 64):  # 64 tokens at a time, so that no NaN or infinity of another token is in the sum
        one = (p[0][t:t + 64].contiguous(), p[1][t:t + 64].contiguous())
        for rows in (64, 130):
            for k in range(0, 64, 16):
                dz = torch.zeros(64, rows, dtype=BF16, device=DEV)
                dz[k, 0] = 1.0
                got = mm.weight_grad(dz, one, out_dtype=F32)[0]
                finite = want[t:t + 64].isfinite().all(0)
                assert torch.equal(got[finite], want[t + k][finite])
    # a token alone, NaN and infinity among its values
    for t in list(range(0, 256, 15)) + [254, 255]:
        one = (p[0][t:t + 1].contiguous(), p[1][t:t + 1].contiguous())
        got = mm.weight_grad(torch.ones(1, 1, dtype=BF16, device=DEV), one, out_dtype=F32)[0]
        assert torch.equal(got.isnan(), want[t].isnan())
        low = want[t].abs() < 2.0 ** -126  # the matrix cores may take such operands as zero
        assert torch.equal(got.nan_to_num(nan=0.0)[~low], want[t].nan_to_num(nan=0.0)[~low])
        assert bool((got[low].abs() <= 2.0 ** -126).all())
