"""Activations in 8 bits, bit for bit against the format's definition."""
import math

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def oracle(x):
    """(values, scale bytes) in fp64: the least power of two with no finite value of a
    block above 448 of it, values to the nearest e4m3, ties to even."""
    v = x.double().cpu()
    n, d = v.shape
    pad = torch.zeros(n, -(-d // 32) * 32, dtype=torch.float64)
    pad[:, :d] = v
    b = pad.view(n, -1, 32)
    fin = torch.where(b.isfinite(), b.abs(), 0.0)
    top = fin.amax(2, keepdim=True)
    e = torch.full_like(top, -117.0)
    for k in range(-117, 121):  # the largest k still too small decides
        e = torch.where(top > 448 * 2.0 ** k, float(k + 1), e)
    t = b / 2.0 ** e
    mag = t.abs().nan_to_num(nan=0.0, posinf=0.0)
    unit = 2.0 ** (torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    q = torch.where(b.isfinite(), torch.round(t / unit) * unit, math.nan)  # torch.round: ties to even
    return (q * 2.0 ** e).view(n, -1)[:, :d], (e[:, :, 0] + 127).to(torch.uint8)


def check(x):
    p = mm.mx_pack(x.to(DEV))
    want, scales = oracle(x)
    assert torch.equal(p.scales.cpu().view(torch.uint8), scales)
    f = scales.double().sub(127).exp2().repeat_interleave(32, 1)[:, :x.shape[1]]
    got = p.q.cpu().to(F32).double() * f
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    for t in (F32, BF16):
        back = mm.mx_unpack(p, out_dtype=t)
        # exact; from 1.9375 * 2^127 on a value's nearest e4m3 is 2^128, beyond both types
        same = back.double().cpu() == torch.where(want.abs() >= 2.0 ** 128, want.sign() * math.inf, want)
        assert back.dtype == t and bool((same | want.isnan()).all())
        assert torch.equal(back.isnan().cpu(), want.isnan())
    return p


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,width", [(1, 1), (3, 7), (2, 8), (5, 31), (5, 32), (4, 33), (70, 96), (9, 331), (130, 1000),
                                     (3, 2048), (2, 2080), (7, 4099), (1, 14336)])
def test_round_trip(n, width, dtype):
    print(f"[case] 8 bits {n} x {width} {dtype}", flush=True)
    g = torch.Generator(device="cpu")
    g.manual_seed(n * 1000 + width)
    x = torch.randn(n, width, generator=g) * torch.exp2(torch.randint(-12, 12, (n, 1), generator=g).float())
    x[:, width // 2] *= 1000.0
    p = check(x.to(dtype))
    # what was read back is kept as it is
    again = mm.mx_pack(mm.mx_unpack(p, out_dtype=dtype))
    assert torch.equal(mm.mx_unpack(again), mm.mx_unpack(p))


def test_every_code_and_tie():
    print("[case] 8 bits, every code", flush=True)
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    grid = codes[codes.isfinite()].sort().values.unique()
    mid = (grid[1:] + grid[:-1]) / 2  # exact in fp32
    rows = []
    for v in torch.cat([grid, mid, torch.nextafter(mid, torch.tensor(math.inf)), torch.nextafter(mid, torch.tensor(-math.inf))]):
        row = torch.zeros(32)
        row[0], row[1] = 448.0, v  # the block's scale is 1
        rows.append(row)
    check(torch.stack(rows))


def test_scale_borders_and_extremes():
    print("[case] 8 bits, borders", flush=True)
    edge = torch.tensor(448.0)
    rows = [torch.full((40,), float(v)) for v in (0.0, 1.0, edge, torch.nextafter(edge, torch.tensor(math.inf)),
            torch.nextafter(edge, torch.tensor(0.0)), 3.4e38, 1.1754944e-38, 1e-45, 2.0 ** -117 * 448, 2.0 ** -126, 2.0 ** 127)]
    special = torch.randn(40)
    special[3], special[4], special[35] = math.nan, math.inf, -math.inf
    only = torch.full((40,), math.nan)
    inf = torch.full((40,), -math.inf)
    check(torch.stack(rows + [special, only, inf, -rows[5]]))
    check(torch.stack([special, only, inf]).bfloat16())


def test_foreign_scales():
    """Every scale byte is read, also those that are not written."""
    print("[case] 8 bits, every scale", flush=True)
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    got = mm.mx_unpack((q.to(DEV).view(torch.float8_e4m3fn), s.to(DEV).view(torch.float8_e8m0fnu)), out_dtype=F32).cpu()
    want = (q.view(torch.float8_e4m3fn).double() * 2.0 ** (s[:, :1].double() - 127)).float()  # one rounding
    want[255] = math.nan
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    got = mm.mx_unpack((q.to(DEV).view(torch.float8_e4m3fn), s.to(DEV).view(torch.float8_e8m0fnu))).cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.float().nan_to_num(nan=0.0), want.bfloat16().float().nan_to_num(nan=0.0))


def test_shapes_buffers_and_alignment():
    print("[case] 8 bits, shapes", flush=True)
    x = torch.randn(4, 5, 70, device=DEV)
    p = mm.mx_pack(x)
    assert p.q.shape == x.shape and p.scales.shape == (4, 5, 3)
    out = torch.empty(4, 5, 70, device=DEV)
    assert mm.mx_unpack(p, out=out) is out
    flat = mm.mx_unpack(mm.mx_pack(x.view(20, 70)), out_dtype=F32)
    assert torch.equal(out.view(20, 70), flat)
    assert torch.equal(mm.mx_unpack(mm.mx_pack(x[0, 0])), mm.mx_unpack(p)[0, 0])
    # buffers off every grid; what lies around them stays
    lib = mm.load()
    for off in (1, 3, 6):
        xb = torch.empty(20 * 70 + 4, device=DEV)
        xb[1:1401] = x.view(-1)
        q, s = torch.full((1410,), 99, dtype=torch.uint8, device=DEV), torch.full((70,), 99, dtype=torch.uint8, device=DEV)
        assert lib.muonh_mx_pack(xb.data_ptr() + 4, 0, 20, 70, q.data_ptr() + off, s.data_ptr() + off,
                                 torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(q[off:off + 1400], p.q.view(torch.uint8).view(-1)) and torch.equal(s[off:off + 60], p.scales.view(torch.uint8).view(-1))
        assert bool((q[:off] == 99).all()) and bool((q[off + 1400:] == 99).all())
        assert bool((s[:off] == 99).all()) and bool((s[off + 60:] == 99).all())
        o = torch.full((1408,), 5.0, dtype=BF16, device=DEV)
        assert lib.muonh_mx_unpack(q.data_ptr() + off, s.data_ptr() + off, 20, 70, o.data_ptr() + 2 * off, 1,
                                   torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(o[off:off + 1400], flat.bfloat16().view(-1))
        assert bool((o[:off] == 5).all()) and bool((o[off + 1400:] == 5).all())
    e = mm.mx_pack(torch.zeros(0, 64, device=DEV))
    assert mm.mx_unpack(e).shape == (0, 64)
    with pytest.raises(ValueError):
        mm.mx_unpack((p.q, p.scales[..., :2]))
    with pytest.raises(ValueError):
        mm.mx_unpack((p.q, p.scales.cpu()))
    with pytest.raises(ValueError):
        mm.mx_unpack(p, out=out[:2])
    with pytest.raises(TypeError):
        mm.mx_unpack(p, out=out, out_dtype=BF16)
    with pytest.raises(TypeError):
        mm.mx_unpack(p, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        mm.mx_pack(x.half())
    with pytest.raises(ValueError):
        mm.mx_pack(x.transpose(0, 1))


def test_large_offsets():
    """More than 2^31 values."""
    print("[case] 8 bits, more than 2^31 values", flush=True)
    n, width = 33000, 65600
    x = torch.zeros(n, width, dtype=BF16, device=DEV)
    tail = torch.randn(9, width, device=DEV).bfloat16()
    x[-9:] = tail
    p = mm.mx_pack(x)
    want = mm.mx_pack(tail)
    assert torch.equal(p.q[-9:].view(torch.uint8), want.q.view(torch.uint8))
    assert torch.equal(p.scales[-9:].view(torch.uint8), want.scales.view(torch.uint8))
    assert int(p.q[:-9].view(torch.uint8).amax()) == 0
    del x
    back = mm.mx_unpack(p)
    assert torch.equal(back[-9:], mm.mx_unpack(want)) and float(back[:-9].abs().max()) == 0.0
