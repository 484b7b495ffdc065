"""The norm's 8-bit rows are the e4m3 values nearest to the row in fp64, also where its fp32
form passes below that type's normal range."""
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = float(torch.tensor(1e-6))


def nearest(v):
    """(values, scale bytes) of rows in fp64 whose width is a multiple of 32."""
    b = v.view(v.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-117)
    t = b / torch.exp2(e.double())
    unit = torch.exp2((torch.frexp(t)[1] - 4).clamp(min=-9).double())
    return (torch.round(t / unit) * unit).view_as(v), (e[..., 0] + 127).to(torch.uint8)


def check(x, gain, pack):
    r = mm.rms_norm(x, gain, pack=pack, output=False)
    v = x.double() * (x.double().square().mean(1, keepdim=True) + EPS) ** -0.5
    want, scales = nearest(v * gain.double() if pack == "output" else v)
    assert torch.equal(r.packed.scales.view(torch.uint8), scales)
    assert torch.equal(r.packed.q.double(), want)


@pytest.mark.parametrize("pack", ["normalized", "output"])
@pytest.mark.parametrize("low,high", [(1e-39, 1e3), (1e-40, 1e20), (1e-44, 1e30), (1e-30, 1e-12), (1e-38, 1.0)])
def test_channels_below_the_normal_range(low, high, pack):
    """Blocks of next to nothing beside ordinary ones, and a gain that brings them back:
    the product with rstd has few bits there, its fp32 value is far off."""
    print(f"[case] packed rows, channels of {low} and gains of {high}, {pack}", flush=True)
    n, d = 4000, 1024
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn(n, d, generator=g, device=DEV)
    gain = torch.rand(d, generator=g, device=DEV) + 0.5
    x[:, :d // 2] *= low
    gain[:d // 2] *= high
    check(x, gain, pack)


# a row of c but for one value v, the gain of that column, and where it stands in fp32 and
# in fp64: on either side of 1.9375, where two e4m3 values meet.  rstd, below 2^-126, is 2^-22 off
FAR = [("0x1.ff70f0p+127", "0x1.16bf04p+127", "0x1.c6df46p+1"), ("0x1.fe60aap+127", "0x1.086174p+126", "0x1.de8982p+2"),
       ("0x1.fe60aap+127", "0x1.257292p+127", "0x1.af312ep+1"), ("0x1.ff2e4ep+127", "0x1.01ef02p+126", "0x1.eb44f4p+2"),
       ("0x1.ff2e4ep+127", "0x1.006942p+127", "0x1.ee3b50p+1"), ("0x1.fe102ap+127", "0x1.ff6622p+126", "0x1.ee8606p+1")]


@pytest.mark.parametrize("at", [0, 5, 700])
def test_rows_of_the_largest_values(at):
    print(f"[case] packed rows, the largest values, at {at}", flush=True)
    for c, v, g in FAR:
        x, gain = torch.full((3, 1024), float.fromhex(c), device=DEV), torch.ones(1024, device=DEV)
        x[1, at], gain[at] = float.fromhex(v), float.fromhex(g)
        for pack in ("output", "normalized"):
            check(x, gain, pack)
