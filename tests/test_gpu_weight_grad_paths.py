"""The weight gradient by each of its tiles, told by the scratch memory that they need: 256
tiles all cut into parts, several streams, graphs, every code under every scale."""
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402
from test_gpu_weight_grad import check, inputs  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def up(v, m):
    return -(-v // m) * m


def scratch(dz, n, rows, width):
    return mm.load().muonh_weight_grad_workspace(dz.data_ptr(), n, rows, width)


def parts_of_256(dz, n, rows, width):
    """Bytes of the sums of parts, with 256 tiles; below 0: other tiles (x is not kept in bf16)."""
    copied = 2 * up(rows, 256) * (up(n, 128) + 64) if width >= 8192 else 0
    if not copied and (rows % 8 or dz.data_ptr() % 16):
        copied = 2 * up(n, 64) * up(rows, 8)
    elif not copied:
        copied = 2 * (up(n, 64) - n // 64 * 64) * rows
    return scratch(dz, n, rows, width) - 2 * up(width, 256) * (up(n, 128) + 64) - up(copied, 256)


def tiles_of_256(rows, width):
    return up(rows, 256) // 256 * (up(width, 256) // 256)


# 51 tiles of 256 in parts (dz's last stage copied; all of dz, 8 rows off), 64 in parts, 272 of
# which 16 are in parts, and dz turned as well
PARTS = [(6575, 4176, 750), (6575, 4171, 750), (16384, 2048, 2048), (4099, 4107, 4090), (6150, 2100, 8440)]


def in_parts(dz, n, rows, width):
    tiles = tiles_of_256(rows, width)
    cut = tiles % 256
    sums = parts_of_256(dz, n, rows, width)
    assert sums >= 2 * cut * 4 * 65536 and sums % (cut * 4 * 65536) == 0, sums
    return sums // (cut * 4 * 65536)


@pytest.mark.parametrize("n,rows,width", PARTS[:3])
@pytest.mark.parametrize("out", [BF16, F32])
def test_all_tiles_in_parts(n, rows, width, out):
    print(f"[case] weight gradient, 256 tiles in parts {n} {rows} {width} {out}", flush=True)
    dz, p, gain = inputs(n, rows, width)
    assert 2 <= in_parts(dz, n, rows, width) <= 32
    check(mm.weight_grad(dz, p, gain=gain, scale=0.5, out_dtype=out), dz, p, gain, 0.5)
    base = torch.randn(rows, width, device=DEV).to(out)
    acc = base.clone()
    check(mm.weight_grad(dz, p, out=acc, accumulate=True, scale=-2.0), dz, p, None, -2.0, base)


@pytest.mark.parametrize("n,rows,width", PARTS)
def test_streams(n, rows, width):
    """Several launches a call, their scratch memory from torch's allocator: two streams at once."""
    print(f"[case] weight gradient, streams {n} {rows} {width}", flush=True)
    dz, p, gain = inputs(n, rows, width)
    dz2, p2, gain2 = inputs(n, rows, width, seed=5)
    assert in_parts(dz, n, rows, width) > 1 and in_parts(dz2, n, rows, width) > 1
    want, want2 = mm.weight_grad(dz, p, gain=gain, out_dtype=F32), mm.weight_grad(dz2, p2, gain=gain2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got, got2 = [], []
    for _ in range(4):
        with torch.cuda.stream(s1):
            got.append(mm.weight_grad(dz, p, gain=gain, out_dtype=F32))
        got2.append(mm.weight_grad(dz2, p2, gain=gain2, stream=s2))
    torch.cuda.synchronize()
    for a, b in zip(got, got2):
        assert torch.equal(a, want) and torch.equal(b, want2)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("n,rows,width", PARTS)
def test_graphs(n, rows, width, shared):
    """Captured as the first calls of these sizes, in pools of their own or one together; replayed
    on new contents of the same buffers, with eager work in between."""
    print(f"[case] weight gradient, graphs {n} {rows} {width} {shared}", flush=True)
    n += 2  # other sizes than the eager calls above
    dz, p, gain = inputs(n, rows, width)
    q, s = p
    assert in_parts(dz, n, rows, width) > 1
    total = torch.zeros(rows, width, device=DEV)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if shared and k else None):
            outs.append(mm.weight_grad(dz, (q, s), gain=gain))
            mm.weight_grad(dz, (q, s), gain=gain, out=total, accumulate=True)
        graphs.append(g)
    for rep in range(4):
        dz2, p2, gain2 = inputs(n, rows, width, seed=20 + rep)
        dz.copy_(dz2)
        q.view(torch.uint8).copy_(p2.q.view(torch.uint8))
        s.view(torch.uint8).copy_(p2.scales.view(torch.uint8))
        gain.copy_(gain2)
        total.zero_()
        for g in graphs:
            g.replay()
        eager = mm.weight_grad(dz2, p2, gain=gain2)
        sums = torch.zeros(rows, width, device=DEV)
        for _ in range(2):
            mm.weight_grad(dz2, p2, gain=gain2, out=sums, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(total, sums), rep
        for o in outs:
            assert torch.equal(o, eager), rep
    del graphs
    torch.cuda.synchronize()


# one launch of 64 tiles; of 128 tiles, as those of 64 would be more than 64 on each unit; of 256
@pytest.mark.parametrize("n,rows,width,tile", [(300, 130, 700, 64), (200, 8200, 8200, 128), (6575, 4176, 750, 256),
                                               (2100, 4096, 8192, 256)])
def test_every_code_and_scale_by_itself(n, rows, width, tile):
    """One token of the n holds every code under one scale byte and has a gradient of ones, the
    others hold zeros: each row of the result is that token, NaN and infinity among its values."""
    print(f"[case] weight gradient, every code under every scale {n} {rows} {width}", flush=True)
    q, s = torch.zeros(n, width, dtype=torch.uint8, device=DEV), torch.full((n, -(-width // 32)), 127, dtype=torch.uint8, device=DEV)
    dz = torch.zeros(n, rows, dtype=BF16, device=DEV)
    codes = (torch.arange(width, device=DEV) % 256).to(torch.uint8)
    p = (q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu))
    large = parts_of_256(dz, n, rows, width) >= 0
    assert large == (tile == 256)
    if tile == 128:
        assert up(rows, 64) // 64 * (up(width, 64) // 64) > 64 * 256
    out = torch.empty(rows, width, device=DEV)
    finite = 0
    for t in range(256):
        at = (t * 37 + 5) % n
        q[at], s[at], dz[at] = codes, t, 1.0
        want = mm.mx_unpack((p[0][at:at + 1], p[1][at:at + 1])).float()  # rounded to bf16
        mm.weight_grad(dz, p, out=out)
        assert torch.equal(out.isnan(), want.isnan().expand(rows, -1)), t
        low = (want.abs() < 2.0 ** -126)[0]  # the matrix cores may take such operands as zero
        same = (out == want).all(0) | want.isnan()[0]
        assert bool((same | low).all()), t
        assert bool((out[:, low].abs() <= 2.0 ** -126).all()), t
        finite += int(want.isfinite().sum())
        q[at], s[at], dz[at] = 0, 127, 0.0
    # 254 of 256 codes are numbers, scales up to 246 give finite ones alone
    assert finite >= 247 * (width // 256 * 254)
