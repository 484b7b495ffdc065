"""What the operators between the embedding and the output layer are handed in other ways
than a program's own tuple of tensors."""
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


class Fetched:
    """A pair that makes its tensors on access and keeps none, as one brought back from
    elsewhere would."""

    def __init__(self, packed):
        self.kept = packed

    def __len__(self):
        return 2

    def __getitem__(self, k):
        if k > 1:
            raise IndexError(k)
        return self.kept[k].clone()


# rows by columns in one launch; partial sums of 2.4 MB and more beside 8-bit rows of as much
@pytest.mark.parametrize("n,width", [(300, 1100), (3100, 768), (8192, 768), (6000, 2048)])
def test_pairs_that_keep_nothing(n, width):
    """Tensors of a pair that nobody else holds last until the call's work is queued: its
    outputs and scratch memory are not allocated over them."""
    print(f"[case] pairs that keep nothing {n} {width}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(n + width)
    x = torch.randn(n, width, generator=g, device=DEV)
    dy = torch.randn(n, width, generator=g, device=DEV).bfloat16()
    dz = torch.randn(n, 200, generator=g, device=DEV).bfloat16()
    gain = torch.rand(width, generator=g, device=DEV) + 0.5
    r = mm.rms_norm(x, gain, pack="normalized", output=False)
    want = mm.rms_norm_grad(dy, r.packed, r.rstd, gain, out_dtype=F32)
    dw, back = mm.weight_grad(dz, r.packed), mm.mx_unpack(r.packed)
    for _ in range(3):
        for pair in (lambda: Fetched(r.packed), lambda: (t.clone() for t in r.packed), lambda: [t.clone() for t in r.packed]):
            dx, dgain = mm.rms_norm_grad(dy, pair(), r.rstd, gain, out_dtype=F32)
            assert torch.equal(dx, want[0]) and torch.equal(dgain, want[1])
            assert torch.equal(mm.weight_grad(dz, pair()), dw)
        assert torch.equal(mm.mx_unpack(Fetched(r.packed)), back)
        del dx, dgain
    with pytest.raises(ValueError, match="pair"):
        mm.rms_norm_grad(dy, iter(r.packed[:1]), r.rstd, gain)


def test_no_tokens_clear_the_gradient():
    """Without a token there is nothing that a gain could scale, whatever it holds."""
    print("[case] weight gradient of no tokens", flush=True)
    gain = torch.ones(64, device=DEV)
    gain[3], gain[7], gain[40] = float("inf"), float("nan"), -float("inf")
    none = mm.mx_pack(torch.zeros(0, 64, device=DEV))
    for rows in (16, 2000):
        out = torch.full((rows, 64), 5.0, device=DEV)
        assert mm.weight_grad(torch.zeros(0, rows, device=DEV, dtype=BF16), none, gain=gain, scale=-2.0, out=out) is out
        assert torch.equal(out.view(torch.int32), torch.zeros(rows, 64, device=DEV, dtype=torch.int32))
        assert bool((mm.weight_grad(torch.zeros(0, rows, device=DEV, dtype=BF16), none, gain=gain) == 0).all())


class FetchedList:
    """Gradients that are made on access and not kept."""

    def __init__(self, tensors):
        self.kept = tensors

    def __len__(self):
        return len(self.kept)

    def __getitem__(self, k):
        return self.kept[k].clone()


def test_gradients_that_nobody_keeps():
    """The norm's scratch memory and results are not allocated over gradients still to be read."""
    print("[case] gradients that nobody keeps", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    for sizes in ([40], [130, 7, 4096], [2000] * 60, [3 << 20, 5, 1 << 20]):
        ts = [torch.randn(s, generator=g, device=DEV).to(BF16 if k % 2 else F32) for k, s in enumerate(sizes)]
        want = mm.grad_norm(ts, max_norm=0.5)
        outs = [torch.empty_like(t) for t in ts]
        mm.clip_grads(ts, 0.5, outputs=outs)
        for _ in range(3):
            for given in (FetchedList(ts), (t.clone() for t in ts)):
                got = mm.grad_norm(given, max_norm=0.5)
                assert all(torch.equal(a, b) for a, b in zip(got, want))
            into = [torch.zeros_like(t) for t in ts]
            total, coef = mm.clip_grads(FetchedList(ts), 0.5, outputs=into)
            assert torch.equal(total, want[0]) and torch.equal(coef, want[1])
            assert all(torch.equal(a, b) for a, b in zip(into, outs))
            del got, into
