"""The operators between the embedding and the output layer as a training program runs
them: a step of a small model, other streams, graphs, buffers off the grid, large
tensors."""
import math

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _model(seed, rows=301, width=128, inner=320, layers=2):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    m = {"table": rnd(rows, width), "head": rnd(rows, width) * (2.0 / math.sqrt(width)), "last": 1 + 0.2 * rnd(width)}
    for k in range(layers):
        m[f"gain{k}"] = 1 + 0.2 * rnd(width)
        m[f"up{k}"] = rnd(inner, width) / math.sqrt(width)
        m[f"down{k}"] = rnd(width, inner) / math.sqrt(inner)
    return {k: v.to(DEV) for k, v in m.items()}, layers


def _batch(seed, shape=(3, 50), rows=301):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    ids, tgt = torch.randint(0, rows, shape, generator=g), torch.randint(0, rows, shape, generator=g)
    tgt[0, 3::7] = -100
    return ids.to(DEV), tgt.to(DEV)


def _gradients(m, layers, ids, tgt):
    """Loss and gradients of a residual model (h += down tanh(up norm(h))) through the
    library; the products with the weights by torch, in fp32.  Of the forward pass each
    layer keeps its normalised rows and its inner activation in 8 bits."""
    stream = mm.embedding(m["table"], ids)                               # fp32
    delta, kept = None, []
    for k in range(layers):
        if delta is None:
            r = mm.rms_norm(stream, m[f"gain{k}"], pack="normalized", out_dtype=BF16)
        else:
            r = mm.rms_norm(delta, m[f"gain{k}"], residual=stream, h=stream, pack="normalized", out_dtype=BF16)
        a = torch.tanh(r.y.float() @ m[f"up{k}"].t()).bfloat16()
        kept.append((r.rstd, r.packed, mm.mx_pack(a), a))
        delta = (a.float() @ m[f"down{k}"].t()).bfloat16()
    last = mm.rms_norm(delta, m["last"], residual=stream, h=stream, pack="normalized", out_dtype=BF16)
    head = m["head"].bfloat16()
    loss, _, dy, dw = mm.cross_entropy(last.y, head, tgt, dw_dtype=F32)
    grads = {"head": dw}
    dh, grads["last"] = mm.rms_norm_grad(dy, last.packed, last.rstd, m["last"], out_dtype=F32)
    for k in reversed(range(layers)):
        rstd, xn, a8, a = kept[k]
        dout = dh.bfloat16()                                             # the layer's result is added to the stream
        grads[f"down{k}"] = mm.weight_grad(dout, a8, out_dtype=F32)
        dz = ((dh @ m[f"down{k}"]) * (1 - a.float().square())).bfloat16()
        grads[f"up{k}"] = mm.weight_grad(dz, xn, gain=m[f"gain{k}"], out_dtype=F32)
        dy = dz.float() @ m[f"up{k}"]
        dh, grads[f"gain{k}"] = mm.rms_norm_grad(dy, xn, rstd, m[f"gain{k}"], dres=dh, out=dh)
    grads["table"] = mm.embedding_grad(ids, dh, m["table"].shape[0])
    return loss, grads


def _reference(m, layers, ids, tgt):
    p = {k: v.double().cpu().requires_grad_(True) for k, v in m.items()}
    norm = lambda h, g: h * (h.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * g  # noqa: E731
    h = p["table"][ids.cpu()]
    for k in range(layers):
        h = h + torch.tanh(norm(h, p[f"gain{k}"]) @ p[f"up{k}"].t()) @ p[f"down{k}"].t()
    logits = norm(h, p["last"]) @ p["head"].t()
    loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), tgt.cpu().flatten(), ignore_index=-100)
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


def test_training_step():
    print("[case] a training step with kept activations", flush=True)
    (m, layers), (ids, tgt) = _model(1), _batch(2)
    loss, grads = _gradients(m, layers, ids, tgt)
    want_loss, want = _reference(m, layers, ids, tgt)
    # the forward pass rounds to bf16 (2^-8 of a value, four times a layer)
    assert abs(float(loss) - want_loss) <= 2.0 ** -5 * want_loss
    for k in grads:
        err = float((grads[k].double().cpu() - want[k]).norm() / want[k].norm())
        print(k, err, flush=True)
        # an activation in 8 bits is at most 2^-4 of itself off; such errors of either sign in
        # sums of 150 products stay below that, with the bf16 roundings of the rest
        assert err <= 2.0 ** -4, (k, err)
    # clipped, and stepped on
    names = list(m)
    total, coef, _ = mm.grad_norm([grads[k] for k in names], max_norm=0.1)
    assert 0 < float(coef) < 1
    hidden = [k for k in names if k.startswith(("up", "down"))]
    before = {k: m[k].clone() for k in names}
    rho = [float(m[k].norm()) for k in hidden]
    mm.muonh_step([m[k] for k in hidden], [grads[k] for k in hidden], [torch.zeros_like(m[k]) for k in hidden], 0.02, 0.95, 5,
                  rho=rho, ns_dtype="f32", grad_scale=coef)
    for k, r in zip(hidden, rho):
        assert not torch.equal(m[k], before[k]) and abs(float(m[k].norm()) / r - 1) <= 1e-5
    assert torch.isfinite(_gradients(m, layers, ids, tgt)[0])


def _all(t):
    """Every operator of one layer; the buffers are the caller's."""
    r = mm.rms_norm(t["x"], t["gain"], residual=t["res"], pack="normalized")
    o = mm.rms_norm(t["x"], t["gain"], pack="output", output=False)
    dx, dg = mm.rms_norm_grad(t["dy"], r.packed, r.rstd, t["gain"], dres=t["res"])
    dx2, dg2 = mm.rms_norm_grad(t["dy"], r.h, r.rstd, t["gain"])
    p = mm.mx_pack(t["x"])
    out = [r.y, r.h, r.rstd, *r.packed, o.rstd, *o.packed, dx, dg, dx2, dg2, *p, mm.mx_unpack(p)]
    out += [mm.weight_grad(t["dz"], r.packed, gain=t["gain"]), mm.weight_grad(t["dz"], p, out_dtype=F32)]
    return [v.view(torch.uint8) if v.dtype.itemsize == 1 else v for v in out]


def _tensors(seed, n, width, rows):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return {"x": rnd(n, width).bfloat16(), "res": rnd(n, width), "gain": 1 + 0.2 * rnd(width), "dy": rnd(n, width).bfloat16(),
            "dz": rnd(n, rows).bfloat16()}


# the last ones: parts of the tokens, the 256 tile with its copy, sums by a second launch
SIZES = [(90, 128, 72), (601, 520, 264), (5000, 96, 64), (1500, 2048, 4104), (1300, 2056, 4101)]


@pytest.mark.parametrize("n,width,rows", SIZES)
def test_other_streams(n, width, rows):
    print(f"[case] streams {n} {width} {rows}", flush=True)
    t = _tensors(n, n, width, rows)
    want = _all(t)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(_all(t))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    r = mm.rms_norm(t["x"], t["gain"], residual=t["res"], pack="normalized", stream=s1)
    s2.wait_stream(s1)
    dx, dg = mm.rms_norm_grad(t["dy"], r.packed, r.rstd, t["gain"], dres=t["res"], stream=s2)
    dw = mm.weight_grad(t["dz"], r.packed, gain=t["gain"], stream=s2)
    p = mm.mx_pack(t["x"], stream=s1)
    u = mm.mx_unpack(p, stream=s1)
    torch.cuda.synchronize()
    for a, b in ((r.y, want[0]), (dx, want[8]), (dg, want[9]), (dw, want[15]), (u, want[14])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,width,rows", SIZES)
def test_graphs(n, width, rows):
    # captured as the first call of these sizes, twice; replayed on new contents of the same
    # buffers, with eager work in between
    print(f"[case] graphs {n} {width} {rows}", flush=True)
    n, rows = n + 1, rows + 8
    t = _tensors(7, n, width, rows)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_all(t))
        graphs.append(g)
    for rep in range(4):
        for k, v in _tensors(30 + rep, n, width, rows).items():
            t[k].copy_(v)
        for g in graphs:
            g.replay()
        eager = _all(t)
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(o, eager):
                assert torch.equal(a, b), rep
    del graphs
    torch.cuda.synchronize()


@pytest.mark.parametrize("width", [40, 41, 775, 2048, 5001])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_norm_off_the_grid(width, k):
    """Buffers off every grid but their elements'; what lies around results stays."""
    print(f"[case] norm off the grid {width} {k}", flush=True)
    lib = mm.load()
    n, here = 19, torch.cuda.current_stream().cuda_stream
    t = _tensors(width, n, width, 8)
    want = mm.rms_norm(t["x"], t["gain"], residual=t["res"], pack="output", out_dtype=BF16)
    norm = mm.rms_norm(t["x"], t["gain"], residual=t["res"], pack="normalized")
    wdx, wdg = mm.rms_norm_grad(t["dy"], norm.packed, norm.rstd, t["gain"], dres=t["res"], out_dtype=F32)
    wdx2, _ = mm.rms_norm_grad(t["dy"], norm.h, norm.rstd, t["gain"], dres=t["res"])

    def off(v):
        b = torch.empty(v.numel() + k, dtype=v.dtype, device=DEV)
        c = b[k:].view(v.shape)
        c.copy_(v)
        return c

    def guard(shape, dtype):
        b = torch.full((math.prod(shape) + k + 40,), 7, dtype=dtype, device=DEV)
        return b, b[k:k + math.prod(shape)].view(shape)

    def untouched(b, v):
        return bool((b[:k] == 7).all()) and bool((b[k + v.numel():] == 7).all())

    nb = -(-width // 32)
    h, y, rs = guard((n, width), F32), guard((n, width), BF16), guard((n,), F32)
    q, s = guard((n, width), torch.uint8), guard((n, nb), torch.uint8)
    x, res, gain, dy = off(t["x"]), off(t["res"]), off(t["gain"]), off(t["dy"])
    assert lib.muonh_rms_norm(x.data_ptr(), 1, res.data_ptr(), 0, gain.data_ptr(), 1e-6, n, width, h[1].data_ptr(),
                              y[1].data_ptr(), 1, rs[1].data_ptr(), q[1].data_ptr(), s[1].data_ptr(), 1, here) == 0
    for (b, v), w in ((h, want.h), (y, want.y), (rs, want.rstd), (q, want.packed.q.view(torch.uint8)), (s, want.packed.scales.view(torch.uint8))):
        assert torch.equal(v, w) and untouched(b, v)
    hin = off(norm.h)  # held: its memory is read below
    q8, s8, rstd = off(norm.packed.q.view(torch.uint8)), off(norm.packed.scales.view(torch.uint8)), off(norm.rstd)
    size = lib.muonh_rms_norm_grad_workspace(n, width)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    for kept, w in (((None, q8.data_ptr(), s8.data_ptr()), wdx), ((hin.data_ptr(), None, None), wdx2)):
        dx, dg = guard((n, width), F32), guard((width,), F32)
        assert lib.muonh_rms_norm_grad(dy.data_ptr(), 1, *kept, rstd.data_ptr(), gain.data_ptr(), res.data_ptr(), 0, n, width,
                                       dx[1].data_ptr(), dg[1].data_ptr(), 0, ws.data_ptr(), size, here) == 0
        torch.cuda.synchronize()
        assert torch.equal(dx[1], w) and untouched(*dx) and untouched(*dg)
        if kept[0] is None:
            assert torch.equal(dg[1], wdg)


def test_large_offsets():
    """More than 2^31 values."""
    print("[case] norm, more than 2^31 values", flush=True)
    n, width = 140000, 16384
    x = torch.ones(n, width, dtype=BF16, device=DEV)
    tail = torch.randn(5, width, device=DEV).bfloat16()
    x[-5:] = tail
    gain = torch.rand(width, device=DEV) + 0.5
    want = mm.rms_norm(tail, gain, pack="normalized")
    r = mm.rms_norm(x, gain, pack="normalized", output=False)
    assert torch.equal(r.rstd[-5:], want.rstd)
    assert torch.equal(r.packed.q[-5:].view(torch.uint8), want.packed.q.view(torch.uint8))
    assert torch.equal(r.packed.scales[-5:].view(torch.uint8), want.packed.scales.view(torch.uint8))
    dres = x.clone()
    wdx, _ = mm.rms_norm_grad(tail, want.packed, want.rstd, gain, dres=tail)
    dx, dg = mm.rms_norm_grad(x, r.packed, r.rstd, gain, dres=dres, out=dres)
    assert dx is dres and torch.equal(dx[-5:], wdx)
    v = mm.mx_unpack(want.packed, out_dtype=F32).double()
    one = mm.mx_unpack(type(r.packed)(r.packed.q[:1], r.packed.scales[:1]), out_dtype=F32).double()
    exact = (tail.double() * v).sum(0) + (n - 5) * one[0]
    size = (tail.double() * v).abs().sum(0) + (n - 5) * one[0].abs()
    assert bool(((dg.double() - exact).abs() <= (n / 256 + 80) * U * size).all())
