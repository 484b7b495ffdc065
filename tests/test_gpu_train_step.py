"""The operators around the step together, and under what a training program does
to them: other streams, graphs, large tensors, buffers off the grid."""
import math

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def _model(seed, rows=301, width=128):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(table=(rnd(rows, width) * 0.5).to(DEV), hidden=(rnd(width, width) / math.sqrt(width)).to(DEV),
                head=(rnd(rows, width) * (2.0 / math.sqrt(width))).to(DEV))


def _batch(seed, n=90, rows=301):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    ids, tgt = torch.randint(0, rows, (n,), generator=g), torch.randint(0, rows, (n,), generator=g)
    ids[5::13] = -100
    tgt[3::7] = -100
    return ids.to(DEV), tgt.to(DEV)


def _gradients(m, ids, tgt, scale):
    """Loss and gradients of head(hidden(embedding)) through the library (the
    hidden product by torch in fp32)."""
    e = mm.embedding(m["table"], ids, scale=scale)                      # fp32
    h = (e @ m["hidden"]).bfloat16()
    w = m["head"].bfloat16()
    loss, _, dh, dw = mm.cross_entropy(h, w, tgt, dw_dtype=F32)
    dhid = e.t().contiguous() @ dh.float()
    de = dh.float() @ m["hidden"].t().contiguous()
    dtab = mm.embedding_grad(ids, de, m["table"].shape[0], scale=scale)
    return loss, dict(table=dtab, hidden=dhid, head=dw)


def _reference(m, ids, tgt, scale):
    """The same in fp64 by autograd on the CPU, with the roundings of h and w to
    bf16 that the call's operands have (gradients pass through them)."""
    p = {k: v.double().cpu().requires_grad_(True) for k, v in m.items()}
    ids, tgt = ids.cpu(), tgt.cpu()
    ok = (ids >= 0)
    e = torch.where(ok[:, None], p["table"][torch.where(ok, ids, 0)] * scale, 0.0)
    rnd = lambda t: t + (t.detach().float().bfloat16().double() - t.detach())  # noqa: E731
    logits = rnd(e @ p["hidden"]) @ rnd(p["head"]).t()
    loss = torch.nn.functional.cross_entropy(logits, tgt, ignore_index=-100)
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


def test_training_step():
    print("[case] a training step", flush=True)
    m, (ids, tgt) = _model(1), _batch(2)
    scale = 3.0
    loss, grads = _gradients(m, ids, tgt, scale)
    want_loss, want = _reference(m, ids, tgt, scale)
    # h is formed in fp32 here and in fp64 there: a value next to a tie may round
    # the other way, 2^-7 of one value in some hundred; and P carries 2^-8
    assert abs(float(loss) - float(want_loss)) <= 2e-3 * float(want_loss)
    for k in grads:
        err = (grads[k].double().cpu() - want[k]).norm() / want[k].norm()
        assert float(err) <= 2.0 ** -7, (k, float(err))
    order = ["table", "hidden", "head"]
    total, coef, norms = mm.grad_norm([grads[k] for k in order], max_norm=0.05)
    assert torch.allclose(total, torch.stack([grads[k].norm() for k in order]).norm(), rtol=1e-5)
    assert 0 < float(coef) < 1
    # the clipped step: clipping into buffers and stepping on them, or the
    # coefficient handed to the step
    clipped = [torch.empty_like(grads[k]) for k in order]
    mm.clip_grads([grads[k] for k in order], 0.05, outputs=clipped)
    a, b = {k: m[k].clone() for k in order}, {k: m[k].clone() for k in order}
    za, zb = ({k: (torch.zeros_like(m[k]), torch.zeros_like(m[k])) for k in order} for _ in range(2))
    rho = [float(m["hidden"].norm())]
    for w, z, g, kw in ((a, za, dict(zip(order, clipped)), {}), (b, zb, grads, dict(grad_scale=coef))):
        mm.muonh_step([w["hidden"]], [g["hidden"]], [z["hidden"][0]], 0.02, 0.95, 5, rho=rho, ns_dtype="f32", **kw)
        two = ["table", "head"]
        mm.adamh_step([w[k] for k in two], [g[k] for k in two], [z[k][0] for k in two], [z[k][1] for k in two], eta=1e-3,
                      step=1, hook="none", **kw)
    for k in order:
        assert not torch.equal(a[k], m[k])
        # one fp32 rounding of coef * g apart; Adam's first step turns a gradient
        # into about +-1, its change bounded by the relative one of g (2^-24)
        # except near eps; Newton-Schulz amplifies by at most 3.4445^5
        d = (a[k] - b[k]).norm() / (a[k] - m[k]).norm()
        assert float(d) <= 1e-3, (k, float(d))
    # the loss falls along the step it was computed for
    after, _ = _gradients(b, ids, tgt, scale)
    assert torch.isfinite(after)


def test_accumulated_microbatches_and_tied_tables():
    print("[case] micro-batches", flush=True)
    m = _model(3)
    w = m["table"].bfloat16()
    parts = [_batch(s) for s in (4, 5, 6)]
    g = torch.Generator(device="cpu")
    g.manual_seed(9)
    xs = [torch.randn(90, 128, generator=g).bfloat16().to(DEV) for _ in parts]
    acc = torch.zeros(301, 128, device=DEV)
    each = []
    for x, (ids, tgt) in zip(xs, parts):
        mm.cross_entropy(x, w, tgt, reduction="sum", grad="w", dw=acc, accumulate=True)
        each.append(mm.cross_entropy(x, w, tgt, reduction="sum", grad="w", dw_dtype=F32)[3])
        mm.embedding_grad(ids, x, out=acc, accumulate=True, scale=0.5)
        each.append(mm.embedding_grad(ids, x, 301, scale=0.5, out_dtype=F32))
    want = torch.stack(each).double().sum(0)
    mag = torch.stack(each).double().abs().sum(0)
    # six fp32 additions, a fused one each for the embedding's parts
    assert bool(((acc.double() - want).abs() <= 12 * 2.0 ** -24 * mag + 1e-30).all())


def _all(m, ids, tgt, x):
    grads = [m["table"], m["hidden"], m["head"]]
    out = [*mm.grad_norm(grads, max_norm=1.0), *mm.clip_grads(grads, 1.0, outputs=[torch.empty_like(t) for t in grads])]
    out += [mm.embedding(m["table"], ids, scale=2.0, out_dtype=BF16), mm.embedding_grad(ids, x, 301)]
    return out + list(mm.cross_entropy(x, m["head"].bfloat16(), tgt))


def test_other_streams():
    # calls on two streams at once share nothing; a stream handed in, and the
    # current one, give what the default stream gives
    print("[case] streams", flush=True)
    m, (ids, tgt) = _model(11), _batch(12)
    x = torch.randn(90, 128, device=DEV).bfloat16()
    want = _all(m, ids, tgt, x)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(_all(m, ids, tgt, x))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    given = [*mm.grad_norm([m["table"]], max_norm=1.0, stream=s1), mm.embedding(m["table"], ids, stream=s2),
             mm.embedding_grad(ids, x, 301, stream=s1), *mm.cross_entropy(x, m["head"].bfloat16(), tgt, stream=s2)]
    torch.cuda.synchronize()
    plain = [*mm.grad_norm([m["table"]], max_norm=1.0), mm.embedding(m["table"], ids),
             mm.embedding_grad(ids, x, 301), *mm.cross_entropy(x, m["head"].bfloat16(), tgt)]
    for a, b in zip(given, plain):
        assert torch.equal(a, b)


def test_graphs():
    # the first call ever of these shapes is captured; replays on new contents
    # of the same buffers match eager calls, with eager work in between, and
    # two graphs have scratch memory of their own
    print("[case] graphs", flush=True)
    m, (ids, tgt) = _model(21, rows=333, width=192), _batch(22, n=77, rows=333)
    x = torch.randn(77, 192, device=DEV).bfloat16()

    def work():
        grads = [m["table"], m["hidden"], m["head"]]
        out = list(mm.grad_norm(grads, max_norm=1.0))
        out += [mm.embedding(m["table"], ids, out_dtype=BF16), mm.embedding_grad(ids, x, 333)]
        return out + list(mm.cross_entropy(x, m["head"].bfloat16(), tgt))

    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work())
        graphs.append(g)
    for rep in range(4):
        for v in m.values():
            v.mul_(0.9).add_(0.01 * rep)
        x.normal_()
        i2, t2 = _batch(30 + rep, n=77, rows=333)
        ids.copy_(i2)
        tgt.copy_(t2)
        for g in graphs:
            g.replay()
        eager = work()
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(o, eager):
                assert torch.equal(a, b), rep
    del graphs
    torch.cuda.synchronize()


def test_step_graph_reads_the_scale_at_replay():
    print("[case] scale in a captured step", flush=True)
    w = [torch.randn(256, 256, device=DEV) * 0.02]
    g = [torch.randn(256, 256, device=DEV).bfloat16()]
    mom = [torch.zeros(256, 256, device=DEV, dtype=BF16)]
    coef = torch.ones(1, device=DEV)
    kw = dict(eta=0.02, beta=0.9, K=5, rho=[5.12], grad_scale=coef)
    mm.muonh_step(w, g, mom, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mm.muonh_step(w, g, mom, **kw)
    for c in (0.5, 0.0, 2.0):
        w2, m2 = [w[0].clone()], [mom[0].clone()]
        coef.fill_(c)
        graph.replay()
        mm.muonh_step(w2, g, m2, **kw)
        torch.cuda.synchronize()
        assert torch.equal(w[0], w2[0]) and torch.equal(mom[0], m2[0])
    del graph


def test_offsets_beyond_32_bits():
    # a table and a gradient of more than 2^32 bytes, rows at both ends
    print("[case] large offsets", flush=True)
    rows, width = 600_000, 4096  # 2.46e9 values, 4.9e9 bytes
    table = torch.empty(rows, width, device=DEV, dtype=BF16)
    table.view(-1, 1)[:: width // 2] = 1.0
    probe = torch.tensor([0, 262_143, 262_144, 524_288, 524_289, rows - 1], device=DEV)
    table[probe] = torch.arange(6, device=DEV, dtype=BF16)[:, None] + torch.randn(6, width, device=DEV).bfloat16()
    out = mm.embedding(table, probe)
    assert torch.equal(out, table[probe])
    d = torch.randn(6, width, device=DEV).bfloat16()
    grad = mm.embedding_grad(probe, d, rows, out=table)
    assert torch.equal(grad[probe], d)
    assert int((grad[:, 0] != 0).sum()) <= 6 and int((grad[rows - 1000: rows - 1] != 0).sum()) == 0
    total, _, _ = mm.grad_norm([grad])
    want = float(d.double().norm())
    assert abs(float(total) - want) <= 2.0 ** -23 * want
    mm.clip_grads([grad], want / 2)
    assert abs(float(grad[probe].double().norm()) / want - 0.5) <= 2.0 ** -8


@pytest.mark.parametrize("width", [8, 9, 15, 17, 1001])
@pytest.mark.parametrize("k", [0, 1, 3])
def test_embedding_off_the_grid(width, k):
    print(f"[case] embedding off the grid {width} {k}", flush=True)

    def off(t):
        b = torch.empty(t.numel() + k, dtype=t.dtype, device=DEV)
        v = b[k:].view(t.shape)
        v.copy_(t)
        return v

    g = torch.Generator(device="cpu")
    g.manual_seed(width)
    ids = torch.randint(0, 50, (700,), generator=g).to(DEV)
    for dt in (F32, BF16):
        table = torch.randn(50, width, generator=g).to(dt).to(DEV)
        d = torch.randn(700, width, generator=g).to(dt).to(DEV)
        guard = torch.full((50 * width + k + 64,), 7.0, dtype=dt, device=DEV)
        out = guard[k: k + 50 * width].view(50, width)
        want = mm.embedding_grad(ids, d, 50)
        got = mm.embedding_grad(ids, off(d), out=out)
        assert torch.equal(got, want)
        assert bool((guard[:k] == 7).all()) and bool((guard[k + 50 * width:] == 7).all())  # nothing beside it
        start = torch.randn(50, width, generator=g).to(dt).to(DEV)
        assert torch.equal(mm.embedding_grad(ids, off(d), out=off(start), accumulate=True),
                           mm.embedding_grad(ids, d, out=start.clone(), accumulate=True))
        rows = torch.full((700 * width + k + 64,), 7.0, dtype=dt, device=DEV)
        look = mm.embedding(off(table), ids, out=rows[k: k + 700 * width].view(700, width))
        assert torch.equal(look, table[ids])
        assert bool((rows[:k] == 7).all()) and bool((rows[k + 700 * width:] == 7).all())


def test_gradient_of_x_in_its_place():
    print("[case] dx over x", flush=True)
    x = torch.randn(300, 128, device=DEV).bfloat16()
    w = (torch.randn(500, 128, device=DEV) * 0.2).bfloat16()
    t = torch.randint(0, 500, (300,), device=DEV)
    want = mm.cross_entropy(x, w, t)
    got = mm.cross_entropy(x, w, t, dx=x)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert got[2].data_ptr() == x.data_ptr()


def test_a_gradient_listed_twice():
    print("[case] listed twice", flush=True)
    g = torch.randn(1000, device=DEV)
    total, _, norms = mm.grad_norm([g, g])
    assert abs(float(total) - math.sqrt(2) * float(norms[0])) <= 2.0 ** -22 * float(total)
    with pytest.raises(mm.MuonhError):
        mm.clip_grads([g, g], 1.0)


def test_clip_neighbouring_buffers():
    """Views of one flat buffer, in place and into another one; one gradient twice."""
    print("[case] clip neighbours", flush=True)
    torch.manual_seed(5)
    flat = torch.randn(1001, device=DEV) * 3
    want = flat.double() / (flat.double().norm() + 1e-6)
    cut = lambda t: [t[:3], t[3:500], t[500:]]  # noqa: E731
    other = torch.empty_like(flat)
    mm.clip_grads(cut(flat), 1.0, outputs=cut(other))
    mm.clip_grads(cut(flat), 1.0)
    # the coefficient and the product are rounded once each
    assert bool(((flat.double() - want).abs() <= 2.0 ** -22 * want.abs()).all())
    assert torch.equal(flat, other)
    g, a, b = torch.ones(8, device=DEV), torch.empty(8, device=DEV), torch.empty(8, device=DEV)
    mm.clip_grads([g, g], 2.0, outputs=[a, b])
    assert torch.equal(a, b) and abs(float(a[0]) - 0.5) < 1e-6
    with pytest.raises(mm.MuonhError):
        mm.clip_grads([a, b], 1.0, outputs=[b, a])


def test_python_refusals():
    print("[case] refusals", flush=True)
    t, i = torch.randn(6, 8, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    x, w = torch.randn(4, 8, device=DEV).bfloat16(), torch.randn(6, 8, device=DEV).bfloat16()
    bad = [
        (ValueError, lambda: mm.grad_norm([t.t()])), (ValueError, lambda: mm.grad_norm([t, t.cpu()])),
        (TypeError, lambda: mm.grad_norm([t.half()])), (mm.MuonhError, lambda: mm.grad_norm([t], max_norm=-1.0)),
        (ValueError, lambda: mm.clip_grads([t], 1.0, outputs=[t.bfloat16()])),
        (ValueError, lambda: mm.clip_grads([t], 1.0, outputs=[t, t])),
        (ValueError, lambda: mm.clip_grads([t], 1.0, outputs=[t[:3]])), (mm.MuonhError, lambda: mm.clip_grads([t], float("nan"))),
        (ValueError, lambda: mm.embedding(t.t(), i)), (TypeError, lambda: mm.embedding(t, i.short())),
        (TypeError, lambda: mm.embedding(t.half(), i)), (ValueError, lambda: mm.embedding(t, i, out=t)),
        (TypeError, lambda: mm.embedding(t, i, out_dtype=torch.float16)),
        (ValueError, lambda: mm.embedding_grad(i, t, 6)), (ValueError, lambda: mm.embedding_grad(i, t[:4])),
        (ValueError, lambda: mm.embedding_grad(i, t[:4], 6, accumulate=True)),
        (ValueError, lambda: mm.embedding_grad(i, t[:4], 7, out=t)), (TypeError, lambda: mm.embedding_grad(i, t[:4].half(), 6)),
        (TypeError, lambda: mm.cross_entropy(x.float(), w, i)), (TypeError, lambda: mm.cross_entropy(x, w.float(), i)),
        (ValueError, lambda: mm.cross_entropy(x[:3], w, i)), (TypeError, lambda: mm.cross_entropy(x, w, i.float())),
        (ValueError, lambda: mm.cross_entropy(x, w, i, dw=torch.empty_like(x))),
        (ValueError, lambda: mm.cross_entropy(x, w, i, grad=False, dx=x)),
        (ValueError, lambda: mm.cross_entropy(x, w, i, accumulate=True)),
        (ValueError, lambda: mm.cross_entropy(x.t().contiguous().t(), w, i)),
        (TypeError, lambda: mm.cross_entropy(x, w, i, dw_dtype=torch.float16)),
    ]
    for k, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            print("accepted:", k)
    torch.cuda.synchronize()
