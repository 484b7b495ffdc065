"""The paths of the token sort and of the norm's second kernel that long lists take."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402
from test_gpu_gradients import BF16, DEV, F32, U, _grad_ref, _ids, _rand  # noqa: E402

pytestmark = pytest.mark.gpu


# more than 262144 tokens: sort tiles above 1024 tokens; more than 2^22 rows
# with more than 8192 tokens: three passes; and both
@pytest.mark.parametrize("rows,width,n,kind", [
    (5000, 8, 262145, "skewed"), (5000, 3, 300001, "padded"), (2 ** 22 + 5, 1, 9000, "padded"),
    (2 ** 22 + 5, 9, 8193, "uniform"), (2 ** 23 + 1, 2, 300001, "skewed"), (40, 8, 300001, "one"),
])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_long_sorts(rows, width, n, kind, idt):
    print(f"[case] embedding grad {rows} x {width}, {n} tokens {kind} {idt}", flush=True)
    ids = _ids(n, rows, kind, idt, 3)
    dout = _rand((n, width), BF16, 4)
    got = mm.embedding_grad(ids, dout, rows, scale=0.5, out_dtype=F32)
    want, mag, cnt = _grad_ref(ids, dout, rows, 0.5)
    # at most as many fp32 additions as tokens, each off by 2^-24 of a partial
    # sum that the sum of magnitudes bounds; then the output's rounding
    tol = cnt[:, None] * U[F32] * mag
    tol = tol + U[F32] * (np.abs(want) + tol)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol + 1e-300).all(), float((err - tol).max())
    start = torch.ones((rows, width), device=DEV)
    acc = mm.embedding_grad(ids, dout, scale=0.5, out=start.clone(), accumulate=True)
    err = np.abs(acc.double().cpu().numpy() - (want + 1.0))
    assert (err <= tol + U[F32] * (np.abs(want + 1.0) + tol) + 1e-300).all()
    assert torch.equal(acc[torch.from_numpy(cnt == 0).to(DEV)], start[: int((cnt == 0).sum())])


# up to 2047 tensors and 4096 blocks the second kernel stages its lists
@pytest.mark.parametrize("n", [2047, 2048, 5000])
def test_norm_and_clip_of_long_lists(n):
    print(f"[case] norm of {n} tensors", flush=True)
    flat = _rand((n * 23,), F32, 7, 1e-2)
    ts = [flat[23 * i: 23 * i + 1 + (7 * i) % 23] for i in range(n)]
    ts = [t.bfloat16() if i % 3 == 0 else t for i, t in enumerate(ts)]
    sq = np.array([float((t.double() ** 2).sum()) for t in (t.cpu() for t in ts)])
    want = math.sqrt(sq.sum())
    total, coef, norms = mm.grad_norm(ts, max_norm=1.0)
    assert abs(float(total) - want) <= 1.01 * U[F32] * want
    assert (np.abs(norms.double().cpu().numpy() - np.sqrt(sq)) <= 1.01 * U[F32] * np.sqrt(sq)).all()
    outs = [torch.empty_like(t) for t in ts]
    total2, coef2 = mm.clip_grads(ts, 1.0, outputs=outs)
    assert torch.equal(total, total2) and torch.equal(coef, coef2) and 0 < float(coef) < 1
    for t, o in zip(ts, outs):
        assert torch.equal(o, (t.float() * coef).to(t.dtype))
