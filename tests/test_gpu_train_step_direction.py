"""A clipped step on the gradients of the operators goes down them, by the formula's amount."""
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402
from test_gpu_train_step import _batch, _gradients, _model  # noqa: E402

pytestmark = pytest.mark.gpu


def test_direction_of_a_clipped_step():
    print("[case] direction of a step", flush=True)
    m, (ids, tgt) = _model(1), _batch(2)
    _, grads = _gradients(m, ids, tgt, 3.0)
    _, coef, _ = mm.grad_norm([grads[k] for k in ("table", "hidden", "head")], max_norm=0.05)
    assert 0 < float(coef) < 1
    new = {k: v.clone() for k, v in m.items()}
    two, eta, eps = ["table", "head"], 1e-3, 1e-8
    mom = [torch.zeros_like(m[k]) for k in two], [torch.zeros_like(m[k]) for k in two]
    mm.adamh_step([new[k] for k in two], [grads[k] for k in two], *mom, eta=eta, step=1, eps=eps, hook="none",
                  grad_scale=coef)
    buf = torch.zeros_like(m["hidden"])
    mm.muonh_step([new["hidden"]], [grads["hidden"]], [buf], 0.02, 0.95, 5, rho=[float(m["hidden"].norm())],
                  ns_dtype="f32", grad_scale=coef)
    torch.cuda.synchronize()
    for k in two:
        g = grads[k].double() * coef.double()
        # Adam's first step: both moments are the gradient's own
        want = -eta * g / (g.abs() + eps)
        got = new[k].double() - m[k].double()
        # some ten fp32 operations on the update, one rounding of the weight
        tol = 16 * 2.0 ** -24 * eta + 2.0 ** -24 * (m[k].double().abs() + eta)
        assert bool(((got - want).abs() <= tol).all()), (k, float((got - want).abs().max()))
    for k in m:
        d = (new[k] - m[k]).double()
        assert float((grads[k].double() * d).sum()) < 0, k
    g = grads["hidden"].double() * coef.double()
    assert bool(((buf.double() - g).abs() <= 2 * 2.0 ** -24 * g.abs()).all())
