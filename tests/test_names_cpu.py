"""The functions of gradients.py and activations.py as the package shows them."""
import subprocess
import sys

import pytest

pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402
from matrix_orthogonalizing_optimizer_momentum_amd import activations, gradients  # noqa: E402


@pytest.mark.parametrize("name", ["clip_grads", "cross_entropy", "embedding", "embedding_grad", "grad_norm"])
def test_a_replaced_function_is_seen(name, monkeypatch):
    own = getattr(gradients, name)
    assert getattr(mm, name) is own
    other = lambda *a, **k: None  # noqa: E731
    with monkeypatch.context() as m:
        m.setattr(gradients, name, other)
        assert getattr(mm, name) is other
    assert getattr(mm, name) is own


def test_the_names_of_the_activations():
    for name in ("Normed", "Packed", "mx_pack", "mx_unpack", "rms_norm", "rms_norm_grad", "weight_grad"):
        assert getattr(mm, name) is getattr(activations, name)
    with pytest.raises(AttributeError, match="no attribute 'rms'"):
        mm.rms


def test_the_package_alone_needs_no_torch():
    code = "import sys, {0} as p; assert 'torch' not in sys.modules; p.cross_entropy; assert 'torch' in sys.modules".format(mm.__name__)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
