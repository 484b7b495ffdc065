"""What build() needs for which of the two libraries, without compiling."""
import os
import sys

import pytest

from matrix_orthogonalizing_optimizer_momentum_amd import build as b


@pytest.fixture
def dry(monkeypatch, tmp_path):
    """build() with outputs under tmp_path and commands that only write their output file."""
    ran = []

    def run(cmd):
        ran.append(cmd)
        if "fail" in cmd:
            raise RuntimeError("command failed: headers")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        return ""

    for name, to in (("OUT", "libmuonh.so"), ("BINDING_OUT", "_tensors.so"), ("BUILD_DIR", "obj")):
        monkeypatch.setattr(b, name, str(tmp_path / to))
    monkeypatch.setattr(b, "HIPCC", sys.executable)  # present on any machine
    monkeypatch.setattr(b, "_run", run)
    return ran


def test_both_are_built(dry):
    assert b.build() == b.OUT
    assert os.path.exists(b.OUT) and os.path.exists(b.BINDING_OUT)
    assert any(b.BINDING in c for c in dry)


@pytest.mark.parametrize("error", [ImportError("No module named 'torch'"), OSError("libtorch_cpu.so: cannot open")])
def test_the_library_needs_no_torch(dry, monkeypatch, capsys, error):
    def none(out):
        raise error

    monkeypatch.setattr(b, "binding_cmd", none)
    with open(b.BINDING_OUT, "w") as f:
        f.write("an old one")
    assert b.build() == b.OUT and os.path.exists(b.OUT)
    # what stands there was built from other sources
    assert not os.path.exists(b.BINDING_OUT)
    assert "_tensors.so" in capsys.readouterr().err


def test_a_binding_that_does_not_compile_leaves_the_library(dry, monkeypatch):
    monkeypatch.setattr(b, "binding_cmd", lambda out: ["g++", "fail", "-o", out])
    with pytest.raises(RuntimeError, match="headers"):
        b.build()
    assert os.path.exists(b.OUT)
