"""Scratch memory over another buffer of the call is refused, by host validation before any
HIP call: the kernels of the gradients write there while others still read."""
import os

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = [pytest.mark.skipif(not os.path.exists(mm.LIB_PATH), reason="libmuonh.so not built"),
              pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that are never followed")]

MB = 1 << 20
A, B, C, D, E, F, G, H, WS = (64 * MB * k for k in range(1, 10))  # 64 megabytes apart


def grad(ws=WS, more=0, x=None, q=B, scales=C, dres=F, dx=G, dgain=H, n=700, width=2000):
    lib = mm.load()
    size = lib.muonh_rms_norm_grad_workspace(n, width) + more
    return lib.muonh_rms_norm_grad(A, 1, x, q, scales, D, E, dres, 0, n, width, dx, dgain, 0, ws, size, None)


def weight(ws=WS, more=0, n=600, rows=300, width=500, dw=E):
    lib = mm.load()
    size = lib.muonh_weight_grad_workspace(A, n, rows, width) + more
    return lib.muonh_weight_grad(A, B, C, D, 1.0, n, rows, width, dw, 0, 0, ws, size, None)


def test_scratch_over_a_buffer_of_the_norms_gradient():
    size = mm.load().muonh_rms_norm_grad_workspace(700, 2000)
    assert size >= 4 * 2000 * 256  # sums of the gain's gradient of 256 workgroups at least
    # bf16 dy, 8-bit rows and their scales, rstd, gain, residual's gradient, dx and dgain
    ends = {A: 2 * 700 * 2000, B: 700 * 2000, C: 700 * 63, D: 4 * 700, E: 4 * 2000, F: 4 * 700 * 2000, G: 4 * 700 * 2000, H: 4 * 2000}
    for at, bytes in ends.items():
        for ws in (at, at + (bytes - 1) // 256 * 256, at - (size - 1) // 256 * 256):
            assert grad(ws=ws) == mm.MUONH_EINVAL, (at // (64 * MB), ws - at)
        for ws in (at + -(-bytes // 256) * 256, at - size):
            assert grad(ws=ws) == mm.MUONH_EHIP  # no GPU: the checks were passed
    assert grad(ws=B, x=B, q=None, scales=None) == mm.MUONH_EINVAL
    # what is given beyond the need is not used
    assert grad(ws=A - size, more=4096) == mm.MUONH_EHIP
    # without the gain's gradient there is none
    assert grad(ws=A, dgain=None) == mm.MUONH_EHIP


def test_scratch_over_a_buffer_of_the_weight_gradient():
    for n, rows, width in ((600, 300, 500), (4100, 300, 500), (8192, 1200, 900)):
        size = mm.load().muonh_weight_grad_workspace(A, n, rows, width)
        ends = {A: 2 * n * rows, B: n * width, C: n * ((width + 31) // 32), D: 4 * width, E: 4 * rows * width}
        for at, bytes in ends.items():
            for ws in (at, at + (bytes - 1) // 256 * 256, at - (size - 1) // 256 * 256):
                assert weight(ws, 0, n, rows, width) == mm.MUONH_EINVAL, (n, at // (64 * MB), ws - at)
            for ws in (at + -(-bytes // 256) * 256, at - size):
                assert weight(ws, 4096, n, rows, width) == mm.MUONH_EHIP
