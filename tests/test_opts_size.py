"""muonh_opts grew by a field at its end: programs built on the shorter structure
keep working, byte for byte."""
import ctypes
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muonh.h")

pytestmark = pytest.mark.skipif(not os.path.exists(mm.LIB_PATH), reason="libmuonh.so not built")

SHORT = mm.Opts.grad_scale.offset  # the structure before grad_scale
FULL = ctypes.sizeof(mm.Opts)


def test_defaults_of_a_short_structure_stay_inside_it():
    buf = (ctypes.c_ubyte * (FULL + 64))(*([0xA5] * (FULL + 64)))
    mm.load().muonh_default_opts(ctypes.cast(buf, ctypes.POINTER(mm.Opts)))
    assert bytes(buf[SHORT:]) == b"\xa5" * (FULL + 64 - SHORT)
    o = ctypes.cast(buf, ctypes.POINTER(mm.Opts)).contents
    assert o.deterministic == 1 and o.ns_precision == mm.MUONH_NS_H16 and o.outward == 0.5


def test_a_short_structure_at_the_end_of_memory():
    # the page behind it cannot be read: in a process of its own
    code = f"""
import ctypes, mmap
import matrix_orthogonalizing_optimizer_momentum_amd as mm
lib = mm.load()
page = mmap.PAGESIZE
m = mmap.mmap(-1, 2 * page)
base = ctypes.addressof(ctypes.c_char.from_buffer(m))
libc = ctypes.CDLL(None, use_errno=True)
assert libc.mprotect(ctypes.c_void_p(base + page), page, 0) == 0
at = base + page - {SHORT}
opts = ctypes.cast(at, ctypes.POINTER(mm.Opts))
lib.muonh_default_opts(opts)
out = (ctypes.c_int64 * 7)()
sh = (ctypes.c_int64 * 2)(64, 64)
assert lib.muonh_plan_query(sh, 1, 5, 0, opts, 0, out) == 0 and out[2] == 1
print("through", flush=True)
import os
os._exit(0)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, HIP_VISIBLE_DEVICES=""))
    assert r.returncode == 0 and "through" in r.stdout, (r.returncode, r.stderr[-500:])


@pytest.mark.parametrize("size", [SHORT, FULL, FULL + 24])
def test_defaults_by_size(size):
    total = FULL + 64
    buf = (ctypes.c_ubyte * total)(*([0xA5] * total))
    mm.load().muonh_default_opts_sized(ctypes.cast(buf, ctypes.POINTER(mm.Opts)), size)
    assert bytes(buf[size:]) == b"\xa5" * (total - size)
    o = ctypes.cast(buf, ctypes.POINTER(mm.Opts)).contents
    assert o.deterministic == 1
    assert o.opts_bytes == (FULL if size >= FULL else 0)
    if size >= FULL:
        assert o.grad_scale is None and bytes(buf[FULL:size]) == b"\0" * (size - FULL)


def test_the_binding_names_its_size():
    assert mm.make_opts(stream=0)[0].opts_bytes == FULL


def test_a_c_program_gets_the_whole_structure(tmp_path):
    # the header's muonh_default_opts knows the size it was compiled with
    src, exe = tmp_path / "p.c", tmp_path / "p"
    src.write_text('#include "muonh.h"\n#include <stddef.h>\n#include <string.h>\nint main(void) {\n'
                   "  muonh_opts o;\n  memset(&o, 0xA5, sizeof o);\n  muonh_default_opts(&o);\n"
                   f"  return o.grad_scale != NULL || o.opts_bytes != sizeof o || sizeof o != {FULL} ||\n"
                   f"         offsetof(muonh_opts, grad_scale) != {SHORT} || offsetof(muonh_opts, opts_bytes) != "
                   f"{mm.Opts.opts_bytes.offset if hasattr(mm.Opts, 'opts_bytes') else -1};\n}}\n")
    # the HIP runtime that this process has loaded: a second one is not wanted beside it
    lib = os.path.dirname(mm.LIB_PATH)
    rocm = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "lib")
    subprocess.run(["gcc", "-Wall", "-Werror", f"-I{os.path.dirname(HEADER)}", str(src), "-o", str(exe), f"-L{lib}",
                    "-lmuonh", f"-Wl,-rpath,{lib}", f"-Wl,-rpath,{rocm}", f"-L{rocm}", "-Wl,--allow-shlib-undefined"],
                   check=True)
    assert subprocess.run([str(exe)], timeout=300).returncode == 0


@pytest.mark.gpu
def test_steps_read_the_scale_of_whole_structures_only():
    print("[case] grad_scale behind a short structure", flush=True)
    scale = torch.full((1,), 0.5, device="cuda")

    def step(full):
        w, g, m = (torch.full((64, 96), v, device="cuda") for v in (0.5, 0.01, 0.0))
        m2 = torch.zeros_like(w)
        o, _ = mm.make_opts(state_dtype=mm.MUONH_F32, hook="none")
        if not full:
            mm.load().muonh_default_opts(ctypes.byref(o))
            o.state_dtype, o.hook = mm.MUONH_F32, mm.MUONH_HOOK_NONE
            o.stream = torch.cuda.current_stream().cuda_stream
        o.grad_scale = scale.data_ptr()  # for a short structure: whatever stands behind it
        ptr = lambda t: (ctypes.c_void_p * 1)(t.data_ptr())  # noqa: E731
        sh = (ctypes.c_int64 * 2)(64, 96)
        lib = mm.load()
        assert lib.muonh_step(ptr(w), ptr(g), ptr(m), sh, 1, 0.02, 0.5, 3, None, 0, ctypes.byref(o)) == 0
        v = torch.zeros_like(w)
        assert lib.adamh_step(ptr(w), ptr(g), ptr(m2), ptr(v), sh, 1, 1e-3, 0.5, 0.5, 1e-8, 1, None, ctypes.byref(o)) == 0
        torch.cuda.synchronize()
        return m, m2

    for m, part in zip(step(False), (1.0, 0.5)):
        assert torch.equal(m, torch.full_like(m, 0.01) * part)
    for m, part in zip(step(True), (0.5, 0.25)):
        assert torch.equal(m, torch.full_like(m, 0.01) * part)
