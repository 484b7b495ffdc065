"""Build libmuonh.so for gfx950 with hipcc (in-tree, no JIT cache).

    python -m matrix_orthogonalizing_optimizer_momentum_amd.build

compiles every csrc/*.hip with hipcc --offload-arch=gfx950, the host-only
planner with g++, and links them into libmuonh.so next to this file; beside it
_tensors.so, the Python extension that reads lists of torch tensors and makes the
calls of activations.py (binding/*.cpp, host code only).  libmuonh.so needs hipcc and g++ alone;
the extension, torch with its headers.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libmuonh.so")
BINDING = os.path.join(HERE, "binding", "tensors.cpp")
BINDING_CALLS = os.path.join(HERE, "binding", "activations.cpp")
BINDING_OUT = os.path.join(HERE, "_tensors.so")
BUILD_DIR = os.path.join(ROOT, "_build", "muonh")

ARCH = os.environ.get("MUONH_ARCH", "gfx950")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.path.join(ROCM, "bin", "hipcc")

HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 ALU ops off: scalar / float2 code stays unpacked
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
    f"-I{INCLUDE}", f"-I{CSRC}",
]
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", f"-I{INCLUDE}", f"-I{CSRC}"]


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # the host pass of hipcc does not know the packed-fp32 feature: drop that noise
    lines = [ln for ln in r.stdout.splitlines() if "packed-fp32-ops" not in ln]
    if r.returncode != 0:
        raise RuntimeError("command failed: " + " ".join(cmd) + "\n" + "\n".join(lines))
    return "\n".join(lines)


def sources():
    hip = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))
    cpp = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cpp"))
    return hip, cpp


def binding_cmd(out):
    """The g++ line of the extension, against the installed torch."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    return ["g++", *HOST_FLAGS, "-shared", f"-I{sysconfig.get_paths()['include']}", f"-isystem{inc}",
            f"-isystem{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", BINDING, BINDING_CALLS, "-o", out,
            f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Compile and link; returns the path of the built library."""
    if not os.path.exists(HIPCC):
        raise RuntimeError(f"hipcc not found at {HIPCC}")
    os.makedirs(BUILD_DIR, exist_ok=True)
    hip, cpp = sources()
    cmds = []
    objs = []
    for src in hip:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmds.append([HIPCC, *HIP_FLAGS, "-c", src, "-o", obj])
        objs.append(obj)
    for src in cpp:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmds.append(["g++", *HOST_FLAGS, "-c", src, "-o", obj])
        objs.append(obj)
    # The library needs no torch: it is linked whatever becomes of the extension.
    try:
        binding = binding_cmd(BINDING_OUT + ".tmp")
    except (ImportError, OSError) as e:  # OSError: a torch whose libraries do not load
        binding = None
        print(f"without {os.path.basename(BINDING_OUT)} (lists of torch tensors, activations): {e}", file=sys.stderr)
    jobs = jobs or min(len(cmds) + 1, max(1, (os.cpu_count() or 4)))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        done = [ex.submit(_run, cmd) for cmd in cmds]
        extension = ex.submit(_run, binding) if binding else None
        for f in done:
            out = f.result()
            if verbose and out.strip():
                print(out)
    tmp = OUT + ".tmp"
    _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, OUT)
    if os.path.exists(BINDING_OUT):
        os.remove(BINDING_OUT)  # of other sources, until it is replaced
    if extension:
        out = extension.result()
        if verbose and out.strip():
            print(out)
        os.replace(BINDING_OUT + ".tmp", BINDING_OUT)
    return OUT


def clean():
    shutil.rmtree(BUILD_DIR, ignore_errors=True)
    for f in (OUT, BINDING_OUT):
        if os.path.exists(f):
            os.remove(f)


if __name__ == "__main__":
    p = build(verbose="-v" in sys.argv)
    print(p)
