"""Builds libfp8mot.so (the HIP kernels and the C ABI) in-tree for gfx950, and
_binding.so, the native front of the binding's small calls (host code: g++
against Python, torch and libfp8mot).

Compiler flags:
  --offload-arch=gfx950          the only target (no other architecture);
  -ffp-contract=off              arithmetic as written: no implicit FMA, so
                                 the observer update and the epilogue round
                                 exactly where the code says;
  -target-feature -packed-fp32-ops
                                 no packed FP32 instructions are generated;
  no fast-math                   FP32 division stays correctly rounded.
"""

import os
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libfp8mot.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = ["elementwise.hip", "gemm.hip", "linear_act_tile.hip", "linear_act.hip", "layer_norm.hip",
           "mfma_ceiling.hip", "verify.hip", "capi.hip"]

BINDING_PATH = os.path.join(PKG, "_binding.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("command failed: " + " ".join(cmd))
    return r


def build(verbose=False, jobs=4) -> str:
    """Compile every source, link libfp8mot.so and build the native front of
    the binding; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        _run(cmd)
        return obj

    with ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp])
    os.replace(tmp, LIB_PATH)
    build_front(verbose)
    return LIB_PATH


def build_front(verbose=False):
    """build_binding, or where that is not possible (no g++, no torch headers)
    no front at all, with a warning: the binding then runs its checks in
    Python, and a front of another library's build must not stay beside this
    one."""
    try:
        build_binding(verbose)
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)
        warnings.warn(f"the native front of the binding was not built: {e}")


def build_binding(verbose=False) -> str:
    """Compile the native front against the installed torch and the in-tree
    libfp8mot.so (found at run time beside it); returns its path."""
    import sysconfig

    from torch.utils import cpp_extension as ext

    tmp = BINDING_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
           "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"]]
    for d in ext.include_paths():
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", PKG, "-lfp8mot"]
    for d in ext.library_paths():
        cmd += ["-L", d]
    cmd += ["-lc10", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    _run(cmd)
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def device_assembly(src) -> str:
    """gfx950 assembly text of one source (for inspection by tests)."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    out = os.path.join(BUILD_DIR, src.replace(".hip", ".gfx950.s"))
    _run([HIPCC, *FLAGS, "--cuda-device-only", "-S",
          os.path.join(CSRC, src), "-o", out])
    with open(out) as f:
        return f.read()


if __name__ == "__main__":
    print(build(verbose=True))
