"""Build libllar.so (the C-ABI library) from the HIP sources for gfx950.

Every HIP translation unit is compiled separately (in parallel) with
hipcc --offload-arch=gfx950 and linked into one shared library next to this
file.  Packed-FP32 instructions are disabled for the device code.
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
LIB = os.path.join(HERE, "libllar.so")
BINDING = os.path.join(HERE, "_llar_py.so")
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["llar_kernels.hip", "llar_multi.hip", "llar_host.hip", "llar_floor.hip", "llar_ffn.hip",
           "llar_ffn_kernels.hip", "llar_int8.hip", "llar_int8_kernels.hip", "llar_moe.hip",
           "llar_moe_kernels.hip"]
# the matrix product, compiled once for each element type and operand order
INSTANCES = [("llar_gemm_inst.hip", "llar_gemm_%s_%d%d" % (e.lower(), x, w),
              ["-DLLAR_ELEM=" + e, "-DLLAR_XR=%d" % x, "-DLLAR_WR=%d" % w])
             for e in ("F32", "F16", "BF16") for x in (0, 1) for w in (0, 1)]
# and both products of a backward pass in one launch
INSTANCES += [("llar_gemm_pair.hip", "llar_gemm_pair_%s_%d" % (e.lower(), w), ["-DLLAR_ELEM=" + e, "-DLLAR_WR=%d" % w])
              for e in ("F32", "F16", "BF16") for w in (0, 1)]
INSTANCES += [("llar_gemm_int8.hip", "llar_gemm_int8_" + e.lower(), ["-DLLAR_ELEM=" + e]) for e in ("F32", "F16", "BF16")]
ARCH = "gfx950"

CFLAGS = [
    "--offload-arch=" + ARCH,
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-munsafe-fp-atomics",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", INCLUDE,
    "-I", CSRC,
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the HIP toolchain is required to build libllar.so")
    return path


def _compile(unit) -> str:
    src, name, defines = unit
    obj = os.path.join(BUILD_DIR, name + ".o")
    cmd = [hipcc(), *CFLAGS, *defines, "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr[-4000:]))
    return obj


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libllar.so; returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    units = [(src, os.path.splitext(src)[0], []) for src in SOURCES] + INSTANCES
    with cf.ThreadPoolExecutor(max_workers=min(len(units), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, units))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr[-4000:]))
    os.replace(tmp, LIB)
    _build_binding()
    if verbose:
        print("built", LIB, file=sys.stderr)
    return LIB


def _c_compiler():
    """gcc, or the clang that comes with hipcc."""
    for name in ("gcc", "cc", "clang", "amdclang", "/opt/rocm/llvm/bin/clang"):
        path = shutil.which(name)
        if path:
            return path
    return None


def _build_binding() -> bool:
    """The feed-forward operators' Python entry points (plain C against libllar.so and the CPython API).

    Only they need a C compiler and Python's headers.  Where those are missing the rest stays usable: no binding
    is left (an older one would not fit the library), a line says so, and the operators raise when called."""
    python = sysconfig.get_paths()["include"]
    compiler = _c_compiler()
    if compiler is None or not os.path.exists(os.path.join(python, "Python.h")):
        if os.path.exists(BINDING):
            os.remove(BINDING)
        print("not built: %s (no %s), so linear, gated_ffn, moe_ffn and the like are not available from Python"
              % (os.path.basename(BINDING), "C compiler" if compiler is None else "Python.h in " + python),
              file=sys.stderr)
        return False
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [compiler, "-O2", "-std=c11", "-Wall", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", python, os.path.join(CSRC, "llar_py.c"), "-o", tmp,
           "-L", HERE, "-l:libllar.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("building the binding failed:\n%s\n%s" % (" ".join(cmd), res.stderr[-4000:]))
    os.replace(tmp, BINDING)
    return True


if __name__ == "__main__":
    build(verbose=True)
