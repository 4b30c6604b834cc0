"""Build libsp24.so (HIP, gfx950 only) and the Python module _sp24.so in-tree.

    python bf16_gemm_linear_amd/build.py

(run as a script: importing the package first would load the library being
replaced, and fail if it predates a symbol the binding declares).

Every source in csrc/ is compiled with hipcc for gfx950 and linked into
bf16_gemm_linear_amd/libsp24.so; csrc/sp24_python.cpp, host code against PyTorch's
headers, becomes bf16_gemm_linear_amd/_sp24.so, which loads it.  No fast-math: float32 division and square
root stay correctly rounded (the FP8 scale and the per-value division depend on
it), and denormals are kept.  Packed-fp32 VALU forms are switched off.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libsp24.so")
MODULE = os.path.join(HERE, "_sp24.so")

ARCH = "gfx950"
CXX = os.environ.get("CXX", shutil.which("g++") or "g++")
HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=" + ARCH,
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; that is harmless
    err = "\n".join(ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, err))
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _compile_module() -> str:
    """The Python module's object file (host C++)."""
    import sysconfig

    from torch.utils.cpp_extension import include_paths
    src, obj = os.path.join(CSRC, "sp24_python.cpp"), os.path.join(BUILD_DIR, "sp24_python.o")
    inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], *include_paths(),
           os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"), "/opt/rocm/include"]
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           *("-I" + d for d in inc[:2]), *("-isystem" + d for d in inc[2:]), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed for %s:\n%s" % (CXX, src, r.stderr))
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _link_module(obj: str) -> None:
    import torch
    tmp = MODULE + ".tmp"
    cmd = [CXX, "-shared", "-o", tmp, obj, "-L" + HERE, "-l:libsp24.so", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, MODULE)


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        module = ex.submit(_compile_module)
        objs = list(ex.map(_compile, srcs))
        module = module.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, LIB)
    _link_module(module)
    if verbose:
        print("built", LIB, "and", os.path.basename(MODULE))
    return LIB


if __name__ == "__main__":
    build()
