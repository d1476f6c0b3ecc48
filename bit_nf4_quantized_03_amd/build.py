"""Build the HIP library libqlora_nf4.so in-tree with hipcc for gfx950.

Usage: python bit_nf4_quantized_03_amd/build.py   (or call build()). It is
run as a file, not as a package module, because importing the package loads
the library this script produces.

Every source is compiled with -ffp-contract=off (the quantizer and the
dequantizer need exact fp32 round-to-nearest steps) and with the packed-fp32
target feature disabled.

_fastcall.so, the host code that makes whole calls of the microscaled and norm
entry points for the Python binding, is built next to the library with the
C++ compiler: it uses torch's headers and links the library. Where it cannot be
built the library is complete without it: calls then cost more host time.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libqlora_nf4.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
FASTCALL_PATH = os.path.join(PKG_DIR, "_fastcall.so")

SOURCES = ["api.cpp", "codebook.cpp", "profile.cpp", "nf4_quant.hip", "linear.hip", "gemv.hip", "merge.hip", "adamw.hip",
           "noalloc.hip", "api_mx.cpp", "mx_quant.hip", "rmsnorm.hip", "mx_linear.hip",
           "api_block.cpp", "mx_gated.hip", "rope.hip", "gated.hip",
           "gated_stream.hip"]
ARCH = os.environ.get("QLORA_OFFLOAD_ARCH", "gfx950")


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def _flags():
    return [
        "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
        "-ffp-contract=off",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wno-unused-command-line-argument",
        "-I", INCLUDE, "-I", CSRC,
    ]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [_hipcc()] + _flags() + ["-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    _run(cmd, "compile")
    return obj


def _run(cmd, what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")


def _compile_fastcall() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD_DIR, "fastcall.cpp.o")
    _run([shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
          "-c", os.path.join(CSRC, "fastcall.cpp"), "-o", obj], "compile")
    return obj


def _link_fastcall(obj: str) -> None:
    import torch
    tmp = FASTCALL_PATH + ".tmp"
    _run([shutil.which("g++") or "c++", "-shared", "-o", tmp, obj, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
          "-lc10", "-ltorch_cpu", "-ltorch_python", "-L", PKG_DIR, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"], "link")
    os.replace(tmp, FASTCALL_PATH)


def build(verbose: bool = False) -> str:
    """Compile every source and link libqlora_nf4.so and, where it can be built, _fastcall.so next to this file."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = min(len(SOURCES) + 1, max(1, min(8, os.cpu_count() or 1)))
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        fast = ex.submit(_compile_fastcall)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp"
    _run([_hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs, "link")
    os.replace(tmp, LIB_PATH)
    try:
        _link_fastcall(fast.result())
    except Exception as e:   # no torch, its headers, Python's headers or a C++ compiler
        if os.path.exists(FASTCALL_PATH):
            os.remove(FASTCALL_PATH)   # it belongs to an older library
        print(f"{os.path.basename(FASTCALL_PATH)} was not built, calls cost more host time: {e}", file=sys.stderr)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
