"""Build libtrace_fp4.so in-tree with nvcc for sm_100a (no torch involved), and
the Python module beside it that calls it for torch tensors (g++)."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "trace_fp4.cu")
CSRC_DIR = os.path.join(PKG, "csrc")
BIND_SRC = os.path.join(PKG, "csrc", "binding.cpp")
BIND = os.path.join(PKG, "_binding.so")
HDR = os.path.join(ROOT, "include", "trace_fp4.h")
LIB = os.path.join(PKG, "libtrace_fp4.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    # IEEE single precision everywhere: no flush-to-zero, correctly rounded
    # division and square root, no contraction of a*b+c into an FMA
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=false",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library, and the Python module beside it where torch, the
    Python headers and g++ are there; returns the library's path.  A caller from
    C needs nothing but nvcc: without the module only ops.binding() fails."""
    build_library(force, verbose)
    try:
        build_binding(force)
    except (ImportError, OSError, RuntimeError) as e:
        sys.stderr.write(f"{os.path.basename(BIND)} has not been built: {e}\n")
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/trace_fp4.cu (which includes the csrc/*.cuh kernels) into
    the package directory; returns the library's path."""
    deps = [HDR] + [os.path.join(CSRC_DIR, f) for f in os.listdir(CSRC_DIR)
                    if f.endswith((".cu", ".cuh", ".h"))]
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(d) for d in deps)):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", tmp, SRC]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc failed building libtrace_fp4.so")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, LIB)
    return LIB


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp against the installed torch; returns the path."""
    if (not force and os.path.exists(BIND)
            and os.path.getmtime(BIND) >= max(os.path.getmtime(d) for d in (HDR, BIND_SRC))):
        return BIND
    if os.path.exists(BIND):  # outdated: not to be loaded if this fails
        os.unlink(BIND)
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_path("include"),
           "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-o", tmp, BIND_SRC,
           "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed building _binding.so")
    os.replace(tmp, BIND)
    return BIND


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB, BIND)
