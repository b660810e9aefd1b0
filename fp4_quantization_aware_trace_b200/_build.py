"""Build libtrace_fp4.so in-tree with nvcc for sm_100a (no torch involved), and
the Python module beside it that calls it for torch tensors (g++)."""
from __future__ import annotations

import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "trace_fp4.cu")
CSRC_DIR = os.path.join(PKG, "csrc")
BIND_SRC = os.path.join(PKG, "csrc", "binding.cpp")
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
        sys.stderr.write(f"the Python module of csrc/binding.cpp has not been built: {e}\n")
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


def binding_path() -> str:
    """The module for this Python and the installed torch, whose C++ classes it is
    compiled against: one built for others has another name and is not loaded."""
    import torch
    git = getattr(torch.version, "git_version", None) or ""
    torch_id = re.sub(r"[^0-9A-Za-z.]", "_", f"{torch.__version__}-{git[:8]}")
    return os.path.join(PKG, f"_binding.torch{torch_id}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp against the installed torch; returns the path."""
    import torch
    path = binding_path()
    if (not force and os.path.exists(path)
            and os.path.getmtime(path) >= max(os.path.getmtime(d) for d in (HDR, BIND_SRC))):
        return path
    if os.path.exists(path):  # outdated: not to be loaded if this fails
        os.unlink(path)
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = path + f".tmp{os.getpid()}"
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
        raise RuntimeError("g++ failed")
    os.replace(tmp, path)
    return path


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
