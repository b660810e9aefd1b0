"""The FP4 expert operators' host side off the usual path (no GPU)."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import warnings

import pytest
import torch

from fp4_quantization_aware_trace_b200 import ops

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp4_quantization_aware_trace_b200", "csrc")


def test_plans_hold_on_any_gpu(tmp_path):
    exe = str(tmp_path / "plan_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(HERE, "plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_operands_of_other_lengths_are_refused():
    """By the shape of their scales, which for row-major ones gives the length of
    a row: bytes of the right number may be rows of another."""
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    f32 = torch.ones(1)
    for cols, scales, fits in ((64, (4, 4), True), (32, (4, 4), False), (128, (4, 4), False),
                               (64, (2, 8), False), (64, (512,), True), (64, (16,), False),
                               (64, (1, 512), False), (64, (4, 4, 1), False), (64, (2, 16, 16), False)):
        a = ops.Capture(u8(4 * 32), None, u8(*scales), f32)
        if fits:
            assert ops._matmul_operand(a, cols, 16, "a")[0] == 4
        else:
            with pytest.raises(ops.TraceError, match="scales of"):
                ops._matmul_operand(a, cols, 16, "a")
    a, w = ops.Capture(u8(4 * 64), None, u8(4, 8), f32), ops.Capture(u8(6 * 128), None, u8(6, 16), f32)
    for pair in ((a, w), (w, a)):
        with pytest.raises(ops.TraceError, match="scales of"):
            ops.fp4_matmul(*pair)
    ma, mw = ops.MxCapture(u8(4 * 64), None, u8(4, 4)), ops.MxCapture(u8(6 * 128), None, u8(6, 8))
    with pytest.raises(ops.TraceError, match="scales of"):
        ops.mx_matmul(ma, mw)


def _tree(tmp_path, monkeypatch):
    """A copy of the build files whose compilers only write their outputs: the
    module _build of it, and the commands that it has run."""
    root = tmp_path / "tree"
    shutil.copytree(CSRC, root / "pkg" / "csrc")
    shutil.copytree(os.path.join(os.path.dirname(HERE), "include"), root / "include")
    shutil.copy(os.path.join(os.path.dirname(CSRC), "_build.py"), root / "pkg")
    spec = importlib.util.spec_from_file_location("_build_of_a_copy", root / "pkg" / "_build.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    ran = []

    def run(cmd, **kw):
        ran.append(os.path.basename(cmd[0]))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mod.subprocess, "run", run)
    return mod, ran


def _modules(mod):
    return sorted(f for f in os.listdir(mod.PKG) if f.startswith("_binding"))


@pytest.mark.parametrize("missing", ["torch", "g++", "headers"])
def test_the_library_is_built_without_the_module(tmp_path, monkeypatch, missing):
    mod, ran = _tree(tmp_path, monkeypatch)
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    run = mod.subprocess.run

    def some(cmd, **kw):
        if os.path.basename(cmd[0]) == "g++" and missing == "g++":
            raise FileNotFoundError("g++")
        r = run(cmd, **kw)
        if os.path.basename(cmd[0]) == "g++" and missing == "headers":
            r.returncode = 1
        return r

    monkeypatch.setattr(mod.subprocess, "run", some)
    assert mod.build(force=True) == mod.LIB and os.path.exists(mod.LIB)
    assert ran[0] == "nvcc" and not [f for f in _modules(mod) if f.endswith(".so")]
    assert mod.build() == mod.LIB and ran.count("nvcc") == 1


def test_the_module_belongs_to_its_torch(tmp_path, monkeypatch):
    """Built again for another torch or Python, and never loaded by them."""
    mod, ran = _tree(tmp_path, monkeypatch)
    first = mod.build_binding()
    assert mod.build_binding() == first and ran == ["g++"]
    monkeypatch.setattr(torch, "__version__", "99.0.1+cu999")
    second = mod.build_binding()
    assert second != first and ran == ["g++", "g++"]
    monkeypatch.setattr(torch.version, "git_version", "0123456789abcdef")
    third = mod.build_binding()
    monkeypatch.setattr(mod.sysconfig, "get_config_var", lambda name: ".cpython-399-test.so")
    assert len({first, second, third, mod.build_binding()}) == 4 and len(_modules(mod)) == 4
    # the real one: only under the installed torch's name
    monkeypatch.setattr(ops, "_bind", None)
    with pytest.raises(ops.TraceError, match="has not been built"):
        ops.binding()


def test_calls_without_the_module(monkeypatch):
    """A warning, once, and the calls go on to their own checks; binding() says
    what is missing, and finds the module once it is there."""
    monkeypatch.setattr(ops, "_bind", None)
    with monkeypatch.context() as m:
        m.setattr(ops._build, "binding_path", lambda: os.path.join(HERE, "no_such_module.so"))
        with pytest.raises(ops.TraceError, match="has not been built"):
            ops.binding()
        ids = torch.zeros(3, 2, dtype=torch.int32)
        route = ops.MoeRoute(torch.zeros(6, dtype=torch.int64), ids, ids.view(-1))
        x, y, w = torch.zeros(3, 32).bfloat16(), torch.zeros(6, 32).bfloat16(), torch.zeros(3, 2)
        a = ops.Capture(torch.zeros(128, dtype=torch.uint8), None, torch.zeros(4, 4, dtype=torch.uint8),
                        torch.ones(1))
        calls = (lambda: ops.moe_sort(ids, 4), lambda: ops.moe_dispatch(x, route),
                 lambda: ops.moe_combine(y, route, w), lambda: ops.fp4_matmul(a, a))
        with pytest.warns(RuntimeWarning, match="has not been built"):
            with pytest.raises(ops.TraceError, match="must be CUDA tensors"):
                calls[0]()
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            for call in calls:
                with pytest.raises(ops.TraceError, match="must be CUDA tensors"):
                    call()
        with pytest.raises(ops.TraceError, match="has not been built"):
            ops.binding()
    assert ops.binding().sort(ids, 4) is None and ops._bind is ops.binding()
