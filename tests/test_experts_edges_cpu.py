"""The FP4 expert operators' host side off the usual path (no GPU)."""
from __future__ import annotations

import os
import subprocess

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
