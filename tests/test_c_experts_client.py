"""The expert operators from plain C: tests/c_experts_client.c (no Python, no
torch) is compiled with gcc against include/trace_fp4.h and libtrace_fp4.so; on a
GPU it runs a layer whose outputs are compared with plain forms."""
from __future__ import annotations

import os
import subprocess

import numpy as np
import pytest

import _experts as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "fp4_quantization_aware_trace_b200")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
T, K, E, COLS, N, BACK = 50, 3, 4, 192, 72, 64
S = T * K


def _build(tmp_path) -> str:
    exe = str(tmp_path / "c_experts_client")
    subprocess.run(["gcc", "-O2", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(CUDA, "include"), os.path.join(ROOT, "tests", "c_experts_client.c"),
                    "-L", PKG, "-ltrace_fp4", "-L", os.path.join(CUDA, "lib64"), "-lcudart",
                    f"-Wl,-rpath,{PKG}:{os.path.join(CUDA, 'lib64')}", "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def test_client_compiles_and_links(tmp_path):
    assert os.path.exists(_build(tmp_path))


def _bf16(words):
    return (words.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


@pytest.mark.gpu
def test_a_layer_of_experts_from_c(tmp_path, oracle_mod):
    out_file = tmp_path / "client.bin"
    r = subprocess.run([_build(tmp_path), str(out_file)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    buf, pos = out_file.read_bytes(), 0

    def take(dtype, *shape):
        nonlocal pos
        a = np.frombuffer(buf, dtype=dtype, count=int(np.prod(shape)), offset=pos).reshape(shape)
        pos += a.nbytes
        return a

    ids, p = take(np.int32, T, K), take(np.float32, T, K).astype(np.float64)
    x, w = take(np.uint16, T, COLS), take(np.uint16, E * N, COLS)
    offsets, rows, slots = take(np.int64, E + 2), take(np.int32, T, K), take(np.int32, S)
    y = take(np.uint16, S, COLS)
    ac, asc, ag = take(np.uint8, S * COLS // 2), take(np.uint8, 2 * 3 * 512), take(np.float32, E + 1)
    wc, wsc, wg = take(np.uint8, E * N * COLS // 2), take(np.uint8, E * N, COLS // 16), take(np.float32, E)
    first, second = take(np.uint16, S, N), take(np.uint16, S, N)
    out = _bf16(take(np.uint16, T * N)[:T * BACK]).reshape(T, BACK)
    gy = _bf16(take(np.uint16, S * N)[:S * BACK]).reshape(S, BACK)
    gp = take(np.float32, T, K)
    assert pos == len(buf)

    for got, want in zip((offsets, rows, slots), ref.sort(ids, E)):
        assert np.array_equal(got, want)
    live = slots >= 0
    assert np.array_equal(y[live], x[slots[live] // K]) and not y[~live].any()
    codes, _, scales, gscale = oracle_mod.capture(np.ascontiguousarray(y), E + 1, offsets.copy())
    asc = ref.untile(asc, S, COLS // 16)
    assert np.array_equal(ac, codes) and np.array_equal(asc.reshape(-1), np.asarray(scales).reshape(-1))
    assert np.array_equal(ag, np.asarray(gscale))
    codes, _, scales, gscale = oracle_mod.capture(w.copy(), E, np.arange(E + 1, dtype=np.int64) * N)
    assert np.array_equal(wc, codes) and np.array_equal(wsc.reshape(-1), np.asarray(scales).reshape(-1))
    assert np.array_equal(wg, np.asarray(gscale))
    exact, mag = ref.product(ref.operand(ac, asc, S, COLS, "nvfp4"), ref.operand(wc, wsc, E * N, COLS, "nvfp4"),
                             ag, wg, offsets.tolist(), N)
    for got in (first, second):
        assert np.all(np.abs(_bf16(got) - exact) <= ref.product_bound(exact, mag, COLS))
    # back to token order and its gradients, of the first 64 columns: K steps in fp32
    # and a rounding; one product and a rounding; a sum of 64 exact products in fp32
    yr = np.where((rows >= 0)[..., None], _bf16(first)[:, :BACK][np.maximum(rows, 0)], 0.0)
    terms = yr * p[..., None]
    want, m = terms.sum(1), np.abs(terms).sum(1)
    assert np.all(np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * K * 2.0 ** -24 * m)
    want = np.zeros((S, BACK))
    want[live] = out[slots[live] // K] * p.reshape(-1)[slots[live]][:, None]
    assert np.all(np.abs(gy - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -134)
    dots = out[:, None, :] * yr
    assert np.all(np.abs(gp - dots.sum(-1)) <= (BACK + 5) * 2.0 ** -24 * np.abs(dots).sum(-1))
