"""Refusals of the FP4 expert operators, before any CUDA call (no GPU), and
the size queries."""
from __future__ import annotations

import ctypes

import pytest
import torch

from fp4_quantization_aware_trace_b200 import _build, ops

P = ctypes.c_void_p
A = P(1 << 20)            # aligned fake pointers: never dereferenced
ODD = P((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ops.library()


def test_sort_workspace_query(lib):
    f = ops.trace_moe_sort_workspace_bytes
    assert f(0, 8, 128) == 256 and f(512, 8, 128) == 256
    assert f(513, 8, 128) == -(-2 * 129 * 4 // 256) * 256
    for bad in [(-1, 8, 4), (4, 0, 4), (4, 8, 0), (4, 8, 4097), (1 << 31, 1, 4), (1 << 30, 2, 4),
                (4, 65537, 4)]:
        assert f(*bad) == 0


def test_sort_refusals(lib):
    f = lib.trace_moe_sort
    assert f(A, 4, -1, 8, 4, A, A, A, A, 256, None) == 2
    assert f(A, 4, 4, 0, 4, A, A, A, A, 256, None) == 2
    assert f(A, 2, 4, 8, 4, A, A, A, A, 256, None) == 2
    assert f(A, 4, 4, 8, 4097, A, A, A, A, 256, None) == 2
    assert f(A, 4, 1 << 30, 2, 4, A, A, A, A, 256, None) == 2
    assert f(None, 4, 4, 8, 4, A, A, A, A, 256, None) == 1
    assert f(A, 4, 4, 8, 4, A, A, A, None, 256, None) == 1
    assert f(P((1 << 20) + 4), 8, 4, 8, 4, A, A, A, A, 256, None) == 3
    assert f(A, 4, 4, 8, 4, P((1 << 20) + 4), A, A, A, 256, None) == 3
    assert f(A, 4, 4, 8, 4, A, A, A, A, 255, None) == 4


def test_token_refusals(lib):
    d, c, b = lib.trace_moe_dispatch, lib.trace_moe_combine, lib.trace_moe_combine_bwd
    assert d(A, 4, 2, 48, A, A, A, None) == 2 and c(A, 4, 2, 0, A, A, A, None) == 2
    assert d(A, -1, 2, 32, A, A, A, None) == 2 and b(A, A, 1 << 31, 1, 32, A, A, A, A, A, None) == 2
    assert d(None, 4, 2, 32, A, A, A, None) == 1 and c(A, 4, 2, 32, None, A, A, None) == 1
    assert b(A, A, 4, 2, 32, A, A, None, A, A, None) == 1
    assert d(P((1 << 20) + 16), 4, 2, 32, A, A, A, None) == 3
    assert c(A, 4, 2, 32, A, ODD, A, None) == 3
    assert b(A, A, 4, 2, 32, A, A, A, P((1 << 20) + 16), A, None) == 3
    assert d(None, 0, 2, 32, None, None, None, None) == 0


def test_product_refusals(lib):
    def nv(rows=4, cols=64, groups=1, offs=None, la=0, n=8, mats=1, lw=0, a=A, out=A, ws=A, ag=A):
        return lib.trace_fp4_matmul(a, A, ag, rows, cols, groups, offs, la, A, ws, A, n, mats, lw,
                                    out, None)

    def mx(rows=4, cols=64, groups=1, offs=None, la=0, n=8, mats=1, lw=0, a=A, out=A):
        return lib.trace_mx_matmul(a, A, rows, cols, groups, offs, la, A, A, n, mats, lw, out, None)

    for f in (nv, mx):
        assert f(cols=48) == 2 and f(cols=0) == 2 and f(rows=-1) == 2 and f(n=0) == 2
        assert f(la=2) == 2 and f(lw=-1) == 2 and f(mats=0) == 2
        assert f(groups=2, offs=A, mats=3) == 2 and f(groups=4098, offs=A) == 2
        assert f(rows=(1 << 31) - 511) == 2 and f(n=1 << 31) == 2
        assert f(groups=4000, offs=A, n=1 << 20, mats=4000) == 2
        assert f(groups=2) == 1 and f(a=None) == 1 and f(out=None) == 1
        assert f(a=P((1 << 20) + 8)) == 3 and f(out=P((1 << 20) + 8)) == 3
        assert f(groups=2, offs=P((1 << 20) + 4)) == 3
        assert f(rows=0, a=None, out=None) == 0
    assert nv(ag=None) == 1
    assert nv(lw=1, ws=P((1 << 20) + 8)) == 3


def test_binding_refusals(lib):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    f32 = torch.ones(1)
    a = ops.Capture(u8(4 * 32), None, u8(4, 4), f32)
    m = ops.MxCapture(u8(4 * 32), None, u8(4, 2))
    flat = ops.Capture(u8(4 * 32), None, u8(512), f32)
    for call in (lambda: ops.fp4_matmul(a, a),                        # host tensors
                 lambda: ops.fp4_matmul(flat, flat),                  # cols unknown
                 lambda: ops.fp4_matmul(a, a, 48),
                 lambda: ops.fp4_matmul(a, a, 32),                    # scales of another shape
                 lambda: ops.fp4_matmul(a, m),
                 lambda: ops.mx_matmul(m, a),
                 lambda: ops.mx_matmul(m, m, groups=3),
                 lambda: ops.mx_matmul(ops.MxCapture(u8(4 * 64), None, u8(4, 2)), m),  # E4M3 codes
                 lambda: ops.moe_sort(torch.zeros(3, dtype=torch.int32), 4),
                 lambda: ops.moe_sort(torch.zeros(3, 2), 4),
                 lambda: ops.moe_sort(torch.zeros(3, 2, dtype=torch.int32), 4),
                 lambda: ops.moe_sort(torch.zeros(3, 2, dtype=torch.int32), 0)):
        with pytest.raises(ops.TraceError):
            call()
    route = ops.MoeRoute(torch.zeros(6, dtype=torch.int64), torch.zeros(3, 2, dtype=torch.int32),
                         torch.zeros(6, dtype=torch.int32))
    x, y, w = torch.zeros(3, 32).bfloat16(), torch.zeros(6, 32).bfloat16(), torch.zeros(3, 2)
    for call in (lambda: ops.moe_dispatch(x, route), lambda: ops.moe_dispatch(y, route),
                 lambda: ops.moe_dispatch(x.float(), route), lambda: ops.moe_combine(x, route, w),
                 lambda: ops.moe_combine(y, route, w.double()), lambda: ops.moe_combine(y, route, w)):
        with pytest.raises(ops.TraceError):
            call()


def test_product_workspace(lib):
    """Bytes of the tiled copies: 512 for 128 rows x 4 scale columns."""
    nv, mx = lib.trace_fp4_matmul_workspace_bytes, lib.trace_mx_matmul_workspace_bytes
    assert nv(2048, 4096, 1, 1, 4096, 1, 1) == 0                     # both tiled
    assert nv(2048, 4096, 1, 0, 4096, 1, 1) == 16 * 64 * 512
    assert nv(2048, 4096, 1, 1, 4096, 1, 0) == 32 * 64 * 512
    assert nv(2049, 4128, 1, 0, 4097, 1, 0) == (17 + 33) * 65 * 512
    assert nv(2048, 4128, 1, 1, 4096, 1, 1) == (16 + 32) * 65 * 512  # k ends inside a piece
    assert nv(4096, 4096, 4, 1, 1000, 4, 1) == 4 * 8 * 64 * 512      # matrices inside a block
    assert nv(4096, 4096, 4, 1, 1024, 4, 1) == 0
    assert mx(2048, 4096, 1, 0, 4096, 1, 0) == (16 + 32) * 32 * 512
    assert nv(128, 4096, 1, 0, 4096, 1, 0) == 0 and nv(4096, 4096, 1, 0, 128, 1, 0) == 0
    assert mx(1024, 2048, 1, 0, 2048, 1, 0) == 0                     # too small to pay
    for f in (nv, mx):
        for bad in [(-1, 64, 1, 0, 8, 1, 0), (4, 48, 1, 0, 8, 1, 0), (4, 64, 1, 2, 8, 1, 0),
                    (4, 64, 2, 0, 8, 3, 0), (4, 64, 1, 0, 0, 1, 0)]:
            assert f(*bad) == 0
    big = (2048, 4096, 1, None, 0)
    for ws, n, st in [(A, 48 * 64 * 512 - 1, 4), (P((1 << 20) + 128), 1 << 30, 3)]:
        assert lib.trace_fp4_matmul_ws(A, A, A, *big, A, A, A, 4096, 1, 0, A, ws, n, None) == st
    assert lib.trace_mx_matmul_ws(A, A, *big, A, A, 4096, 1, 0, A, A, 48 * 32 * 512 - 1, None) == 4
    assert lib.trace_fp4_matmul_ws(A, A, A, 4, 48, 1, None, 0, A, A, A, 8, 1, 0, A, A, 0, None) == 2


def test_native_calls_leave_the_unusual(lib):
    """None, and nothing asked of CUDA, for host tensors, other objects and
    other numbers of arguments."""
    b = ops.binding()
    i, h = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 32).bfloat16()
    u = torch.zeros(64, dtype=torch.uint8)
    for args in [(i, 4), (i, 4.5), (None, 4), ()]:
        assert b.sort(*args) is None
    for args in [(h, i, i.view(-1)), (1, 2, 3), (h,)]:
        assert b.dispatch(*args) is None
    for args in [(h, i, i.view(-1), torch.zeros(3, 2)), (None,) * 4, ()]:
        assert b.combine(*args) is None
    for args in [(16, 32, 1, None, u, u, None, u, u, None), (16, 0, 1, None, u, u, None, u, u, None),
                 (32, 1 << 80, 1, None, u, u, None, u, u, None), (8, 32, "x", *([None] * 7)), ()]:
        assert b.matmul(*args) is None
    with pytest.raises(TypeError):
        b.setup(1)
