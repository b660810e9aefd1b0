"""Calls of the FP4 expert operators off the usual path, on the GPU: forward-mode
differentiation, one group with bounds of its own, operands that do not fit,
scales at the ends of their range, sums in which no term may be lost."""
from __future__ import annotations

import types

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwd

import _experts as ref
from fp4_quantization_aware_trace_b200 import inputs, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = ["nvfp4", "mxfp4"]


def _gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


@pytest.fixture(params=["native", "ctypes"])
def way(request, monkeypatch):
    """Both ways of a call: the module that makes the usual one, and ops.py's own."""
    if request.param == "ctypes":
        none = lambda *a: None  # noqa: E731
        monkeypatch.setattr(ops, "_bind", types.SimpleNamespace(
            sort=none, dispatch=none, combine=none, matmul=none))
    else:
        ops.binding()
    return request.param


def _route(tokens, k, experts, seed):
    ids = torch.randint(-1, experts, (tokens, k), generator=_gen(seed))
    return ops.moe_sort(ids.to(DEV), experts)


@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(way, grad):
    """A tensor with a tangent is refused, as trace_fake_quant refuses it: no
    output comes without its derivative.  The tensors themselves still pass."""
    route = _route(6, 2, 3, 1)
    x = torch.randn(6, 64, generator=_gen(2)).bfloat16().to(DEV)
    w = torch.rand(6, 2, generator=_gen(3)).to(DEV)
    y = ops.moe_dispatch(x, route)
    with fwd.dual_level(), torch.set_grad_enabled(grad):
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))  # noqa: E731
        cache = ops.capture(x)
        for call in (lambda: ops.trace_fake_quant(dual(x), cache),
                     lambda: ops.moe_dispatch(dual(x), route),
                     lambda: ops.moe_combine(dual(y), route, w),
                     lambda: ops.moe_combine(y, route, dual(w)),
                     lambda: ops.moe_combine(dual(y), route, dual(w))):
            with pytest.raises(RuntimeError):
                call()
        assert torch.equal(ops.moe_dispatch(x, route), y)
        assert fwd.unpack_dual(ops.moe_combine(y, route, w)).tangent is None
