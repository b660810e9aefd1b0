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


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("rows,n,cols,lo,hi", [
    (70, 96, 128, 0, 41), (70, 96, 128, 13, 41), (9, 2048, 2048, 2, 5), (900, 256, 128, 101, 700),
    (900, 520, 512, 0, 513), (400, 250, 192, 399, 400), (700, 384, 256, 64, 64), (300, 129, 96, 128, 300),
    (3000, 1000, 256, 130, 2900)])
def test_one_group_with_bounds(way, fmt, tiled, rows, n, cols, lo, hi):
    """A batch that is padded around its one group: the rows in front of
    offsets[0] and from offsets[1] on are left as they were, in every form of the
    product (single CTAs, k split, pairs, pairs that would write out transposed)."""
    a = inputs.tiny_site(1, rows, cols).x_roll.to(DEV)
    w = inputs.tiny_site(2, n, cols).x_roll.to(DEV)
    offs = torch.tensor([lo, hi], dtype=torch.int64, device=DEV)
    out = torch.full((rows, n), 5.0, dtype=torch.bfloat16, device=DEV)
    if fmt == "nvfp4":
        cap = ops.capture_tiled if tiled else ops.capture
        ca, cw = cap(a), cap(w)
        whole = ops.fp4_matmul(ca, cw, cols)
        ca.offsets = offs
        ops.fp4_matmul(ca, cw, cols, out=out)
        fresh = ops.fp4_matmul(ca, cw, cols)
    else:
        cap = ops.mx_capture_tiled if tiled else ops.mx_capture
        ca, cw = cap(a), cap(w)
        whole = ops.mx_matmul(ca, cw, cols)
        ops.mx_matmul(ca, cw, cols, offsets=offs, out=out)
        fresh = ops.mx_matmul(ca, cw, cols, offsets=offs)
    s, scols = (ca.scales, cw.scales), cols // (16 if fmt == "nvfp4" else 32)
    sa, sw = (v.cpu().numpy() if v.dim() == 2 else ref.untile(v.cpu().numpy(), r, scols)
              for v, r in zip(s, (rows, n)))
    ga, gw = (ca.gscale.cpu().numpy(), cw.gscale.cpu().numpy()) if fmt == "nvfp4" else (None, None)
    exact, mag = ref.product(ref.operand(ca.codes.cpu().numpy(), sa, rows, cols, fmt),
                             ref.operand(cw.codes.cpu().numpy(), sw, n, cols, fmt), ga, gw, [0, rows], n)
    bound = ref.product_bound(exact, mag, cols)
    for got in (out, fresh):
        assert np.all(np.abs(ref.f64(got) - exact)[lo:hi] <= bound[lo:hi])
    assert np.all(np.abs(ref.f64(whole) - exact) <= bound)
    assert bool((out[:lo] == 5.0).all()) and bool((out[hi:] == 5.0).all())
    assert ops.matmul_status()


def test_operands_of_other_lengths_are_refused(way):
    """Rows of another length, whose bytes would make other rows of this one."""
    x, w = (torch.randn(r, c, generator=_gen(r)).bfloat16().to(DEV) for r, c in ((64, 128), (40, 256)))
    a, b = ops.capture(x), ops.capture(w)
    ma, mb = ops.mx_capture(x), ops.mx_capture(w)
    for call in (lambda **k: ops.fp4_matmul(a, b, **k), lambda **k: ops.fp4_matmul(b, a, **k),
                 lambda **k: ops.fp4_matmul(b, b, 128, **k), lambda **k: ops.mx_matmul(ma, mb, **k),
                 lambda **k: ops.mx_matmul(mb, mb, 512, **k)):
        for kw in ({}, {"stream": torch.cuda.current_stream()}):
            with pytest.raises(ops.TraceError):
                call(**kw)
    # one matrix per expert kept as [experts, n, cols / 16]: neither rows nor tiled
    s = b.scales
    e = ops.capture(torch.randn(4 * 64, 64, generator=_gen(1)).bfloat16().to(DEV),
                    torch.arange(5, device=DEV) * 64)
    e.scales = e.scales.view(4, 64, 4)
    t = ops.capture(torch.randn(16, 64, generator=_gen(2)).bfloat16().to(DEV),
                    torch.tensor([0, 4, 8, 12, 16], device=DEV))
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        with pytest.raises(ops.TraceError):
            ops.fp4_matmul(t, e, 64, **kw)
    assert s.dim() == 2 and ops.fp4_matmul(b, b).shape == (40, 40)


@pytest.mark.parametrize("ga,gw", [(-1e-38, 1e30), (3e35, -1e-36), (-1e30, 1e30), (-3.0, 2.0),
                                   (-1e-25, -1e-10), (1e-25, -1e-10), (2.0 ** -140, -(2.0 ** 100))])
def test_signs_of_global_scales(way, ga, gw):
    """A caller's negative global scale turns the sign at every magnitude."""
    rows, n, cols = 20, 24, 64
    g = _gen(3)
    codes = lambda r: torch.randint(0, 256, (r * cols // 2,), generator=g, dtype=torch.uint8)  # noqa: E731
    s = torch.randint(0x20, 0x50, (rows + n, cols // 16), generator=g, dtype=torch.uint8)
    a = ops.Capture(codes(rows).to(DEV), None, s[:rows].to(DEV), torch.tensor([ga], device=DEV))
    w = ops.Capture(codes(n).to(DEV), None, s[rows:].to(DEV), torch.tensor([gw], device=DEV))
    out = ref.f64(ops.fp4_matmul(a, w))
    wide = ref.operand(a.codes.cpu().numpy(), s[:rows].numpy(), rows, cols, "nvfp4")
    tall = ref.operand(w.codes.cpu().numpy(), s[rows:].numpy(), n, cols, "nvfp4")
    exact, mag = ref.product(wide, tall, a.gscale.cpu().numpy(), w.gscale.cpu().numpy(), [0, rows], n)
    over, inside = np.abs(exact) > 3.4e38, np.abs(exact) < 3.3e38
    bound = ref.product_bound(exact, np.abs(mag), cols)
    assert np.all(out[over] == np.sign(exact[over]) * np.inf)
    assert np.all(np.abs(out - exact)[inside] <= bound[inside])


def test_status_of_products_from_several_threads():
    """Each thread and stream asks for itself, while products run on both."""
    import threading
    a = ops.capture_tiled(inputs.tiny_site(1, 300, 512).x_roll.to(DEV))
    w = ops.capture_tiled(inputs.tiny_site(2, 384, 512).x_roll.to(DEV))
    said = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(50):
            ops.fp4_matmul(a, w, 512, stream=s)
            said.append(ops.matmul_status(s))
        said.append(ops.matmul_status())

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(said) == 4 * 51 and all(said)


@pytest.mark.parametrize("rows,n,cols", [(20, 24, 64), (5, 256, 1024), (300, 264, 320)])
@pytest.mark.parametrize("ea,ew", [(0xF0, 0x0E), (0xFE, 0x00), (0x00, 0xFE), (0x40, 0x3F), (0x3C, 0x3B),
                                   (0xC0, 0xC4), (0xFE, 0xFE), (0x00, 0x00), (0x7F, 0x05), (0x20, 0x20)])
def test_mx_scales_at_the_ends_of_their_range(way, rows, n, cols, ea, ew):
    """Block scales of 2^-127 to 2^127: large against small ones with ordinary
    sums, sums in and below bf16's subnormal range, and sums past its end.  A block's
    two scales move by +-2 around ea and ew in opposite directions, so that the
    terms of a sum are of like size."""
    g = _gen(ea * 256 + ew)
    c = cols // 32
    codes = lambda r: torch.randint(0, 256, (r, cols // 2), generator=g, dtype=torch.uint8)  # noqa: E731
    step = torch.randint(-2, 3, (c,), generator=g)
    sa = (torch.full((rows, c), ea) + step).clamp(0, 254).to(torch.uint8)
    sw = (torch.full((n, c), ew) - step).clamp(0, 254).to(torch.uint8)
    a = ops.MxCapture(codes(rows).to(DEV), None, sa.to(DEV))
    w = ops.MxCapture(codes(n).to(DEV), None, sw.to(DEV))
    out = ref.f64(ops.mx_matmul(a, w))
    va = ref.operand(a.codes.cpu().numpy(), sa.numpy(), rows, cols, "mxfp4")
    vw = ref.operand(w.codes.cpu().numpy(), sw.numpy(), n, cols, "mxfp4")
    exact, mag = ref.product(va, vw, None, None, [0, rows], n)
    # as product_bound, and a term below fp32's normal range is off by one unit of its
    # subnormals, 2^-149
    bound = ref.product_bound(exact, mag, cols) + cols * 2.0 ** -149
    over, inside = np.abs(exact) - bound > 3.4e38, mag < 3.3e38
    assert np.all(np.abs(out - exact)[inside] <= bound[inside])
    assert np.all(~np.isfinite(out[over]))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("rows,n,cols,counts", [
    (1, 4096, 4096, None), (29, 300, 8224, None), (140, 136, 4128, None), (700, 520, 4160, None),
    (600, 389, 4096, None), (64, 256, 4096, [20, 1, 43]), (900, 256, 4128, [300, 2, 598])])
def test_no_term_of_a_long_sum_is_lost(way, fmt, tiled, rows, n, cols, counts):
    """Codes of -1, 0 and 1 and block scales that are powers of two and cancel
    between the operands: sums of whole numbers up to 256, exact in fp32 in any
    order and in bf16, so a lost or doubled term shows."""
    g = _gen(rows + n + cols)
    bs = 16 if fmt == "nvfp4" else 32
    matrices = 1 if counts is None else len(counts)
    bounds = [0, rows] if counts is None else np.concatenate([[0], np.cumsum(counts)]).tolist()

    def draw(r):
        v = torch.randint(-1, 2, (r, cols), generator=g)
        v[torch.rand(r, cols, generator=g) < 0.4] = 0
        nib = torch.where(v > 0, 2, torch.where(v < 0, 10, 0)).to(torch.uint8)
        return v.float().to(DEV), (nib[:, 0::2] | nib[:, 1::2] << 4).reshape(-1).contiguous().to(DEV)

    (va, ca), (vw, cw) = draw(rows), draw(matrices * n)
    p = torch.randint(-3, 4, (cols // bs,), generator=g)
    one, unit = (0x38, 8) if fmt == "nvfp4" else (127, 1)
    sa = (one + unit * p).to(torch.uint8).expand(rows, -1).contiguous()
    sw = (one - unit * p).to(torch.uint8).expand(matrices * n, -1).contiguous()
    if tiled:
        sa, sw = (torch.from_numpy(ref.tile(s.numpy(), 0xFF)) for s in (sa, sw))
    sa, sw = sa.to(DEV), sw.to(DEV)
    offs = None if counts is None else torch.tensor(bounds, device=DEV)
    if fmt == "nvfp4":
        one = torch.ones(matrices, device=DEV)
        out = ops.fp4_matmul(ops.Capture(ca, None, sa, one, offs), ops.Capture(cw, None, sw, one), cols)
    else:
        out = ops.mx_matmul(ops.MxCapture(ca, None, sa), ops.MxCapture(cw, None, sw), cols, offs, matrices)
    for e in range(matrices):
        lo, hi = bounds[e], bounds[e + 1]
        want = va[lo:hi].double() @ vw[e * n:(e + 1) * n].double().t()
        assert want.numel() == 0 or want.abs().max() <= 256
        assert torch.equal(out[lo:hi].double(), want)


def test_calls_under_inference_mode(way):
    """The chain of a rollout without autograd, on tensors that have no version, and
    on a route of theirs outside of it."""
    x = torch.randn(37, 64, generator=_gen(2)).bfloat16().to(DEV)
    w = torch.rand(37, 3, generator=_gen(3)).to(DEV)
    plain = _route(37, 3, 5, 1)
    want = ops.moe_combine(ops.moe_dispatch(x, plain), plain, w)
    with torch.inference_mode():
        route = _route(37, 3, 5, 1)
        out = ops.moe_combine(ops.moe_dispatch(x, route), route, w)
        a, b = ops.capture(x), ops.capture(x[:8].contiguous())
        product = ops.fp4_matmul(a, b)
    assert out.is_inference() and torch.equal(out, want)
    assert torch.equal(product, ops.fp4_matmul(a, b))
    assert torch.equal(ops.moe_combine(ops.moe_dispatch(x, route), route, w), want)
    with torch.no_grad():
        xg = x.clone().requires_grad_()
        assert not ops.moe_combine(ops.moe_dispatch(xg, plain), plain, w).requires_grad
