"""The FP4 expert operators on the GPU against plain 64-bit forms: routing
sort, dispatch, combine with their gradients, the product of captured
operands, and a whole expert layer of them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import _experts as ref
from fp4_quantization_aware_trace_b200 import inputs, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# Sort
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,experts", [
    (1, 1, 1), (1, 8, 128), (3, 2, 5), (37, 8, 128), (511, 8, 128), (512, 8, 128), (513, 8, 128),
    (4096, 1, 4096), (4099, 3, 7), (1000, 5, 4096), (20001, 8, 300)])
def test_sort(tokens, k, experts, dtype):
    g = _gen(tokens * 31 + k + experts)
    ids = torch.randint(-1, experts + 1, (tokens, k), generator=g).to(dtype)  # both ends are dropped
    if dtype == torch.int64 and tokens > 2:
        ids[1, 0] = (1 << 40) + min(3, experts - 1)  # in range only in its low word
        ids[2, 0] = -(1 << 40) + min(3, experts - 1)
    route = ops.moe_sort(ids.to(DEV), experts)
    offsets, rows, slots = ref.sort(ids.numpy(), experts)
    assert np.array_equal(route.offsets.cpu().numpy(), offsets)
    assert np.array_equal(route.rows.cpu().numpy(), rows)
    assert np.array_equal(route.slots.cpu().numpy(), slots)
    assert ops.validate_offsets(route.offsets, tokens * k) == 0


@pytest.mark.parametrize("fill", [-1, 0, 6])
def test_sort_one_value(fill):
    """Every slot dropped; every slot to the first or the last expert."""
    ids = torch.full((2500, 4), fill, dtype=torch.int32)
    route = ops.moe_sort(ids.to(DEV), 7)
    for got, want in zip((route.offsets, route.rows, route.slots), ref.sort(ids.numpy(), 7)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_no_tokens():
    route = ops.moe_sort(torch.empty(0, 8, dtype=torch.int64, device=DEV), 16)
    assert route.offsets.tolist() == [0] * 18 and route.rows.shape == (0, 8)


def test_sort_reuses_a_dirty_workspace_and_outputs():
    ids = torch.randint(0, 40, (3000, 8), generator=_gen(5), dtype=torch.int32)
    ws = torch.full((ops.trace_moe_sort_workspace_bytes(3000, 8, 40),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    route = None
    for seed in (1, 2):
        ids = torch.randint(0, 40, (3000, 8), generator=_gen(seed), dtype=torch.int32)
        route = ops.moe_sort(ids.to(DEV), 40, out=route, workspace=ws)
        for got, want in zip((route.offsets, route.rows, route.slots), ref.sort(ids.numpy(), 40)):
            assert np.array_equal(got.cpu().numpy(), want)


# ---------------------------------------------------------------------------
# Dispatch and combine
# ---------------------------------------------------------------------------

def _route(tokens, k, experts, seed, dropped=0.2):
    g = _gen(seed)
    ids = torch.randint(0, experts, (tokens, k), generator=g)
    ids[torch.rand(tokens, k, generator=g) < dropped] = -1
    return ops.moe_sort(ids.to(DEV), experts), ref.sort(ids.numpy(), experts)


TOKEN_CASES = [(1, 1, 32, 1), (1, 8, 2048, 128), (7, 3, 96, 4), (33, 8, 544, 16), (130, 1, 512, 8),
               (257, 9, 1056, 64)]


@pytest.mark.parametrize("tokens,k,cols,experts", TOKEN_CASES)
def test_dispatch_and_its_gradient(tokens, k, cols, experts):
    route, (offsets, rows, slots) = _route(tokens, k, experts, 11 * tokens + k)
    g = _gen(tokens)
    x = torch.randn(tokens, cols, generator=g).to(torch.bfloat16)
    dy = torch.randn(tokens * k, cols, generator=g).to(torch.bfloat16)
    xg = x.to(DEV).requires_grad_()
    y = ops.moe_dispatch(xg, route)
    want = np.zeros((tokens * k, cols))
    live = slots >= 0
    want[live] = ref.f64(x)[slots[live] // k]
    assert np.array_equal(ref.f64(y), want)
    (dx,) = torch.autograd.grad(y, xg, dy.to(DEV))
    d = ref.f64(dy)
    parts = np.where((rows >= 0)[..., None], d[np.maximum(rows, 0)], 0.0)
    exact, mag = parts.sum(1), np.abs(parts).sum(1)
    # k additions in fp32 and one rounding to bf16
    err = np.abs(ref.f64(dx) - exact)
    assert np.all(err <= 2.0 ** -8 * np.abs(exact) + (1 + 2.0 ** -8) * k * 2.0 ** -24 * mag)


@pytest.mark.parametrize("tokens,k,cols,experts", TOKEN_CASES)
def test_combine_and_its_gradients(tokens, k, cols, experts):
    route, (offsets, rows, slots) = _route(tokens, k, experts, 13 * tokens + k)
    g = _gen(tokens + 1)
    y = torch.randn(tokens * k, cols, generator=g).to(torch.bfloat16)
    w = torch.softmax(torch.randn(tokens, k, generator=g), 1)
    do = torch.randn(tokens, cols, generator=g).to(torch.bfloat16)
    # what dropped slots hold must not matter
    yb, wb = y.clone(), w.clone()
    yb[torch.from_numpy(slots < 0)] = float("nan")
    wb[torch.from_numpy(rows < 0)] = float("inf")
    yg, wg = yb.to(DEV).requires_grad_(), wb.to(DEV).requires_grad_()
    out = ops.moe_combine(yg, route, wg)
    dyg, dwg = torch.autograd.grad(out, (yg, wg), do.to(DEV))
    live = rows >= 0
    yr = np.where(live[..., None], ref.f64(y)[np.maximum(rows, 0)], 0.0)
    terms = yr * ref.f64(w)[..., None]
    exact, mag = terms.sum(1), np.abs(terms).sum(1)
    err = np.abs(ref.f64(out) - exact)
    # k fused multiply-adds in fp32 and one rounding to bf16
    assert np.all(err <= 2.0 ** -8 * np.abs(exact) + (1 + 2.0 ** -8) * k * 2.0 ** -24 * mag)
    # dweights: products exact in fp32 (8 x 8 bits), at most cols + 5 additions
    dots = ref.f64(do)[:, None, :] * yr
    dw, dmag = dots.sum(-1), np.abs(dots).sum(-1)
    assert np.all(np.abs(ref.f64(dwg) - dw) <= (cols + 5) * 2.0 ** -24 * dmag)
    # grad_y: one product in fp32, one rounding to bf16
    dy = np.zeros((tokens * k, cols))
    s = slots[slots >= 0]
    dy[slots >= 0] = ref.f64(do)[s // k] * ref.f64(w).reshape(-1)[s][:, None]
    assert np.all(np.abs(ref.f64(dyg) - dy) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(dy) + 2.0 ** -134)


def test_gradients_against_differences():
    """Small whole numbers, so that every sum is exact and a difference
    quotient of the (linear) forward is the gradient."""
    tokens, k, cols, experts = 5, 3, 64, 4
    route, _ = _route(tokens, k, experts, 3)
    g = _gen(4)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).float().to(DEV)  # noqa: E731
    x, y = ints(tokens, cols).bfloat16(), ints(tokens * k, cols).bfloat16()
    w, do, dyy = ints(tokens, k), ints(tokens, cols).bfloat16(), ints(tokens * k, cols).bfloat16()
    xg = x.clone().requires_grad_()
    (dx,) = torch.autograd.grad(ops.moe_dispatch(xg, route), xg, dyy)
    yg, wg = y.clone().requires_grad_(), w.clone().requires_grad_()
    dy, dw = torch.autograd.grad(ops.moe_combine(yg, route, wg), (yg, wg), do)

    def slope(f, v, grad_out, at):
        hi = v.clone()
        hi.view(-1)[at] += 1
        return ((f(hi).double() - f(v).double()) * grad_out.double()).sum().item()

    for at in (0, 17, tokens * cols - 1):
        assert slope(lambda v: ops.moe_dispatch(v, route), x, dyy, at) == dx.view(-1)[at].item()
    for at in (0, 129, tokens * k * cols - 1):
        assert slope(lambda v: ops.moe_combine(v, route, w), y, do, at) == dy.view(-1)[at].item()
    for at in range(tokens * k):
        assert slope(lambda v: ops.moe_combine(y, route, v), w, do, at) == dw.view(-1)[at].item()


def test_gradients_of_views_and_shared_leaves():
    """An expanded (stride 0) upstream gradient; the same tokens dispatched twice."""
    route, (_, rows, _) = _route(9, 2, 4, 21)
    x = torch.ones(9, 64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    a, b = ops.moe_dispatch(x, route), ops.moe_dispatch(x, route)
    (a.sum() + 2 * b.sum()).backward()
    want = 3.0 * (rows >= 0).sum(1)
    assert np.array_equal(ref.f64(x.grad), np.repeat(want[:, None], 64, 1))


def test_bad_route_entries_are_skipped():
    """Entries outside the rows: no access, no term."""
    route, _ = _route(6, 2, 3, 8, dropped=0.0)
    y = torch.ones(12, 64, dtype=torch.bfloat16, device=DEV)
    rows = route.rows.clone()
    rows[2, 0], rows[3, 1] = 12, 2 ** 31 - 1
    bad = ops.MoeRoute(route.offsets, rows, route.slots)
    out = ops.moe_combine(y, bad, torch.ones(6, 2, device=DEV))
    assert out[:, 0].tolist() == [2, 2, 1, 1, 2, 2]


# ---------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------

def _capture(x, fmt, tiled, offsets=None):
    if fmt == "nvfp4":
        return ops.capture_tiled(x, offsets) if tiled else ops.capture(x, offsets)
    return ops.mx_capture_tiled(x) if tiled else ops.mx_capture(x)


def _operand(cap, rows, cols, fmt):
    scols = cols // (16 if fmt == "nvfp4" else 32)
    s = cap.scales.cpu().numpy()
    s = s if s.ndim == 2 else ref.untile(s, rows, scols)
    return ref.operand(cap.codes.cpu().numpy(), s, rows, cols, fmt)


def _poison(cap, rows, cols, fmt):
    """NaN bytes in the padding of a tiled scale array."""
    scols = cols // (16 if fmt == "nvfp4" else 32)
    s = ref.untile(cap.scales.cpu().numpy(), rows, scols)
    cap.scales = torch.from_numpy(ref.tile(s, 0xFF)).to(DEV)


def _matmul(a, w, cols, fmt, offsets, groups, out=None, stream=None):
    if fmt == "nvfp4":
        return ops.fp4_matmul(a, w, cols, out=out, stream=stream)
    return ops.mx_matmul(a, w, cols, offsets=offsets, groups=groups, out=out, stream=stream)


def _product_case(rows, n, cols, fmt, tiled_a, tiled_w, counts=None, seed=0):
    """counts: rows of each group; the last one of a `None`-terminated list
    has no matrix."""
    matrices = 1
    offs = None
    if counts is not None:
        matrices = len(counts) - (1 if counts[-1] is None else 0)
        known = [c for c in counts if c is not None]
        bounds = np.concatenate([[0], np.cumsum(known)])
        if counts[-1] is None:
            bounds = np.concatenate([bounds, [rows]])
        assert bounds[-1] == rows
        offs = torch.from_numpy(bounds.astype(np.int64)).to(DEV)
    a = inputs.tiny_site(seed + 1, rows, cols).x_roll.to(DEV)
    w = (0.05 * inputs.tiny_site(seed + 2, matrices * n, cols).x_roll.float()).bfloat16().to(DEV)
    wo = torch.arange(matrices + 1, dtype=torch.int64, device=DEV) * n if matrices > 1 else None
    ca, cw = _capture(a, fmt, tiled_a, offs), _capture(w, fmt, tiled_w, wo)
    for cap, r, t in ((ca, rows, tiled_a), (cw, matrices * n, tiled_w)):
        if t:
            _poison(cap, r, cols, fmt)
    pad = 4096
    buf = torch.full((rows * n + 2 * pad,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[pad:pad + rows * n].view(rows, n)
    _matmul(ca, cw, cols, fmt, offs, matrices, out=out)
    ga = ca.gscale.cpu().numpy() if fmt == "nvfp4" else None
    gw = cw.gscale.cpu().numpy() if fmt == "nvfp4" else None
    bounds = [0, rows] if offs is None else offs.tolist()
    exact, mag = ref.product(_operand(ca, rows, cols, fmt), _operand(cw, matrices * n, cols, fmt),
                             ga, gw, bounds, n)
    err = np.abs(ref.f64(out) - exact)
    bound = ref.product_bound(exact, mag, cols)
    assert np.all(err <= bound), (int(np.sum(~(err <= bound))), np.argwhere(~(err <= bound))[:4],
                                  float(np.nanmax(err - bound)))
    edge = torch.cat([buf[:pad], buf[pad + rows * n:]])
    assert bool((edge == 7.0).all())


FORMATS = ["nvfp4", "mxfp4"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,cols", [
    (1, 1, 32), (1, 128, 64), (1, 4096, 2048), (2, 130, 96), (3, 8, 4096), (16, 256, 256),
    (17, 129, 160), (29, 2048, 1024), (33, 40, 288), (64, 384, 512), (65, 127, 544),
    (128, 128, 128), (129, 257, 320), (200, 1000, 768), (256, 512, 2048), (300, 264, 1056),
    (1000, 640, 224), (2049, 136, 1024)])
def test_product(fmt, rows, n, cols):
    _product_case(rows, n, cols, fmt, rows % 2 == 0, n % 2 == 0, seed=rows + n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled_a", [False, True])
@pytest.mark.parametrize("tiled_w", [False, True])
def test_product_layouts(fmt, tiled_a, tiled_w):
    for cols in (352, 512):
        _product_case(150, 200, cols, fmt, tiled_a, tiled_w, seed=cols)


GROUPS = [
    [5], [0, 7], [7, 0], [1] * 9, [3, 0, 0, 130, 1, 64], [128, 128, 256], [127, 129, 0, 1, 255],
    [300, 2, 17], [4, 9, None], [0, 0, None], [40, None], [16] * 24]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", GROUPS, ids=str)
@pytest.mark.parametrize("n,cols,tiled", [(136, 288, True), (128, 512, True), (72, 96, False)])
def test_grouped_product(fmt, counts, n, cols, tiled):
    rows = sum(c for c in counts if c is not None) + (21 if counts[-1] is None else 0)
    _product_case(rows, n, cols, fmt, tiled, tiled, counts, seed=len(counts) + rows)


def test_grouped_product_many_groups():
    g = _gen(77)
    counts = torch.randint(0, 6, (1024,), generator=g).tolist()
    counts[500] = 300
    _product_case(sum(counts), 40, 64, "nvfp4", True, True, counts, seed=9)


def test_product_rows_behind_the_last_group_are_left():
    rows, n, cols = 70, 96, 128
    a = inputs.tiny_site(1, rows, cols).x_roll.to(DEV)
    w = inputs.tiny_site(2, 2 * n, cols).x_roll.to(DEV)
    offs = torch.tensor([0, 30, 70], dtype=torch.int64, device=DEV)
    ca = ops.capture(a, offs)
    cw = ops.capture(w, torch.tensor([0, n, 2 * n], dtype=torch.int64, device=DEV))
    whole = ops.fp4_matmul(ca, cw)
    out = torch.full((rows, n), 5.0, dtype=torch.bfloat16, device=DEV)
    ca.offsets = torch.tensor([0, 30, 41], dtype=torch.int64, device=DEV)
    ops.fp4_matmul(ca, cw, out=out)
    assert torch.equal(out[:41], whole[:41]) and bool((out[41:] == 5.0).all())


@pytest.mark.parametrize("ga,gw", [(1e-38, 1e30), (3e35, 1e-36), (1e-20, 1e-20), (1e30, 1e30),
                                   (2.0 ** -140, 2.0 ** 100)])
def test_product_extreme_global_scales(ga, gw):
    """The product of the scales may leave fp32's range where the output does not."""
    rows, n, cols = 20, 24, 64
    g = _gen(3)
    codes = lambda r: torch.randint(0, 256, (r * cols // 2,), generator=g, dtype=torch.uint8)  # noqa: E731
    ac, wc = codes(rows).to(DEV), codes(n).to(DEV)
    s = torch.randint(0x20, 0x50, (rows + n, cols // 16), generator=g, dtype=torch.uint8).to(DEV)
    a = ops.Capture(ac, None, s[:rows].contiguous(), torch.tensor([ga], device=DEV))
    w = ops.Capture(wc, None, s[rows:].contiguous(), torch.tensor([gw], device=DEV))
    out = ref.f64(ops.fp4_matmul(a, w))
    exact, mag = ref.product(_operand(a, rows, cols, "nvfp4"), _operand(w, n, cols, "nvfp4"),
                             a.gscale.cpu().numpy(), w.gscale.cpu().numpy(), [0, rows], n)
    over = np.abs(exact) > 3.3e38
    inside = np.abs(exact) < 3.3e38
    bound = ref.product_bound(exact, mag, cols)
    assert np.all(np.isinf(out[over]))
    assert np.all(np.abs(out - exact)[inside] <= bound[inside])


def test_product_of_the_largest_and_of_zero_codes():
    """Every term at its largest (6 * 448 each side), and operands of zeros."""
    rows, n, cols = 5, 136, 4096
    full = lambda r: torch.full((r * cols // 2,), 0x77, dtype=torch.uint8, device=DEV)  # noqa: E731
    top = lambda r: torch.full((r, cols // 16), 0x7E, dtype=torch.uint8, device=DEV)  # noqa: E731
    one = torch.ones(1, device=DEV)
    a = ops.Capture(full(rows), None, top(rows), one)
    w = ops.Capture(full(n), None, top(n), one)
    want = torch.tensor(float(cols * 2688 ** 2)).bfloat16().item()
    assert bool((ops.fp4_matmul(a, w) == want).all())
    a.scales = torch.zeros_like(a.scales)
    assert bool((ops.fp4_matmul(a, w) == 0).all())
    z = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    assert bool((ops.fp4_matmul(ops.capture(z), w) == 0).all())
    assert bool((ops.mx_matmul(ops.mx_capture(z), ops.mx_capture(z)) == 0).all())


def test_product_no_rows():
    a = ops.Capture(torch.empty(0, dtype=torch.uint8, device=DEV), None,
                    torch.empty(0, 4, dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV))
    w = ops.capture(inputs.tiny_site(2, 40, 64).x_roll.to(DEV))
    assert ops.fp4_matmul(a, w).shape == (0, 40)


def test_product_repeats_bit_for_bit_and_on_two_streams():
    rows, n, cols = 40, 1024, 4096
    a = ops.capture_tiled(inputs.tiny_site(1, rows, cols).x_roll.to(DEV))
    w = ops.capture_tiled(inputs.tiny_site(2, n, cols).x_roll.to(DEV))
    first = ops.fp4_matmul(a, w, cols)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [ops.fp4_matmul(a, w, cols, stream=s) for _ in range(8) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

def _layer(x, ids, weights, w, experts, n, cols):
    route = ops.moe_sort(ids, experts)
    xs = ops.moe_dispatch(x, route)
    a = ops.capture_tiled(xs, route.offsets)
    y = ops.fp4_matmul(a, w, cols)
    return ops.moe_combine(y, route, weights), route, a, y


@pytest.mark.parametrize("tokens", [1, 45, 300])
def test_expert_layer(tokens):
    """Sort, dispatch, capture, grouped product, combine, as a rollout runs
    them, against 64 bits from capture's codes; then captured into a graph
    and replayed on other inputs."""
    k, experts, n, cols = 4, 12, 160, 256
    g = _gen(tokens)
    ids = torch.stack([torch.randperm(experts, generator=g)[:k] for _ in range(tokens)]).int()
    if tokens > 8:
        ids[5:9] = -1
    x = torch.randn(tokens, cols, generator=g).bfloat16()
    weights = torch.softmax(torch.randn(tokens, k, generator=g), 1)
    wt = (0.1 * torch.randn(experts * n, cols, generator=g)).bfloat16().to(DEV)
    w = ops.capture_tiled(wt, torch.arange(experts + 1, dtype=torch.int64, device=DEV) * n)
    args = [v.to(DEV) for v in (x, ids, weights)]
    out, route, a, y = _layer(*args, w, experts, n, cols)

    def check(out, route, a, y, weights):
        bounds = route.offsets.tolist()
        exact, mag = ref.product(_operand(a, tokens * k, cols, "nvfp4"),
                                 _operand(w, experts * n, cols, "nvfp4"), a.gscale.cpu().numpy(),
                                 w.gscale.cpu().numpy(), bounds, n)
        assert np.all(np.abs(ref.f64(y) - exact) <= ref.product_bound(exact, mag, cols))
        rows = route.rows.cpu().numpy()
        terms = np.where((rows >= 0)[..., None], ref.f64(y)[np.maximum(rows, 0)], 0.0) \
            * ref.f64(weights)[..., None]
        s, m = terms.sum(1), np.abs(terms).sum(1)
        assert np.all(np.abs(ref.f64(out) - s) <= 2.0 ** -8 * np.abs(s)
                      + (1 + 2.0 ** -8) * k * 2.0 ** -24 * m)

    check(out, route, a, y, weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        _layer(*args, w, experts, n, cols)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            held = _layer(*args, w, experts, n, cols)
    torch.cuda.synchronize()
    for seed in (1, 2):
        g = _gen(100 + seed)
        args[0].copy_(torch.randn(tokens, cols, generator=g).bfloat16())
        args[1].copy_(torch.randint(0, experts, (tokens, k), generator=g).int())
        graph.replay()
        torch.cuda.synchronize()
        check(*held, weights)


def test_training_layer_gradients():
    """Dispatch, guided fake-quant against the rollout's capture, an expert
    product in torch, combine: gradients reach tokens, weights and the
    router's weights, and equal those of the plain composition."""
    tokens, k, experts, n, cols = 24, 2, 3, 64, 64
    route, (offsets, rows, slots) = _route(tokens, k, experts, 6, dropped=0.1)
    g = _gen(9)
    x = torch.randn(tokens, cols, generator=g).bfloat16().to(DEV).requires_grad_()
    w = (0.2 * torch.randn(experts, n, cols, generator=g)).bfloat16().to(DEV).requires_grad_()
    p = torch.softmax(torch.randn(tokens, k, generator=g), 1).to(DEV).requires_grad_()
    cache = ops.capture(ops.moe_dispatch(x.detach(), route), route.offsets)
    xs = ops.moe_dispatch(x, route)
    q = ops.trace_fake_quant(xs, cache)
    parts = [q[offsets[e]:offsets[e + 1]] @ w[e].t() for e in range(experts)]
    y = torch.cat(parts + [q.new_zeros(int(offsets[-1] - offsets[-2]), n)])
    out = ops.moe_combine(y, route, p)
    do = torch.randn(tokens, n, generator=g).bfloat16().to(DEV)
    dx, dw, dp = torch.autograd.grad(out, (x, w, p), do)
    # the same steps by hand from the library's own intermediate values
    d = ref.f64(do)
    live = rows >= 0
    yr = np.where(live[..., None], ref.f64(y)[np.maximum(rows, 0)], 0.0)
    dots = d[:, None, :] * yr
    assert np.all(np.abs(ref.f64(dp) - dots.sum(-1)) <= (n + 5) * 2.0 ** -24 * np.abs(dots).sum(-1))
    pd = ref.f64(p)
    dy = np.zeros((tokens * k, n))
    s = slots[slots >= 0]
    dy[slots >= 0] = d[s // k] * pd.reshape(-1)[s][:, None]
    dyb = torch.from_numpy(dy).float().bfloat16().double().numpy()  # rounded as the library does
    wd, qd = ref.f64(w), ref.f64(q)
    mask = ref.f64(torch.autograd.grad(ops.trace_fake_quant(z := xs.detach().requires_grad_(), cache),
                                       z, torch.ones_like(xs))[0])
    dq, dqm = np.zeros((tokens * k, cols)), np.zeros((tokens * k, cols))
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        dq[lo:hi], dqm[lo:hi] = dyb[lo:hi] @ wd[e], np.abs(dyb[lo:hi]) @ np.abs(wd[e])
        we, wm = dyb[lo:hi].T @ qd[lo:hi], np.abs(dyb[lo:hi]).T @ np.abs(qd[lo:hi])
        # dy is off by half a step of bf16 where its product lies at a border
        assert np.all(np.abs(ref.f64(dw)[e] - we) <= 2.0 ** -8 * np.abs(we) + 2.0 ** -7 * wm)
    dq, dqm = dq * mask, dqm * mask
    want = np.where(live[..., None], dq[np.maximum(rows, 0)], 0.0).sum(1)
    mag = np.where(live[..., None], dqm[np.maximum(rows, 0)], 0.0).sum(1)
    # dy (2^-8), the product's rounding (2^-8) and the sum's (2^-8), each of the magnitudes
    assert np.all(np.abs(ref.f64(dx) - want) <= 3.1 * 2.0 ** -8 * mag)


# ---------------------------------------------------------------------------
# Products whose tiles two CTAs share (large groups, tiled scales), and
# products whose k several CTAs share (few tiles)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,cols", [
    (129, 129, 64), (192, 130, 192), (255, 256, 320), (256, 257, 448), (257, 384, 704),
    (384, 1000, 128), (449, 392, 512), (600, 133, 832), (1025, 264, 1024), (3000, 520, 256)])
def test_product_of_pairs(fmt, rows, n, cols):
    """Ends of tokens, of columns and of k (a last stage of 64, 128 or 192
    elements) inside a tile; rows of out with and without 16-byte alignment."""
    _product_case(rows, n, cols, fmt, True, True, seed=rows + n)


PAIR_GROUPS = [
    [300, 2, 400], [129, 256, 1, 0, 700], [0, 600, 0, 3], [63, 500, 65, 191], [64, 64, 640],
    [257, 255, 320], [1000], [100, 700, None], [0, 0, 900, None], [127, 1, 385, 64, 300]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", PAIR_GROUPS, ids=str)
@pytest.mark.parametrize("n,cols", [(256, 320), (384, 512), (640, 64)])
def test_grouped_product_of_pairs(fmt, counts, n, cols):
    """Groups that start at any row of a 128-row block: in its first or second
    half, with more or fewer than 64 rows of another group before it."""
    rows = sum(c for c in counts if c is not None) + (333 if counts[-1] is None else 0)
    groups = len(counts)
    assert -(-rows // groups) > 128 and n % 128 == 0  # the rule that picks pairs
    _product_case(rows, n, cols, fmt, True, True, counts, seed=len(counts) + rows)


def test_rows_around_the_groups_of_pairs_are_left():
    rows, n, cols = 900, 256, 128
    a = inputs.tiny_site(1, rows, cols).x_roll.to(DEV)
    w = inputs.tiny_site(2, 2 * n, cols).x_roll.to(DEV)
    bounds = torch.arange(3, dtype=torch.int64, device=DEV) * n
    cw = ops.capture_tiled(w, bounds)
    ca = ops.capture_tiled(a, torch.tensor([0, 450, 900], dtype=torch.int64, device=DEV))
    whole = ops.fp4_matmul(ca, cw, cols)
    out = torch.full((rows, n), 5.0, dtype=torch.bfloat16, device=DEV)
    ca.offsets = torch.tensor([101, 450, 700], dtype=torch.int64, device=DEV)
    ops.fp4_matmul(ca, cw, cols, out=out)
    assert torch.equal(out[101:700], whole[101:700])
    assert bool((out[:101] == 5.0).all()) and bool((out[700:] == 5.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,cols", [
    (1, 128, 512), (5, 129, 1024), (16, 8, 544), (31, 2048, 768), (100, 4096, 1056),
    (128, 256, 4096), (190, 100, 2048), (700, 128, 1568)])
def test_product_with_k_split(fmt, rows, n, cols):
    _product_case(rows, n, cols, fmt, True, cols % 64 == 0, seed=rows + n)


def test_product_on_two_streams_and_in_graphs():
    """Two captured graphs of pair and split products replayed at once on two
    streams, and products interleaved with them: nothing is shared."""
    cases = []
    for i, (rows, n, cols) in enumerate([(900, 512, 1024), (8, 512, 2048)]):
        a = ops.capture_tiled(inputs.tiny_site(2 * i, rows, cols).x_roll.to(DEV))
        w = ops.capture_tiled(inputs.tiny_site(2 * i + 1, n, cols).x_roll.to(DEV))
        cases.append((a, w, cols, ops.fp4_matmul(a, w, cols)))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = [ops.fp4_matmul(a, w, cols) for a, w, cols, _ in cases * 3]
        graphs.append((s, g, outs))
    for _ in range(5):
        for s, g, outs in graphs:
            with torch.cuda.stream(s):
                g.replay()
        extra = [ops.fp4_matmul(a, w, cols) for a, w, cols, _ in cases]
    torch.cuda.synchronize()
    for outs in [o for _, _, o in graphs] + [extra]:
        for i, o in enumerate(outs):
            assert torch.equal(o, cases[i % 2][3])
    assert ops.matmul_status()


@pytest.mark.parametrize("tokens,k,experts", [(300000, 8, 5), (140000, 8, 64), (1100, 4, 4096)])
def test_sort_of_many_slots(tokens, k, experts):
    """More slots than the most chunks of the usual size; more experts than a
    CTA has threads."""
    g = _gen(tokens)
    ids = torch.randint(-1, experts, (tokens, k), generator=g).to(torch.int32)
    route = ops.moe_sort(ids.to(DEV), experts)
    key = torch.where(ids >= 0, ids, experts).reshape(-1)
    order = torch.sort(key, stable=True).indices
    want = torch.where(key[order] < experts, order, -1).to(torch.int32)
    assert torch.equal(route.slots.cpu(), want)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel())
    rows = torch.where(key < experts, rows, -1).to(torch.int32).view(tokens, k)
    assert torch.equal(route.rows.cpu(), rows)
    counts = torch.bincount(key, minlength=experts + 1)
    assert route.offsets.cpu().tolist() == [0] + torch.cumsum(counts, 0).tolist()


@pytest.mark.parametrize("k", [1, 7, 8, 9, 40])
def test_combine_of_many_choices(k):
    """Choices beyond one batch of rows, and rows that are no multiple of a warp's."""
    tokens, experts, cols = 21, 6, 1056
    route, (_, rows, _) = _route(tokens, k, experts, k, dropped=0.2)
    g = _gen(k)
    y = torch.randn(tokens * k, cols, generator=g).bfloat16().to(DEV)
    w = torch.randn(tokens, k, generator=g).to(DEV)
    out = ref.f64(ops.moe_combine(y, route, w))
    terms = np.where((rows >= 0)[..., None], ref.f64(y)[np.maximum(rows, 0)], 0.0) \
        * ref.f64(w)[..., None]
    s, m = terms.sum(1), np.abs(terms).sum(1)
    # one rounding to bf16 of a sum of k fused steps in fp32
    assert np.all(np.abs(out - s) <= 2.0 ** -8 * np.abs(s) + (1 + 2.0 ** -8) * k * 2.0 ** -24 * m)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled_a,tiled_w", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("rows,n,cols,counts", [
    (300, 1000, 352, None), (1111, 264, 96, None), (2048, 2050, 2080, None),
    (900, 200, 608, [300, 0, 600]), (1500, 136, 1056, [129, 1000, None]),
    (2500, 1000, 4128, [1100, 1400])])
def test_product_of_pairs_on_copied_scales(fmt, tiled_a, tiled_w, rows, n, cols, counts):
    """Scales in rows (of whole words or not), matrices that begin inside a
    128-row block, k that ends inside a piece of four scale columns."""
    _product_case(rows, n, cols, fmt, tiled_a, tiled_w, counts, seed=rows + cols)


def test_product_with_a_workspace_of_the_caller():
    """Poisoned before each call; the same bits as with one of its own, and
    close to those without any copy."""
    a = ops.capture(inputs.tiny_site(3, 700, 512).x_roll.to(DEV))
    w = ops.capture(inputs.tiny_site(4, 384, 512).x_roll.to(DEV))
    want = ops.fp4_matmul(a, w)
    nbytes = ops.trace_matmul_workspace_bytes(False, 700, 512, 1, 0, 384, 1, 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    for fill in (0x7F, 0xFF):
        ws.fill_(fill)
        assert torch.equal(ops.fp4_matmul(a, w, workspace=ws), want)
    with pytest.raises(ops.TraceError):
        ops.fp4_matmul(a, w, workspace=ws[:-256])
    exact, mag = ref.product(_operand(a, 700, 512, "nvfp4"), _operand(w, 384, 512, "nvfp4"),
                             a.gscale.cpu().numpy(), w.gscale.cpu().numpy(), [0, 700], 384)
    out = torch.empty_like(want)
    st = ops.library().trace_fp4_matmul(
        a.codes.data_ptr(), a.scales.data_ptr(), a.gscale.data_ptr(), 700, 512, 1, None, 0,
        w.codes.data_ptr(), w.scales.data_ptr(), w.gscale.data_ptr(), 384, 1, 0, out.data_ptr(),
        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for o in (out, want):
        assert np.all(np.abs(ref.f64(o) - exact) <= ref.product_bound(exact, mag, 512))


@pytest.mark.parametrize("fmt", FORMATS)
def test_products_of_rows_without_a_copy(fmt):
    """The same through the entry points that take no workspace (single CTAs on
    scales as they are)."""
    f = ops.trace_matmul_workspace_bytes
    try:
        ops.trace_matmul_workspace_bytes = lambda *a: 0
        for rows, n, cols, counts in [(300, 1000, 352, None), (1111, 264, 96, None),
                                      (900, 200, 608, [300, 0, 600]), (700, 384, 512, None)]:
            for ta, tw in ((False, False), (True, True), (False, True)):
                _product_case(rows, n, cols, fmt, ta, tw, counts, seed=rows)
    finally:
        ops.trace_matmul_workspace_bytes = f


# ---------------------------------------------------------------------------
# Sizes past 32 bits, nothing at all, and graphs of both directions
# ---------------------------------------------------------------------------

def test_product_with_more_than_2_31_outputs():
    rows, n, cols = 540000, 4096, 64
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device=DEV).bfloat16()
    w = ops.capture_tiled(inputs.tiny_site(2, n, cols).x_roll.to(DEV))
    for cap in (ops.capture_tiled(x), ops.capture(x)):
        out = ops.fp4_matmul(cap, w, cols)
        codes, scols = cap.codes.view(rows, cols // 2), cols // 16
        s = cap.scales
        if s.dim() != 2:  # a 128-row block is 512 bytes here: 4 scale columns
            s = s.view(-1, 32, 4, 4).permute(0, 2, 1, 3).reshape(-1, scols)[:rows]
        wv = _operand(w, n, cols, "nvfp4")
        for lo in (0, 262143, 524287, rows - 130):  # the last three past 2^30 and 2^31 elements
            part = ref.operand(codes[lo:lo + 130].cpu().numpy(), s[lo:lo + 130].cpu().numpy(), 130,
                               cols, "nvfp4")
            exact, mag = ref.product(part, wv, cap.gscale.cpu().numpy(), w.gscale.cpu().numpy(),
                                     [0, 130], n)
            assert np.all(np.abs(ref.f64(out[lo:lo + 130]) - exact)
                          <= ref.product_bound(exact, mag, cols))
        del out


def test_tokens_with_more_than_2_31_elements():
    tokens, k, cols, experts = 300000, 8, 1024, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    ids = torch.randint(0, experts, (tokens, k), generator=g, device=DEV)
    route = ops.moe_sort(ids, experts)
    x = torch.randn(tokens, cols, generator=g, device=DEV).bfloat16()
    y = ops.moe_dispatch(x, route)
    at = torch.tensor([0, 5, 2 ** 31 // cols - 1, 2 ** 31 // cols, tokens * k - 1], device=DEV)
    assert torch.equal(y[at], x[(route.slots[at] // k).long()])
    # 1/8 of a token's own value eight times: exact in every step
    weights = torch.full((tokens, k), 0.125, device=DEV)
    assert torch.equal(ops.moe_combine(y, route, weights), x)
    dy, dw = ops.moe_combine_bwd(x, y, route, weights)
    rows = route.rows.long()
    for t in (0, 131071, 262145, tokens - 1):
        assert torch.equal(dy[rows[t]], (x[t] * 0.125).expand(k, cols))
        want = (x[t].double() ** 2).sum()
        assert bool(((dw[t].double() - want).abs() <= (cols / 32 + 5) * 2.0 ** -24 * want).all())


def test_no_tokens():
    ids = torch.empty(0, 4, dtype=torch.int64, device=DEV)
    route = ops.moe_sort(ids, 6)
    assert route.offsets.tolist() == [0] * 8 and route.rows.shape == (0, 4)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    y = ops.moe_dispatch(x, route)
    w = torch.empty(0, 4, device=DEV, requires_grad=True)
    out = ops.moe_combine(y, route, w)
    dx, dw = torch.autograd.grad(out, (x, w), torch.empty_like(out))
    assert y.shape == out.shape == dx.shape == (0, 64) and dw.shape == (0, 4)


def test_dropped_rows_are_never_read():
    """NaN and infinities in the last group's rows, in their gradient and in
    the weights of dropped slots reach nothing."""
    tokens, k, experts, cols = 40, 3, 5, 96
    route, (offsets, rows, _) = _route(tokens, k, experts, 2, dropped=0.4)
    live, lo = torch.from_numpy(rows >= 0).to(DEV), int(offsets[experts])
    y = torch.randn(tokens * k, cols, generator=_gen(1)).bfloat16().to(DEV)
    w = torch.randn(tokens, k, generator=_gen(2)).to(DEV)
    do = torch.randn(tokens, cols, generator=_gen(3)).bfloat16().to(DEV)
    yb, wb = y.clone(), w.clone()
    yb[lo:] = float("nan")
    yb[lo::2] = float("inf")
    wb[~live] = float("nan")
    for a, b in zip((ops.moe_combine(y, route, w), *ops.moe_combine_bwd(do, y, route, w),
                     ops.moe_dispatch_bwd(y, route)),
                    (ops.moe_combine(yb, route, wb), *ops.moe_combine_bwd(do, yb, route, wb),
                     ops.moe_dispatch_bwd(yb, route))):
        assert torch.equal(a, b) and bool(torch.isfinite(b).all())


def test_both_directions_in_a_graph():
    """Forward and backward captured together and replayed on other inputs.
    No eager autograd graph of the leaves is alive during capture: PyTorch
    cannot capture a backward pass beside one."""
    tokens, k, experts, cols = 50, 4, 9, 512
    route, _ = _route(tokens, k, experts, 4)
    x = torch.randn(tokens, cols, generator=_gen(1)).bfloat16().to(DEV).requires_grad_()
    w = torch.rand(tokens, k, generator=_gen(2)).to(DEV).requires_grad_()
    do = torch.randn(tokens, cols, generator=_gen(3)).bfloat16().to(DEV)

    def both():
        out = ops.moe_combine(ops.moe_dispatch(x, route), route, w)
        return (out.detach(), *torch.autograd.grad(out, (x, w), do))

    eager = both()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        held = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, held))
    with torch.no_grad():
        x.copy_(torch.randn(tokens, cols, generator=_gen(5)).bfloat16())
        w.copy_(torch.rand(tokens, k, generator=_gen(6)))
    graph.replay()
    again = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, held))


def test_no_second_derivative():
    route, _ = _route(5, 2, 3, 1)
    x = torch.randn(5, 64).bfloat16().to(DEV).requires_grad_()
    (dx,) = torch.autograd.grad(ops.moe_dispatch(x, route).float().pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.float().sum().backward()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,cols", [(4100, 1030, 192), (9000, 300, 576), (3329, 776, 1088)])
def test_product_of_pairs_in_several_waves(fmt, rows, n, cols):
    """More tiles of 128 tokens than run at once: tiles of 256, some CTAs with
    more of them than others."""
    assert -(-rows // 128) * -(-n // 256) > torch.cuda.get_device_properties(0).multi_processor_count // 2
    _product_case(rows, n, cols, fmt, True, True, seed=rows + n)


# ---------------------------------------------------------------------------
# The two ways of a call, gradients at odd addresses, one very long sum
# ---------------------------------------------------------------------------

def _both_ways(call):
    """The usual call, and the same on a stream that is named (never one native step)."""
    s = torch.cuda.current_stream()
    return call(), call(stream=s)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
def test_both_ways_of_a_product(fmt, tiled):
    g = _gen(3)
    x = torch.randn(70, 320, generator=g).bfloat16().to(DEV)
    w = torch.randn(3 * 48, 320, generator=g).bfloat16().to(DEV)
    offs = torch.tensor([0, 30, 30, 61, 70], device=DEV)
    for experts, o in ((1, None), (3, offs)):
        bounds = None if experts == 1 else torch.arange(0, 145, 48, device=DEV)
        a, b = _capture(x, fmt, tiled, o), _capture(w, fmt, tiled, bounds)
        if fmt == "nvfp4":
            one, two = _both_ways(lambda **k: ops.fp4_matmul(a, b, 320, **k))
        else:
            one, two = _both_ways(lambda **k: ops.mx_matmul(a, b, 320, o, experts, **k))
        assert one.shape == (70, 144 // experts) and torch.equal(one, two)


def test_both_ways_of_sort_dispatch_and_combine():
    g = _gen(6)
    for dtype in (torch.int32, torch.int64):
        ids = torch.randint(-1, 9, (77, 3), generator=g).to(dtype).to(DEV)
        one, two = _both_ways(lambda **k: ops.moe_sort(ids, 8, **k))
        for u, v in zip((one.offsets, one.rows, one.slots), (two.offsets, two.rows, two.slots)):
            assert u.dtype == v.dtype and torch.equal(u, v)
    x = torch.randn(77, 96, generator=g).bfloat16().to(DEV)
    w = torch.rand(77, 3, generator=g).to(DEV)
    y = ops.moe_dispatch(x, one)
    assert torch.equal(y, ops.moe_dispatch_fwd(x, one))
    assert torch.equal(ops.moe_combine(y, one, w), ops.moe_combine_fwd(y, one, w))
    with torch.no_grad():  # a leaf, but nothing to differentiate
        assert not ops.moe_dispatch(x.requires_grad_(), one).requires_grad
    assert ops.moe_dispatch(x, one).requires_grad


def test_a_route_can_be_saved(tmp_path):
    route, _ = _route(9, 2, 4, 5)
    torch.save((route.offsets, route.rows, route.slots), tmp_path / "route.pt")
    for u, v in zip(torch.load(tmp_path / "route.pt"), (route.offsets, route.rows, route.slots)):
        assert torch.equal(u, v)


def test_gradients_that_start_anywhere():
    """A part of a larger gradient is contiguous and yet not 32-byte aligned."""
    tokens, k, cols = 11, 2, 64
    route, _ = _route(tokens, k, 3, 7)
    g = _gen(8)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).bfloat16().to(DEV)  # noqa: E731
    x, y, w = ints(tokens, cols), ints(tokens * k, cols), ints(tokens, k).float()
    head, up = ints(5), ints(5 + tokens * k * cols)
    x.requires_grad_(), y.requires_grad_(), w.requires_grad_()
    flat = torch.cat((head, ops.moe_dispatch(x, route).view(-1)))
    (dx,) = torch.autograd.grad(flat, x, up)
    assert torch.equal(dx, ops.moe_dispatch_bwd(up[5:].clone().view(-1, cols), route))
    flat = torch.cat((head, ops.moe_combine(y, route, w).view(-1)))
    part = up[:5 + tokens * cols]
    dy, dw = torch.autograd.grad(flat, (y, w), part)
    want = ops.moe_combine_bwd(part[5:].clone().view(tokens, cols), y.detach(), route, w.detach())
    assert torch.equal(dy, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("groups", [1, 2])
def test_product_of_the_longest_rows(groups):
    """2^31 - 1024 terms to a sum, of which the first and the last 2^20 are one
    and the others zero: exact in fp32, in which it is held, and in bf16."""
    cols, ones = (1 << 31) - 1024, 1 << 19
    codes = torch.zeros(groups, cols // 2, dtype=torch.uint8, device=DEV)
    codes[:, :ones] = codes[:, -ones:] = 0x22
    scales = torch.full((groups, cols // 16), 0x38, dtype=torch.uint8, device=DEV)
    offs = None if groups == 1 else torch.arange(groups + 1, device=DEV)
    unit = torch.ones(groups, device=DEV)
    a = ops.Capture(codes.view(-1), None, scales, unit, offs)
    assert ops.matmul_status()
    out = ops.fp4_matmul(a, ops.Capture(a.codes, None, a.scales, unit))
    assert ops.matmul_status() and out.flatten().tolist() == [2.0 ** 21] * groups


def test_outputs_that_a_backward_pass_still_needs():
    """A route or rows written anew between the two directions: refused, not wrong."""
    tokens, k, cols = 12, 2, 64
    g = _gen(9)
    ids = torch.randint(0, 4, (tokens, k), generator=g).to(DEV)
    x = torch.randn(tokens, cols, generator=g).bfloat16().to(DEV).requires_grad_()
    w = torch.rand(tokens, k, generator=g).to(DEV).requires_grad_()
    route = ops.moe_sort(ids, 4)
    y = ops.moe_dispatch(x, route)
    ops.moe_sort(ids.flip(0).contiguous(), 4, out=route)
    with pytest.raises(RuntimeError):
        y.sum().backward()
    rows = ops.moe_dispatch_fwd(x.detach(), route)
    out = ops.moe_combine(rows, route, w)
    ops.moe_dispatch_fwd(x.detach() * 2, route, out=rows)
    with pytest.raises(RuntimeError):
        out.sum().backward()
    with torch.inference_mode():  # tensors without a version
        again = ops.moe_sort(ids, 4)
        ops.moe_sort(ids, 4, out=again)
    ops.moe_combine(ops.moe_dispatch(x, route), route, w).sum().backward()
    assert x.grad is not None and w.grad is not None


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,cols,counts", [
    (700, 1003, 96, [300, 1, 399]), (517, 390, 160, None), (518, 389, 2080, None),
    (901, 1021, 64, [129, 501, 271]), (900, 262, 192, [127, 500, None]), (99, 95, 64, [33, 50, 16]),
    (64, 33, 320, None), (150, 31, 320, None), (400, 2047, 64, None)])
def test_product_rows_that_begin_anywhere(fmt, rows, n, cols, counts):
    """Rows of out at odd elements: whole pieces as words, edges one by one."""
    _product_case(rows, n, cols, fmt, True, True, counts, seed=rows * 3 + n)


def test_gradients_under_checkpoints_anomaly_checks_and_threads():
    """Saved tensors packed and recomputed, traces kept of each node, calls from
    several threads on streams of their own: the same gradients."""
    import threading
    from torch.utils.checkpoint import checkpoint
    tokens, k, cols = 33, 3, 128
    route, _ = _route(tokens, k, 5, 6)
    g = _gen(12)
    x = torch.randn(tokens, cols, generator=g).bfloat16().to(DEV).requires_grad_()
    w = torch.rand(tokens, k, generator=g).to(DEV).requires_grad_()
    do = torch.randn(tokens, cols, generator=g).bfloat16().to(DEV)

    def layer(x, w):
        return ops.moe_combine(ops.moe_dispatch(x, route) * 2, route, w)

    want = torch.autograd.grad(layer(x, w), (x, w), do)
    got = [torch.autograd.grad(checkpoint(layer, x, w, use_reentrant=False), (x, w), do)]
    with torch.autograd.graph.save_on_cpu():
        got.append(torch.autograd.grad(layer(x, w), (x, w), do))
    with torch.autograd.detect_anomaly(check_nan=False):
        got.append(torch.autograd.grad(layer(x, w), (x, w), do))

    def work(to):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            for _ in range(20):
                out = torch.autograd.grad(layer(x, w), (x, w), do)
        s.synchronize()
        to.append(out)

    threads = [threading.Thread(target=work, args=(got,)) for _ in range(4)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 7
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))
