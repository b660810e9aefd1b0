"""The measured operators of the FP4 mixture-of-experts path and their plain forms.

Three operators of a rollout's FP4 experts, next to the capture that feeds them:

* the product of two captured operands, out = A_q W_q^T, with NVFP4 operands
  (E4M3 scales of 16-element blocks and an fp32 global scale per group) or
  MXFP4 ones (E8M0 scales of 32-element blocks), dense or grouped by expert;
* the routing sort: slots (token, choice) ordered by expert;
* tokens copied into expert order and back with the routing weights applied,
  each with its gradient.

``run`` computes the plain form where ``own`` is false and calls the package
where it is true.  ``exact`` is the definition in 64 bits, written apart.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def listed():
    return [
        # one generated token through a dense projection: latency, one read of the weights
        {"name": "nvfp4 one token", "op": "matmul", "fmt": "nvfp4", "rows": 1, "n": 4096,
         "cols": 4096, "experts": 1, "tiled": True},
        # a small decode batch, odd, with the scales as plain rows
        {"name": "mxfp4 29 tokens", "op": "matmul", "fmt": "mxfp4", "rows": 29, "n": 2048,
         "cols": 4096, "experts": 1, "tiled": False},
        # the attention input of a prompt batch through its projection
        {"name": "nvfp4 prompt", "op": "matmul", "fmt": "nvfp4", "rows": 16384, "n": 4096,
         "cols": 2048, "experts": 1, "tiled": True},
        # an odd number of rows through a square projection
        {"name": "mxfp4 odd rows", "op": "matmul", "fmt": "mxfp4", "rows": 4099, "n": 4096,
         "cols": 4096, "experts": 1, "tiled": True},
        # 64 generated tokens, 8 of 128 experts each: one read of the experts' weights
        {"name": "nvfp4 experts decode", "op": "matmul", "fmt": "nvfp4", "rows": 512, "n": 1536,
         "cols": 2048, "experts": 128, "tiled": True},
        # 8192 prompt tokens, 8 of 128 experts each, ragged groups
        {"name": "nvfp4 experts prompt", "op": "matmul", "fmt": "nvfp4", "rows": 65536, "n": 1536,
         "cols": 2048, "experts": 128, "tiled": True},
        # the routing of one generated token, and of a large prompt batch
        {"name": "sort one token", "op": "sort", "tokens": 1, "k": 8, "experts": 128,
         "dropped": 0.0, "wide": False},
        {"name": "sort 65536 tokens", "op": "sort", "tokens": 65536, "k": 8, "experts": 128,
         "dropped": 0.1, "wide": True},
        # a decode batch into expert order; a training batch there with its gradient
        {"name": "dispatch 37 tokens", "op": "dispatch", "tokens": 37, "k": 8, "cols": 2048,
         "experts": 128, "dropped": 0.0, "grad": False},
        {"name": "dispatch 8192 tokens", "op": "dispatch", "tokens": 8192, "k": 8, "cols": 2048,
         "experts": 128, "dropped": 0.05, "grad": True},
        # one generated token back from its experts; a training batch with its gradients
        {"name": "combine one token", "op": "combine", "tokens": 1, "k": 8, "cols": 2048,
         "experts": 128, "dropped": 0.0, "grad": False},
        {"name": "combine 8192 tokens", "op": "combine", "tokens": 8192, "k": 8, "cols": 2048,
         "experts": 128, "dropped": 0.05, "grad": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("matmul", "matmul", "sort", "dispatch", "combine"))
    if op == "matmul":
        experts = rng.choice((1, 1, _log(rng, 2, 128)))
        case = {"op": op, "fmt": rng.choice(("nvfp4", "mxfp4")), "rows": _log(rng, 1, 65536),
                "n": _log(rng, 32, 4096), "cols": 32 * _log(rng, 2, 128), "experts": experts,
                "tiled": rng.random() < 0.7}
        while case["rows"] * case["n"] * case["cols"] > 65536 * 1536 * 2048:
            case["rows"] = case["rows"] // 2
        if experts * case["n"] * case["cols"] > 128 * 1536 * 2048:
            case["experts"] = max(1, 128 * 1536 * 2048 // (case["n"] * case["cols"]))
        return case
    tokens, k, experts = _log(rng, 1, 65536), rng.randint(1, 8), _log(rng, 8, 512)
    dropped = rng.choice((0.0, round(rng.uniform(0.0, 0.5), 3)))
    if op == "sort":
        return {"op": op, "tokens": tokens, "k": k, "experts": experts, "dropped": dropped,
                "wide": rng.random() < 0.5}
    cols = 32 * _log(rng, 2, 128)
    while tokens * k * cols > 8192 * 8 * 2048:
        tokens = tokens // 2
    return {"op": op, "tokens": max(1, tokens), "k": k, "cols": cols, "experts": experts,
            "dropped": dropped, "grad": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _counts(rows, experts):
    """Rows per expert before the experts are shuffled: a router's uneven load."""
    w = [1.0 / math.sqrt(i + 4.0) for i in range(experts)]
    s = sum(w)
    c = [int(rows * v / s) for v in w]
    left = rows - sum(c)
    return [v + left // experts + (1 if i < left % experts else 0) for i, v in enumerate(c)]


def _tile(scales):
    """[r, c] block scales -> the flat 128 x 4 tiled layout (padding zero)."""
    r, c = scales.shape
    rp, cp = -(-r // 128) * 128, -(-c // 4) * 4
    s = scales.new_zeros(rp, cp)
    s[:r, :c] = scales
    return s.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _quantise(x, groups, fmt):
    """(codes, row-major scales, global scales) of x [rows, cols] fp32, whose rows
    are cut into `groups` (row counts): what a capture of x holds."""
    rows, cols = x.shape
    bs = BLOCK[fmt]
    blocks = x.view(rows, cols // bs, bs)
    bmax = blocks.abs().amax(-1)
    if fmt == "nvfp4":
        counts = torch.tensor(groups, device=x.device)
        gid = torch.repeat_interleave(torch.arange(len(groups), device=x.device), counts)
        amax = x.new_zeros(len(groups)).scatter_reduce(0, gid, bmax.amax(-1), "amax")
        gscale = torch.where(amax > 0, amax / 2688.0, torch.ones_like(amax))
        sb = (bmax / (6.0 * gscale[gid, None])).clamp(max=448.0).to(torch.float8_e4m3fn)
        scales, unit = sb.view(torch.uint8), sb.float() * gscale[gid, None]
    else:
        gscale = None
        e = torch.floor(torch.log2(bmax.clamp(min=2.0 ** -120))) - 2.0
        scales, unit = (e + 127.0).clamp(min=0.0).to(torch.uint8), torch.exp2(e)
    z = torch.where(unit[..., None] > 0, blocks / unit[..., None], torch.zeros_like(blocks))
    cuts = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    mag = torch.bucketize(z.abs(), cuts)
    nib = (mag + 8 * (z < 0)).to(torch.uint8).view(rows, cols)
    codes = (nib[:, 0::2] | (nib[:, 1::2] << 4)).reshape(-1)
    return codes.contiguous(), scales.contiguous(), gscale


def _activation(rows, cols, g, dev):
    """N(0,1) times per-channel lognormal scales with 1% outlier channels, as bf16 values."""
    scale = torch.exp(torch.randn(cols, generator=g, device=dev))
    scale[torch.randperm(cols, generator=g, device=dev)[:max(1, cols // 100)]] *= 20.0
    x = torch.randn(rows, cols, generator=g, device=dev) * scale
    return x.to(torch.bfloat16)


def _route(tokens, k, experts, dropped, g, dev):
    """Expert ids [tokens, k] of a router with uneven load; a share of the slots is
    -1 (padding tokens)."""
    load = torch.randn(experts, generator=g, device=dev)
    score = torch.rand(tokens, experts, generator=g, device=dev).log().neg().log().neg() + load
    if experts >= k:
        ids = score.topk(k, dim=1).indices
    else:
        ids = torch.randint(experts, (tokens, k), generator=g, device=dev)
    if dropped:
        ids[torch.rand(tokens, generator=g, device=dev) < dropped] = -1
    return ids


def _sorted(ids, experts):
    """(offsets [experts + 2], rows [tokens, k], slots [tokens * k]) of expert ids."""
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    # one word for each group: how many keys are below each group's number
    bounds = torch.arange(experts + 2, device=flat.device)
    offsets = torch.searchsorted(key[order], bounds)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=order.device)
    rows = torch.where(key < experts, rows, torch.full_like(rows, -1)).to(torch.int32)
    slots = torch.where(key[order] < experts, order, torch.full_like(order, -1)).to(torch.int32)
    return offsets, rows.view(ids.shape), slots


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "matmul":
        rows, n, cols, E = case["rows"], case["n"], case["cols"], case["experts"]
        counts = _counts(rows, E)
        perm = torch.randperm(E, generator=g, device=dev).tolist()
        counts = [counts[p] for p in perm]
        x = _activation(rows, cols, g, dev).float()
        s["a_codes"], scales, s["a_gscale"] = _quantise(x, counts, case["fmt"])
        s["a_scales"] = _tile(scales) if case["tiled"] else scales
        parts = []
        for e in range(E):  # an expert at a time: the draws would not fit at once
            w = torch.randn(n, cols, generator=g, device=dev) * (0.02 * (1.0 + e % 3))
            parts.append(_quantise(w.to(torch.bfloat16).float(), [n], case["fmt"]))
        s["w_codes"] = torch.cat([p[0] for p in parts])
        scales = torch.cat([p[1] for p in parts])
        s["w_scales"] = _tile(scales) if case["tiled"] else scales
        s["w_gscale"] = torch.cat([p[2] for p in parts]) if case["fmt"] == "nvfp4" else None
        if E > 1:
            c = torch.tensor([0] + counts, device=dev)
            s["offsets"] = torch.cumsum(c, 0).to(torch.int64)
            s["most"] = max(counts)
        return s
    ids = _route(case["tokens"], case["k"], case["experts"], case["dropped"], g, dev)
    if case["op"] == "sort":
        s["ids"] = ids.to(torch.int64 if case["wide"] else torch.int32)
        return s
    s["offsets"], s["rows"], s["slots"] = _sorted(ids, case["experts"])
    tokens, k, cols = case["tokens"], case["k"], case["cols"]
    if case["op"] == "dispatch":
        s["x"] = _activation(tokens, cols, g, dev)
        if case["grad"]:
            s["dy"] = torch.randn(tokens * k, cols, generator=g, device=dev).to(torch.bfloat16)
    else:
        s["y"] = _activation(tokens * k, cols, g, dev)
        s["weights"] = torch.softmax(torch.randn(tokens, k, generator=g, device=dev), dim=1)
        if case["grad"]:
            s["dout"] = torch.randn(tokens, cols, generator=g, device=dev).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# Plain forms and calls
# ---------------------------------------------------------------------------

def _plain_scales(scales, rows, cols, fmt, tiled):
    """fp32 [rows, cols / block] of the scale bytes."""
    c = cols // BLOCK[fmt]
    if tiled:
        t = scales.view(-(-rows // 128), -(-c // 4), 32, 4, 4)
        scales = t.permute(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, -1)[:rows, :c]
    if fmt == "nvfp4":
        return scales.contiguous().view(torch.float8_e4m3fn).float()
    return torch.exp2(scales.float() - 127.0)


def _plain_operand(codes, scales, rows, cols, fmt, tiled):
    """fp32 [rows, cols] = codeword times block scale."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), -1).view(rows, -1, BLOCK[fmt]).int()
    s = _plain_scales(scales, rows, cols, fmt, tiled)
    return (grid[nib] * s[..., None]).view(rows, cols)


def _plain_matmul(s):
    rows, n, cols, E, fmt = s["rows"], s["n"], s["cols"], s["experts"], s["fmt"]
    a = _plain_operand(s["a_codes"], s["a_scales"], rows, cols, fmt, s["tiled"])
    w = _plain_operand(s["w_codes"], s["w_scales"], E * n, cols, fmt, s["tiled"])
    if E == 1:
        out = a @ w.t()
        if fmt == "nvfp4":
            out = out * s["a_gscale"] * s["w_gscale"]
        return out.to(torch.bfloat16)
    r = torch.arange(rows, device=a.device)
    gid = torch.searchsorted(s["offsets"], r, right=True) - 1
    pos = r - s["offsets"][gid]
    padded = a.new_zeros(E, s["most"], cols)
    padded[gid, pos] = a
    out = torch.bmm(padded, w.view(E, n, cols).transpose(1, 2))
    if fmt == "nvfp4":
        out = out * s["a_gscale"][:, None, None] * s["w_gscale"][:, None, None]
    return out[gid, pos].to(torch.bfloat16)


def _plain_dispatch(s):
    tokens, k = s["rows"].shape
    slots = s["slots"].long()
    live = slots >= 0
    out = {"y": torch.where(live[:, None], s["x"][slots.clamp(min=0) // k], 0.0)}
    if s["grad"]:
        rows = s["rows"].long()
        picked = s["dy"].float()[rows.clamp(min=0)]
        out["dx"] = torch.where((rows >= 0)[..., None], picked, 0.0).sum(1).to(torch.bfloat16)
    return out


def _plain_combine(s):
    tokens, k = s["rows"].shape
    rows = s["rows"].long()
    y = s["y"].float()[rows.clamp(min=0)]
    y = torch.where((rows >= 0)[..., None], y, 0.0)
    out = {"out": (y * s["weights"][..., None]).sum(1).to(torch.bfloat16)}
    if s["grad"]:
        dout = s["dout"].float()
        out["dweights"] = (y * dout[:, None, :]).sum(-1)
        slots = s["slots"].long()
        live = slots >= 0
        slots = slots.clamp(min=0)
        dy = dout[slots // k] * s["weights"].reshape(-1)[slots][:, None]
        out["dy"] = torch.where(live[:, None], dy, 0.0).to(torch.bfloat16)
    return out


def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "matmul":
            return {"out": _plain_matmul(s)}
        if op == "sort":
            offsets, rows, slots = _sorted(s["ids"], s["experts"])
            return {"offsets": offsets, "rows": rows, "slots": slots}
        return _plain_dispatch(s) if op == "dispatch" else _plain_combine(s)
    from fp4_quantization_aware_trace_b200 import ops
    if op == "matmul":
        offsets = s.get("offsets")
        if s["fmt"] == "nvfp4":
            a = ops.Capture(s["a_codes"], None, s["a_scales"], s["a_gscale"], offsets)
            w = ops.Capture(s["w_codes"], None, s["w_scales"], s["w_gscale"])
            return {"out": ops.fp4_matmul(a, w, s["cols"])}
        a = ops.MxCapture(s["a_codes"], None, s["a_scales"])
        w = ops.MxCapture(s["w_codes"], None, s["w_scales"])
        return {"out": ops.mx_matmul(a, w, s["cols"], offsets=offsets, groups=s["experts"])}
    if op == "sort":
        route = ops.moe_sort(s["ids"], s["experts"])
        return {"offsets": route.offsets, "rows": route.rows, "slots": route.slots}
    route = ops.MoeRoute(s["offsets"], s["rows"], s["slots"])
    if op == "dispatch":
        if not s["grad"]:
            return {"y": ops.moe_dispatch(s["x"], route)}
        x = s["x"].detach().requires_grad_()
        y = ops.moe_dispatch(x, route)
        return {"y": y, "dx": torch.autograd.grad(y, x, s["dy"])[0]}
    if not s["grad"]:
        return {"out": ops.moe_combine(s["y"], route, s["weights"])}
    y, weights = s["y"].detach().requires_grad_(), s["weights"].detach().requires_grad_()
    out = ops.moe_combine(y, route, weights)
    dy, dweights = torch.autograd.grad(out, (y, weights), s["dout"])
    return {"out": out, "dweights": dweights, "dy": dy}


def work(case):
    op = case["op"]
    if op == "matmul":
        rows, n, cols, E, bs = (case["rows"], case["n"], case["cols"], case["experts"],
                                BLOCK[case["fmt"]])
        hit = sum(1 for c in _counts(rows, E) if c)  # experts that no row reaches are not read
        operand = (rows + hit * n) * (cols // 2 + cols // bs)
        small = 8 * hit if case["fmt"] == "nvfp4" else 0
        return {"bytes": operand + small + 2 * rows * n, "flops": 2 * rows * n * cols}
    slots = case["tokens"] * case["k"]
    if op == "sort":
        return {"bytes": slots * ((8 if case["wide"] else 4) + 8) + 8 * (case["experts"] + 2),
                "flops": slots}
    token, spread = 2 * case["tokens"] * case["cols"], 2 * slots * case["cols"]
    passes = 2 if case["grad"] else 1
    if op == "dispatch":
        return {"bytes": passes * (token + spread + 4 * slots),
                "flops": slots * (case["cols"] if case["grad"] else 1)}
    backward = token + 2 * spread + 12 * slots if case["grad"] else 0
    return {"bytes": token + spread + 8 * slots + backward,
            "flops": slots * case["cols"] * (5 if case["grad"] else 2)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_bytes(scales, rows, cols, fmt, tiled):
    """float64 [rows, cols / block]: the scale at (r, c), looked up by its byte address and
    decoded from its exponent and mantissa fields."""
    c = cols // BLOCK[fmt]
    if tiled:
        r = torch.arange(rows, device=scales.device)[:, None]
        q = torch.arange(c, device=scales.device)[None, :]
        at = ((r // 128) * (-(-c // 4)) + q // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + q % 4
        scales = scales.reshape(-1)[at]
    b = scales.to(torch.int64)
    if fmt == "mxfp4":
        return torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
    e, m = b // 8, b % 8
    normal = torch.ldexp(1.0 + m.double() / 8.0, e - 7)
    return torch.where(e > 0, normal, m.double() * 2.0 ** -9)


def _exact_operand(codes, scales, fmt, first, last, cols):
    nib = torch.empty(last - first, cols, dtype=torch.int64, device=codes.device)
    part = codes.view(-1, cols // 2)[first:last].to(torch.int64)
    nib[:, 0::2] = part % 16
    nib[:, 1::2] = part // 16
    e, m = nib % 8 // 2, nib % 2
    mag = torch.where(e > 0, (1.0 + 0.5 * m.double()) * torch.exp2(e.double() - 1.0), 0.5 * m.double())
    value = torch.where(nib >= 8, -mag, mag)
    return value * torch.repeat_interleave(scales[first:last], BLOCK[fmt], dim=1)


def exact(case, seed):
    op = case["op"]
    if op == "sort":  # whole numbers
        return None
    s = prepare(case, seed)
    if op == "matmul":
        rows, n, cols, E, fmt = (case[v] for v in ("rows", "n", "cols", "experts", "fmt"))
        sa = _exact_bytes(s["a_scales"], rows, cols, fmt, case["tiled"])
        sw = _exact_bytes(s["w_scales"], E * n, cols, fmt, case["tiled"])
        bounds = s["offsets"].tolist() if E > 1 else [0, rows]
        out = torch.zeros(rows, n, dtype=torch.float64, device=sa.device)
        for e in range(E):
            lo, hi = bounds[e], bounds[e + 1]
            if lo == hi:
                continue
            a = _exact_operand(s["a_codes"], sa, fmt, lo, hi, cols)
            w = _exact_operand(s["w_codes"], sw, fmt, e * n, (e + 1) * n, cols)
            out[lo:hi] = torch.einsum("rc,nc->rn", a, w)
            if fmt == "nvfp4":
                out[lo:hi] *= s["a_gscale"][e].double() * s["w_gscale"][e].double()
        return {"out": out}
    rows, k = s["rows"].long(), case["k"]
    at = rows.reshape(-1)
    token = torch.arange(case["tokens"], device=at.device).repeat_interleave(k)
    live = at >= 0
    at, token, slot = at[live], token[live], torch.nonzero(live).reshape(-1)
    if op == "dispatch":
        y = torch.zeros(case["tokens"] * k, case["cols"], dtype=torch.float64, device=at.device)
        y[at] = s["x"].double()[token]
        if not case["grad"]:
            return {"y": y}
        dx = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=at.device)
        dx.index_add_(0, token, s["dy"].double()[at])
        return {"y": y, "dx": dx}
    w = s["weights"].double().reshape(-1)
    y = s["y"].double()
    out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=at.device)
    out.index_add_(0, token, y[at] * w[slot, None])
    if not case["grad"]:
        return {"out": out}
    dout = s["dout"].double()
    dweights, dy = torch.zeros_like(w), torch.zeros_like(y)
    dweights[slot] = torch.einsum("sc,sc->s", dout[token], y[at])
    dy[at] = dout[token] * w[slot, None]
    return {"out": out, "dweights": dweights.view(case["tokens"], k), "dy": dy}
