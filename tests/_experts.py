"""Plain 64-bit forms of the FP4 expert operators (numpy; nothing from the
library): decoding of captured operands, the grouped product, the routing
sort, dispatch and combine."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def e4m3(b):
    """E4M3 bytes 0x00..0x7E -> float64."""
    b = np.asarray(b, np.int64)
    e, m = b >> 3, b & 7
    return np.where(e > 0, (8 + m) * np.exp2(e - 10.0), m * 2.0 ** -9)


def e8m0(b):
    return np.exp2(np.asarray(b, np.float64) - 127.0)


def untile(flat, rows, scols):
    """Row-major [rows, scols] of the flat 128 x 4 tiled scale bytes."""
    r, c = np.arange(rows)[:, None], np.arange(scols)[None, :]
    at = ((r // 128) * (-(-scols // 4)) + c // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + c % 4
    return np.asarray(flat)[at]


def tile(scales, fill=0):
    rows, scols = scales.shape
    out = np.full(-(-rows // 128) * (-(-scols // 4)) * 512, fill, np.uint8)
    r, c = np.arange(rows)[:, None], np.arange(scols)[None, :]
    out[((r // 128) * (-(-scols // 4)) + c // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32)
        + c % 4] = scales
    return out


def operand(codes, scales, rows, cols, fmt):
    """float64 [rows, cols] = codeword * block scale (row-major scales)."""
    c = np.asarray(codes, np.uint8).reshape(rows, cols // 2)
    nib = np.empty((rows, cols), np.uint8)
    nib[:, 0::2], nib[:, 1::2] = c & 15, c >> 4
    bs = 16 if fmt == "nvfp4" else 32
    s = np.asarray(scales, np.uint8).reshape(rows, cols // bs)
    s = e4m3(s) if fmt == "nvfp4" else e8m0(s)
    return E2M1[nib] * np.repeat(s, bs, axis=1)


def product(a, w, ga, gw, offsets, n):
    """(out, sum of magnitudes) of the grouped product in float64; a [rows, K],
    w [matrices * n, K]; rows of groups without a matrix are 0."""
    rows = a.shape[0]
    out, mag = np.zeros((rows, n)), np.zeros((rows, n))
    for g in range(len(offsets) - 1):
        lo, hi = offsets[g], offsets[g + 1]
        if (g + 1) * n > w.shape[0] or hi <= lo:
            continue
        m = w[g * n:(g + 1) * n]
        f = 1.0 if ga is None else float(ga[g]) * float(gw[g])
        out[lo:hi] = f * (a[lo:hi] @ m.T)
        mag[lo:hi] = f * (np.abs(a[lo:hi]) @ np.abs(m).T)
    return out, mag


def product_bound(ref, mag, cols):
    """How far a bf16 output may be from `ref`: the terms are exact in fp32
    (2 x 4 significant bits times 2 x 4); adding cols of them in fp32, even by
    truncation, is off by at most 2^-23 of the running magnitude each; the
    global scales round twice more (2^-24 each, 2^-22 allowed); bf16 rounds by
    half a step, 2^-8 relative (2^-134 below its normal range)."""
    e = cols * 2.0 ** -23 * mag + 2.0 ** -22 * np.abs(ref)
    return 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * e + 2.0 ** -134


def sort(ids, experts):
    """(offsets, rows, slots) by a stable sort."""
    flat = np.asarray(ids, np.int64).reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([np.searchsorted(key[order], np.arange(experts + 1)), [flat.size]])
    rows = np.empty(flat.size, np.int32)
    rows[order] = np.arange(flat.size)
    rows[key == experts] = -1
    return offsets.astype(np.int64), rows.reshape(ids.shape), \
        np.where(key[order] < experts, order, -1).astype(np.int32)


def bits(t: torch.Tensor):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def f64(t: torch.Tensor):
    return t.detach().cpu().double().numpy()
