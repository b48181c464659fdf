"""Plain 64-bit implementations of the router and of MXFP4, for the tests.

numpy, one formula at a time; nothing here is shared with the kernels."""
from __future__ import annotations

import numpy as np

GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def route(logits, bias, top_k: int, renormalize: bool):
    """logits float32 [M, E] (exact conversions of the given type) -> ids, weights in 64 bits."""
    logits = np.asarray(logits, dtype=np.float32)
    with np.errstate(all="ignore"):
        score = logits if bias is None else logits + np.asarray(bias, dtype=np.float32)
    M, E = logits.shape
    ids = np.full((M, top_k), -1, dtype=np.int32)
    w = np.zeros((M, top_k))
    for t in range(M):
        part = [e for e in range(E) if score[t, e] > -np.inf]  # False for NaN
        order = sorted(part, key=lambda e: (-float(score[t, e]), e))[:top_k]
        over = order if renormalize else part
        if not order:
            continue
        most = max(float(logits[t, e]) for e in over)

        def z(e):
            x = float(logits[t, e])
            return 1.0 if x == most else float(np.exp(x - most)) if np.isfinite(most) else 0.0
        total = sum(z(e) for e in over)
        for i, e in enumerate(order):
            ids[t, i], w[t, i] = e, z(e) / total
    return ids, w


def mx_quant(x):
    """x [rows, cols] -> codes [rows, cols] (0..15), scale bytes [rows, cols / 32]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[..., None], 0.0, b)
    most = np.abs(b).max(axis=2)
    e = np.where(most > 0, np.frexp(np.where(most > 0, most, 1.0))[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    m = np.minimum(np.abs(b) / np.exp2(e)[..., None], 6.0)
    hi = np.clip(np.searchsorted(GRID, m), 0, 7)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - m, m - GRID[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = code + 8 * np.signbit(b)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(rows, cols).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(code):
    return (code[..., ::2] | code[..., 1::2] << 4).astype(np.uint8)


def mx_values(q, scale):
    """Packed codes [..., cols / 2] and scale bytes [..., cols / 32] -> values [..., cols]."""
    q, scale = np.asarray(q), np.asarray(scale)
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def silu(u):
    with np.errstate(over="ignore"):
        return u / (1 + np.exp(-u))
