"""Float64 restatement of the microscaled formats, the norm, their product and sampling (test
infrastructure only).

A block of 32 values of a row shares the power 2^(floor(log2 max|v|) - top), not below 2^-127, and
holds each value over it as the nearest of the format's numbers, of two equally near ones the one
with the even code.
"""

from __future__ import annotations

import numpy as np

TOP = {"fp4": 2, "fp8": 8}


def numbers(fmt: str) -> np.ndarray:
    """The format's numbers from 0 up, by code."""
    if fmt == "fp4":
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.array([(8 + c % 8) * 2.0 ** (c // 8 - 10) if c >= 8 else c * 2.0 ** -9 for c in range(127)])


def quantize_ref(x: np.ndarray, fmt: str):
    """x [rows][cols] float64 -> codes [rows][cols] (sign in the top bit of 4 or 8), scale bytes
    [rows][blocks]."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    v = np.zeros((rows, blocks * 32))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, 32)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0, v)
    most = np.abs(v).max(-1)
    _, e = np.frexp(most)                                  # most = f 2^e, f in [1/2, 1)
    byte = np.where(most > 0, np.maximum(e - 1 - TOP[fmt] + 127, 0), 0)
    a = np.abs(v) / 2.0 ** (byte - 127.0)[..., None]
    table = numbers(fmt)
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)  # table[hi - 1] < a <= table[hi]
    low, high = a - table[hi - 1], table[hi] - a
    code = np.where((low < high) | ((low == high) & (hi % 2 == 1)), hi - 1, hi)
    code = np.where(a >= table[-1], len(table) - 1, code)
    code = code + np.where(np.signbit(v), 8 if fmt == "fp4" else 128, 0)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(rows, -1)[:, :cols], np.where(bad, 255, byte)


def values_ref(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    sign = 8 if fmt == "fp4" else 128
    table = np.append(numbers(fmt), np.nan)
    v = table[codes % sign] * np.where(codes >= sign, -1.0, 1.0)
    scale = np.where(scales == 255, np.nan, 2.0 ** (scales - 127.0))
    return v * np.repeat(scale, 32, axis=1)[:, :codes.shape[1]]


def held_ref(x: np.ndarray, fmt: str) -> np.ndarray:
    return values_ref(*quantize_ref(x, fmt), fmt)


def tiled_ref(codes: np.ndarray, scales: np.ndarray, fmt: str):
    """The two byte arrays in the matrix units' order, value by value; 0 where a row is padding."""
    rows, cols = codes.shape
    rb, kt, kq = -(-rows // 16), -(-cols // 128), -(-cols // 512)
    size = 1024 if fmt == "fp4" else 2048
    out = np.zeros(rb * kt * size, dtype=np.uint8)
    for r in range(rows):
        for c in range(cols):
            t, k = (r // 16 * kt + c // 128) * size, c % 128
            if fmt == "fp4":
                out[t + 16 * (16 * (k // 32) + r % 16) + k % 32 // 2] |= codes[r, c] << (4 * (k % 2))
            else:
                out[t + 1024 * (k // 64) + 16 * (16 * (k // 16 % 4) + r % 16) + k % 16] = codes[r, c]
    sc = np.zeros((rb, kq, 4, 16, 4), dtype=np.uint8)  # [block of rows][group][block][row][tile]
    sc[:] = 127
    for r in range(rows):
        for b in range(scales.shape[1]):
            sc[r // 16, b // 16, b % 4, r % 16, b // 4 % 4] = scales[r, b]
    return out, sc.reshape(-1)


def norm_ref(x, residual, weight, eps):
    """float32 arrays -> y (fp32 steps, the mean in 64 bits) and h."""
    h = x if residual is None else (x + residual).astype(np.float32)
    mean = (h.astype(np.float64) ** 2).mean(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        r = (1 / np.sqrt(mean + eps)).astype(np.float32)
        return ((h * r).astype(np.float32) * weight).astype(np.float32), h


def sample_ref(logits: np.ndarray, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row -> token, logprob, how many tokens are kept, how near u's target came to another
    token's range (relative to what is kept)."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    top = l.max()
    if np.isneginf(top):
        return -1, -np.inf, 0, 1.0
    order = np.argsort(-l, kind="stable")
    if not temperature > 0 or top_k == 1:
        return int(order[0]), 0.0, 1, 1.0
    s = l[order]
    with np.errstate(invalid="ignore", over="ignore"):
        depth = np.where(s == top, 0.0, np.where(np.isneginf(s) | np.isposinf(top), np.inf, (top - s) / temperature))
        w = np.where(np.isfinite(s) | (s == top), np.exp(-depth), 0.0)
    n = len(w) if top_k <= 0 else min(top_k, len(w))
    w = w[:n]
    cum = np.cumsum(w)
    kept = w > 0
    if top_p < 1:
        kept &= (cum - w < top_p * cum[-1]) | (np.arange(n) == 0)
    if min_p > 0:
        kept &= w >= min(min_p, 1.0)
    n = int(kept.sum())
    cum = np.cumsum(w[:n])
    if u >= 1:  # the last token kept of those that weigh e^-64 or more
        at = int((kept[:n] & (depth[:n] < 64)).sum()) - 1
        return int(order[at]), float(np.log(w[at] / cum[-1])), n, 1.0
    u = max(u, 0.0) if u == u else 0.0
    at = min(int((cum <= u * cum[-1]).sum()), n - 1)
    edges = np.concatenate([cum[:-1], [0.0] if u > 0 else []])
    near = np.min(np.abs(edges / cum[-1] - u), initial=1.0)
    return int(order[at]), float(np.log(w[at] / cum[-1])), n, float(near)
