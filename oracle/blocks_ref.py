"""fp64 reference of the cache's 4-bit blocks and of rotary positions.

Written from the definitions in include/lora_attn.h alone, one block and one pair at a time where that is what the
text says; nothing is shared with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
MOST = {"bf16": 125, "f16": 13}


def values(codes, exps):
    """Values of packed codes (..., n / 2) and exponent bytes (..., n / 32); NaN under exponent 255."""
    grid = np.array(E2M1 + [-x for x in E2M1])
    low, high = grid[codes & 15], grid[codes >> 4]
    x = np.stack([low, high], axis=-1).reshape(*codes.shape[:-1], -1)
    scale = np.where(exps == 255, np.nan, np.ldexp(1.0, exps.astype(np.int64) - 127))
    return x * np.repeat(scale, 32, axis=-1)


def exponent_of(a, most):
    """Exponent (not biased) of a block whose largest magnitude is a."""
    if a == 0:
        return -127
    if math.isinf(a):
        return most
    e = math.frexp(a)[1] - 1 - 2
    if a > 7 * math.ldexp(1.0, e):
        e += 1
    return min(max(e, -127), most)


def code_of(x):
    """Nearest code to x, ties to the even one, held at 6."""
    m = min(abs(x), 6.0)
    best = min(range(8), key=lambda c: (abs(E2M1[c] - m), c % 2))
    return best | (8 if math.copysign(1.0, x) < 0 else 0)


def quantize(x, dtype):
    """(codes, exps) of rows (..., n) as stored from rows of `dtype`; a block with a NaN has exponent 255 and no
    particular codes."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(-1, 32)
    codes = np.zeros((len(blocks), 32), dtype=np.uint8)
    exps = np.zeros(len(blocks), dtype=np.uint8)
    for i, b in enumerate(blocks):
        if np.isnan(b).any():
            exps[i] = 255
            continue
        e = exponent_of(float(np.abs(b).max()), MOST[dtype])
        exps[i] = e + 127
        for d, v in enumerate(b):
            codes[i, d] = code_of(math.ldexp(v, -e) if math.isfinite(v) else v)
    packed = codes[:, 0::2] | codes[:, 1::2] << 4
    return packed.reshape(*x.shape[:-1], x.shape[-1] // 2), exps.reshape(*x.shape[:-1], x.shape[-1] // 32)


def rotate(x, positions, freqs, axis=None, interleaved=False, factor=1.0):
    """Rows (rows, heads, dim) with their first 2 * len(freqs) dimensions rotated; positions (axes, rows) integers."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    for j in range(half):
        angle = np.asarray(positions[axis[j] if axis is not None else 0], dtype=np.float64) * freqs[j]
        c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def partners(x, half, interleaved=False):
    """|x| + |the other of its pair| for rotated dimensions, 0 for the rest: what a rotation's rounding goes by."""
    m = np.abs(np.array(x, dtype=np.float64))
    y = np.zeros_like(m)
    if interleaved:
        s = m[..., 0:2 * half:2] + m[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = y[..., 1:2 * half:2] = s
    else:
        s = m[..., :half] + m[..., half:2 * half]
        y[..., :half] = y[..., half:2 * half] = s
    return y
