"""Plain reference of the quantised K/V cache, in numpy.

The formats fix a few f32 roundings (a scale's quotient, its reciprocal, the
product with it), which are done in float32 here; everything else is in 64 bits.
"""
from __future__ import annotations

import numpy as np

FLOOR, CEIL = np.float32(2.0 ** -100), np.float32(3.4028234663852886e38)
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _e4m3_values():
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return np.array(v[:-1])  # up to 448; the last place of the grid is the NaN's


E4M3 = _e4m3_values()


def nearest(mag, grid):
    """Index of the grid value nearest to each mag >= 0, ties to the even index,
    past the end the last one."""
    mag = np.asarray(mag, np.float64)
    hi = np.minimum(np.searchsorted(grid, mag), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    down, up = mag - grid[lo], grid[hi] - mag
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def _top(x):
    """Largest magnitude of the last axis (a NaN counts as nothing), clamped."""
    a = np.abs(np.where(np.isnan(x), 0, x)).max(-1).astype(np.float32)
    return np.minimum(np.maximum(a, FLOOR), CEIL)


def quant_fp8(x):
    """(codes uint8, scales float32) of float32 rows [..., head_dim]."""
    x = np.asarray(x, np.float32)
    a = _top(x)
    with np.errstate(over="ignore", invalid="ignore"):
        p = x * (np.float32(448) / a)[..., None]
    code = nearest(np.where(np.isnan(p), 0, np.abs(p)), E4M3).astype(np.uint8)
    code = np.where(np.isnan(p), 0x7F, code | np.where(np.signbit(p), 0x80, 0)).astype(np.uint8)
    return code, (a / np.float32(448)).astype(np.float32)


def quant_mxfp4(x):
    """(codes uint8, two a byte, scale bytes) of float32 rows [..., head_dim]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    a = _top(g).astype(np.float64)
    s = np.ceil(np.log2(a / 6))
    # log2 may round at an exact power of two: settle by the defining inequality
    s = np.where(a / 2.0 ** (s - 1) <= 6, s - 1, s)
    s = np.where(a / 2.0 ** s > 6, s + 1, s)
    v = g.astype(np.float64) / 2.0 ** s[..., None]
    code = nearest(np.abs(v), E2M1) | np.where(np.signbit(v), 8, 0)
    code = code.reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, (s + 127).astype(np.uint8)


def quant(x, fmt):
    return quant_fp8(x) if fmt == "fp8" else quant_mxfp4(x)


def held_fp8(codes, scales):
    """The values held, in 64 bits."""
    mag = np.append(E4M3, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag) * scales.astype(np.float64)[..., None]


def held_mxfp4(codes, scales):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -E2M1[c & 7], E2M1[c & 7])
    f = 2.0 ** (scales.astype(np.float64) - 127)
    return (v.reshape(*scales.shape, 32) * f[..., None]).reshape(v.shape)


def held(codes, scales):
    return held_fp8(codes, scales) if scales.dtype == np.float32 else held_mxfp4(codes, scales)


def read(codes, scales, table, cu, rows):
    """[rows, heads, head_dim] in 64 bits; NaN where a row belongs to no sequence."""
    blocks, page = codes.shape[:2]
    values = held(codes, scales)
    out = np.full((rows, codes.shape[2], values.shape[-1]), np.nan)
    for s in range(len(cu) - 1):
        for t in range(cu[s + 1] - cu[s]):
            if cu[s] + t >= rows:
                continue
            b = table[s, t // page] if t // page < table.shape[1] else -1
            out[cu[s] + t] = values[b, t % page] if 0 <= b < blocks else 0.0
    return out
