"""Plain forms of the microscaled operators in 64 bits, for the tests: by
search in the list of representable values, sharing nothing with the library."""
from __future__ import annotations

import numpy as np

FP4, FP8 = 1, 2
EMAX = {FP4: 2, FP8: 8}
_E4M3 = [(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)]
GRID = {FP4: np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6]), FP8: np.array(_E4M3)}


def values(fmt):
    """The value of every code: 16 (FP4) or 256 (FP8, NaN at 0x7f and 0xff)."""
    g = GRID[fmt] if fmt == FP4 else np.append(GRID[fmt], np.nan)
    return np.concatenate([g, -g])


def quantize(x, fmt):
    """(codes [rows, K] one a byte, scale bytes [rows, K/32]) of x [rows, K]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    m = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        s = np.where(m > 0, np.floor(np.log2(np.where((m > 0) & ~bad, m, 1.0))) - EMAX[fmt], -127)
    # log2 of a 53-bit number just below a power of two may round up: take the power that fits
    s = np.where((m > 0) & ~bad & (2.0 ** (s + EMAX[fmt]) > m), s - 1, s)
    s = np.clip(s, -127, 127)
    a = np.abs(np.where(bad[..., None], 0.0, b)) / 2.0 ** s[..., None]
    g = GRID[fmt]
    hi = np.clip(np.searchsorted(g, a), 0, len(g) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = g[hi] - a, a - g[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= g[-1], len(g) - 1, code)
    code = code + np.where(np.signbit(b), 8 if fmt == FP4 else 128, 0)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def pack(codes, fmt):
    """One code a byte -> the stored bytes."""
    return codes if fmt == FP8 else codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(stored, fmt):
    if fmt == FP8:
        return stored
    return np.stack([stored & 15, stored >> 4], -1).reshape(stored.shape[0], -1)


def dequantize(codes, scales, fmt):
    """Values of unpacked codes [rows, K] and scale bytes [rows, K/32], fp64."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return values(fmt)[codes] * np.repeat(s, 32, axis=1)


def tile_scales(scales):
    """[rows, blocks] -> the flat plane of 128 x 4 tiles, padding 0; byte by byte."""
    rows, nb = scales.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    out = np.zeros(rt * kt * 512, np.uint8)
    for r in range(rows):
        for b in range(nb):
            out[((r // 128) * kt + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4] = scales[r, b]
    return out
