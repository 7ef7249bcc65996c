"""Plain 64-bit reference of the microscaled 4-bit formats (numpy), for the tests.

Values are built from the formats' definitions: E2M1 codes, UE8M0 / E4M3 scale bytes and the
blocked scale layout of include/csa.h.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) for e in range(16) for m in range(8)])
E4M3[127] = np.nan  # bytes 0..127


def nearest_even(a, grid):
    """Index of the grid value nearest to a >= 0 (ascending grid; ties to the even index; the last
    one beyond the grid)."""
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def encode(x, fmt, g=None):
    """float32 x [rows, cols] -> (codes [rows, cols], scale bytes [rows, cols / block])."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK[fmt], BLOCK[fmt])
    with np.errstate(all="ignore"):
        amax = np.fmax.reduce(np.abs(b), axis=2, initial=0.0)  # NaNs are left out
        if fmt == "mxfp4":
            amax = np.minimum(amax.astype(np.float64), 2.0 ** 128)  # an infinity counts as 2^128
            E = np.full(amax.shape, -127)
            for e in range(-127, 128):  # smallest E with amax <= 6 * 2^E, at most 127
                E = np.where(amax > 6.0 * 2.0 ** (e - 1), e, E)
            E = np.where(amax > 0, np.maximum(E, -127), -127)
            y = b.astype(np.float64) / 2.0 ** E[..., None].astype(np.float64)
            sbytes = (E + 127).astype(np.uint8)
        else:
            g = np.float32(g)
            d = (amax / (np.float32(6.0) * g)).astype(np.float32)
            sbytes = nearest_even(np.minimum(d, np.float32(448.0)), E4M3[:127]).astype(np.uint8)
            T = (E4M3[sbytes].astype(np.float32) * g).astype(np.float32)[..., None]
            y = np.where(T > 0, (b / T).astype(np.float32), np.float32(0.0)).astype(np.float64)
    codes = nearest_even(np.where(np.isnan(y), 6.0, np.minimum(np.abs(y), 6.0)), GRID)
    sign = np.where(np.isnan(y), False, np.signbit(y))
    return (codes + 8 * sign).astype(np.uint8).reshape(rows, cols), sbytes


def scale_values(sbytes, fmt):
    return 2.0 ** (sbytes.astype(np.float64) - 127) if fmt == "mxfp4" else E4M3[sbytes & 127]


def decode(codes, sbytes, fmt, g=None):
    """The float64 values (NVFP4: code * s * g in full)."""
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    v = v.reshape(codes.shape[0], -1, BLOCK[fmt]) * scale_values(sbytes, fmt)[..., None]
    return v.reshape(codes.shape) * (1.0 if g is None else float(np.float32(g)))


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1)


def block_scales(sbytes):
    """Row-major scale bytes -> the blocked layout, one byte at a time."""
    rows, nb = sbytes.shape
    R, A = -(-rows // 128), -(-nb // 4)
    out = np.zeros(R * A * 512, np.uint8)
    r = np.arange(rows)[:, None]
    b = np.arange(nb)[None, :]
    at = ((r // 128) * A + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    out[at] = sbytes
    return out
