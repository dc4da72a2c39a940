"""Oracle of the 4-bit operands (MX4), in float64.

Test infrastructure, like the rest of this package: the definitions, no code
shared with the HIP path. A block is 32 values along k; 2**e is its power of two
with e = floor(log2(max |x|)) - 2, held as the byte e + 127; elements are
rounded to nearest, ties to the even code, and clamped at 6.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def blocks(k):
    return -(-k // BLOCK)


def quantize(x):
    """(codes, scales) of x (rows, k) float64: one code (0..15) per value, shape
    (rows, 32 * blocks), zeros behind k; one byte per block."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    nb = blocks(k)
    codes = np.zeros((rows, nb * BLOCK), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        bad = ~np.isfinite(v).all(axis=1)
        v = np.where(bad[:, None], 0.0, v)
        top = np.abs(v).max(axis=1)
        e = np.where(top > 0, np.frexp(top)[1] - 3, -127)  # frexp: top = f * 2**i, 0.5 <= f < 1
        e = np.maximum(e, -127)
        a = np.abs(v) / np.ldexp(1.0, e)[:, None]
        code = np.zeros(a.shape, np.int64)
        for i in range(7):
            mid = (GRID[i] + GRID[i + 1]) / 2
            # the upper neighbour above the middle, and at it where its code is even
            code = np.where((a > mid) | ((a == mid) & ((i + 1) % 2 == 0)), i + 1, code)
        code = code + np.where(np.signbit(v), 8, 0)
        code[bad] = 0
        codes[:, b * BLOCK:b * BLOCK + v.shape[1]] = code
        scales[:, b] = np.where(bad, 255, e + 127)
    return codes, scales


def pack(codes, scales):
    """The stored form: two codes a byte (the even one low), scales padded with
    zeros to a multiple of 16."""
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    pad = -scales.shape[1] % 16
    return packed.astype(np.uint8), np.pad(scales, ((0, 0), (0, pad)))


def unpack(packed, scales):
    """pack's inverse."""
    codes = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    return codes, scales[:, :codes.shape[1] // BLOCK]


def values(codes, scales, k):
    """The float64 values (rows, k) that codes and scales stand for."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    p = np.ldexp(1.0, scales.astype(np.int64) - 127)
    p = np.where(scales == 255, np.nan, p)
    return (v * np.repeat(p, BLOCK, axis=1))[:, :k]


def mm(a, b, bias=None):
    """a (m, k) @ b (n, k).T + bias of the values, float64."""
    out = a @ b.T
    return out if bias is None else out + bias
