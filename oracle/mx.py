"""MXFP4 quantisation and products, oracle side (test infrastructure only), in numpy float64.

The definition is the C ABI's (include/qtip_moe.h, "MXFP4"): blocks of 32, e2m1 codes, e8m0 scales.
"""
from __future__ import annotations

import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise_block(v, rule):
    """(16 bytes of codes, scale byte, 32 values) of one block of float64 values."""
    v = np.asarray(v, np.float64)
    if not np.all(np.isfinite(v)):
        return np.zeros(16, np.uint8), 255, np.full(32, np.nan)
    top = float(np.max(np.abs(v)))
    byte = 0
    if top > 0:
        mant, exp = math.frexp(top)                       # top = mant 2^exp, mant in [1/2, 1)
        byte = exp - 1 - 2 + 127 + (1 if rule == "nearest" and mant >= 0.875 else 0)
        byte = min(max(byte, 0), 254)
    scale = math.ldexp(1.0, byte - 127)
    codes = np.zeros(32, np.int64)
    for i, x in enumerate(v):
        a = min(abs(x) / scale, 6.0)
        far = np.abs(GRID - a)
        best = np.flatnonzero(far == far.min())
        c = int(best[0]) if len(best) == 1 or best[0] % 2 == 0 else int(best[1])   # a tie: the even code
        codes[i] = c | (8 if np.signbit(x) else 0)
    values = np.where(codes & 8, -GRID[codes & 7], GRID[codes & 7]) * scale
    return (codes[0::2] | (codes[1::2] << 4)).astype(np.uint8), byte, values


def quantise(x, rule="floor"):
    """(codes [rows][16 blocks], scales [rows][blocks], values [rows][cols]) of a 2-D array."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blocks = -(-cols // 32)
    pad = np.zeros((rows, blocks * 32))
    pad[:, :cols] = x
    codes = np.zeros((rows, blocks * 16), np.uint8)
    scales = np.zeros((rows, blocks), np.uint8)
    values = np.zeros((rows, blocks * 32))
    for r in range(rows):
        for b in range(blocks):
            c, s, v = quantise_block(pad[r, 32 * b:32 * b + 32], rule)
            codes[r, 16 * b:16 * b + 16], scales[r, b], values[r, 32 * b:32 * b + 32] = c, s, v
    return codes, scales, values[:, :cols]


def decode(codes, scales):
    """The float64 values of codes [..., 16 blocks] and scales [..., blocks]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], codes.shape[-1] * 2)
    v = np.where(c & 8, -GRID[c & 7], GRID[c & 7])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def silu(g):
    return g / (1.0 + np.exp(-g))


def swiglu_bound(g, u, dg, du):
    """|error| of silu(g) u from errors dg, du of g and u: |silu'| <= 1.1, |silu(g)| <= |g|."""
    return 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du
