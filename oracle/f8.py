"""e4m3 quantisation, norm and products, oracle side (test infrastructure only), in numpy float64.

The definition is the C ABI's (include/qtip_moe.h, "e4m3"): blocks of 128 (activations) or 128 x 128 (weights), e4m3
codes, fp32 scales.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
TINY = 2.0 ** -126


def code_value(c):
    """What one code byte stands for."""
    e, m = (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return np.nan
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if c & 128 else v


TABLE = np.array([code_value(c) for c in range(256)])
GRID = TABLE[:127]


def scale_of(amax, rule):
    """The fp32 scale of a block whose largest magnitude is the finite fp32 number amax."""
    amax = float(amax)
    if rule == "amax":
        return max(float(np.float32(amax / 448.0)), TINY)
    s = TINY
    while 448.0 * s < amax:
        s *= 2.0
    return s


def codes_of(x, scale):
    """The codes nearest to x / scale, a tie the even code."""
    ratio = np.abs(x) / scale
    middle = (GRID[1:] + GRID[:-1]) / 2
    code = np.searchsorted(middle, ratio, side="left")           # middles below the ratio
    tie = ratio == middle[np.minimum(code, len(middle) - 1)]
    code = np.where(tie & (code % 2 == 1), code + 1, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def quantise(x, rule="amax", block_rows=1):
    """(codes [rows][cols rounded up to 16], scales [row blocks][blocks] float32) of a 2-D float64 array."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    codes = np.zeros((rows, -(-cols // 16) * 16), np.uint8)
    scales = np.zeros((-(-rows // block_rows), -(-cols // BLOCK)), np.float32)
    for i in range(scales.shape[0]):
        for b in range(scales.shape[1]):
            at = slice(i * block_rows, (i + 1) * block_rows), slice(b * BLOCK, min((b + 1) * BLOCK, cols))
            v = x[at]
            if not np.all(np.isfinite(v)):
                scales[i, b] = np.nan
                continue
            scales[i, b] = scale_of(np.max(np.abs(v)), rule)
            codes[at] = codes_of(v, float(scales[i, b]))
    return codes, scales


def decode(codes, scales, block_rows=1):
    """The float64 values of codes [rows][cols] under their scales."""
    v = TABLE[np.asarray(codes)]
    s = np.asarray(scales, np.float64)
    r = np.arange(v.shape[0]) // block_rows
    c = np.arange(v.shape[1]) // BLOCK
    return v * s[r][:, c]


def rms_norm(h, weight, eps):
    """y = h w / sqrt(mean h^2 + eps), rows of float64."""
    h = np.asarray(h, np.float64)
    return h * np.asarray(weight, np.float64) / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
