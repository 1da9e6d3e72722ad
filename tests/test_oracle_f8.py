"""The e4m3 oracle against hand-worked values and independent formulas."""
import math
import struct

import numpy as np
import pytest

from oracle import f8


def test_the_codes_of_the_format():
    assert len(f8.GRID) == 127 and np.all(np.diff(f8.GRID) > 0)
    assert f8.GRID[1] == 2.0 ** -9 and f8.GRID[8] == 2.0 ** -6 and f8.GRID[56] == 1.0 and f8.GRID[126] == 448.0
    assert np.isnan(f8.TABLE[127]) and np.isnan(f8.TABLE[255])
    assert f8.TABLE[0x80 + 57] == -1.125 and math.copysign(1.0, f8.TABLE[0x80]) == -1.0


def test_quantise_hand_worked_block():
    # amax 896: scale 2 by both rules; ratios are the values halved
    v = np.zeros((1, 128))
    v[0, :9] = [896.0, -2.0, 2.125, 2.375, -2.374, 832.0, 2.0 ** -9, 2.0 ** -9 * 1.001, -0.0]
    for rule in ("amax", "pow2"):
        codes, scales = f8.quantise(v, rule)
        assert scales.tolist() == [[2.0]]
        # 1.0625: a tie of 1 and 1.125, to the even 1; 1.1875 to the even 1.25; 416 is a code
        assert f8.TABLE[codes[0, :9]].tolist() == [448.0, -1.0, 1.0, 1.25, -1.125, 416.0, 0.0, 2.0 ** -9, -0.0]
        assert not codes[0, 9:].any()


@pytest.mark.parametrize("amax,want", [(448.0, 0), (449.0, 1), (447.0, 0), (1.75, -8), (1.7500001, -7), (1.0, -8),
                                       (2.0, -7), (2.0 ** -126, -126), (0.0, -126), (3.4e38, 120)])
def test_powers_of_two(amax, want):
    s = f8.scale_of(np.float32(amax), "pow2")
    assert s == 2.0 ** want
    assert amax <= 448 * s and (s == f8.TINY or 448 * s / 2 < amax)


def test_amax_scale_is_the_rounded_quotient():
    rng = np.random.default_rng(0)
    for bits in rng.integers(1 << 27, 0x7f800000, 2000):
        a = struct.unpack("<f", struct.pack("<I", int(bits)))[0]
        s = f8.scale_of(a, "amax")
        near = [float(np.nextafter(np.float32(s), np.float32(d))) for d in (-np.inf, np.inf)]
        assert s == f8.TINY or all(abs(448 * s - a) <= abs(448 * t - a) for t in near)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rule", ["amax", "pow2"])
def test_decoded_values_are_near_and_stay(rule, block_rows):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((130, 333)) * np.exp2(rng.integers(-9, 9, (130, 1)))).astype(np.float32).astype(float)
    codes, scales = f8.quantise(x, rule, block_rows)
    assert codes.shape == (130, 336) and not codes[:, 333:].any()
    v = f8.decode(codes, scales, block_rows)[:, :333]
    s = scales.astype(float)[np.arange(130) // block_rows][:, np.arange(333) // 128]
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), s * 2.0 ** -10) * (1 + 1e-12))
    if rule == "pow2" and block_rows == 1:      # on the grid already: the same values again
        again = f8.quantise(v, rule, block_rows)
        assert np.array_equal(f8.decode(*again, block_rows)[:, :333], v)


def test_blocks_that_hold_no_number():
    x = np.ones((2, 300))
    x[0, 5], x[1, 299] = np.inf, np.nan
    codes, scales = f8.quantise(x)
    assert np.isnan(scales).tolist() == [[True, False, False], [False, False, True]]
    assert not codes[0, :128].any() and np.all(f8.TABLE[codes[0, 128:300]] == 448.0)
    assert np.isnan(f8.decode(codes, scales)[0, :128]).all()


def test_norm_of_a_row_by_hand():
    y = f8.rms_norm([[3.0, -4.0, 0.0, 0.0]], [1.0, 2.0, 1.0, 1.0], 0.0)
    assert y.tolist() == [[1.2, -3.2, 0.0, 0.0]]            # mean of squares 25 / 4
    assert f8.rms_norm([[3.0, -4.0]], [1.0, 1.0], 12.5)[0].tolist() == [0.6, -0.8]
