"""Pins of the 8-bit checkpoint oracle: hand-made blocks, the nearest integer
in rationals, the error bound, and the edges of the range."""

from fractions import Fraction

import numpy as np
import pytest

import oracle
from oracle import act8


def test_hand_made_block():
    x = np.zeros((1, 64), np.float32)
    x[0, :5] = [127.0, -127.0, 63.5, 1.5, -0.5]
    codes, scale = act8.encode(x)
    assert scale[0, 0] == 1.0
    # ties go to even: 63.5 -> 64, 1.5 -> 2, -0.5 -> 0
    assert codes[0, :6].tolist() == [127, -127, 64, 2, 0, 0]


def test_bf16_codes_are_the_nearest_integers_ties_to_even():
    rng = np.random.default_rng(11)
    bits = oracle.bf16_rne_bits(rng.standard_normal((200, 64)).astype(np.float32))
    bits[:, 1] = bits[:, 0] - 0x80          # half of the first: often a tie
    v = oracle.bf16_bits_to_f64(bits)
    codes, _ = act8.encode(bits)
    for i in range(bits.shape[0]):
        a = Fraction(float(np.abs(v[i]).max()))
        for j in range(64):
            q = Fraction(float(v[i, j])) * 127 / a
            assert codes[i, j] == round(q), (i, j)    # Fraction rounds half to even


@pytest.mark.parametrize("cols", [1, 63, 64, 65, 200])
def test_error_is_at_most_half_a_step(cols):
    rng = np.random.default_rng(cols)
    x = (rng.standard_normal((37, cols)) * 10.0 ** rng.integers(-20, 20, (37, 1))).astype(np.float32)
    codes, scale = act8.encode(x)
    back = codes.astype(np.float64) * np.repeat(scale, 64, 1)[:, :cols]
    step = np.repeat(scale, 64, 1)[:, :cols].astype(np.float64)
    # half a step, the scale's rounding on up to 127 steps, the quotient's
    assert np.all(np.abs(back - x) <= step * (0.5 + 127 * 2.0 ** -24 + 127 * 2.0 ** -23))
    assert np.abs(codes.astype(int)).max() == 127


def test_edges_of_the_range():
    big = np.float32(3.3895314e38)
    x = np.zeros((5, 64), np.float32)
    x[0] = 2.0 ** -101                   # below the smallest block
    x[1, 3] = 2.0 ** -100                # the smallest block
    x[2, :2] = [big, -big]               # the largest bf16 values
    x[3, 7] = np.inf
    x[4, 9] = np.nan
    codes, scale = act8.encode(x)
    assert scale[0, 0] == 0 and not codes[0].any()
    assert codes[1, 3] == 127 and scale[1, 0] > 0
    assert codes[2, :2].tolist() == [127, -127] and np.isfinite(scale[2, 0])
    assert np.isnan(scale[3, 0]) and np.isnan(scale[4, 0]) and not codes[3:].any()
    assert np.isnan(act8.decode_f32(codes, scale)[3:]).all()
