"""Pins of the 8-bit and 4-bit formats' oracle to arithmetic done another way (exact fractions, one element at a time),
and to hand-worked rows."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import low_precision as lp


def nearest(num: Fraction) -> int:
    return round(num)  # Python rounds a Fraction to the nearest integer, ties to even


@pytest.mark.parametrize("seed", [0, 1])
def test_i8_codes_match_exact_fractions(seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((9, 48)).astype(np.float32)).bfloat16().double().numpy()
    x[0] = 0
    x[1, 0] = 2 * np.abs(x[1, 1:]).max()      # many elements near half steps of a coarse scale
    x[1, 1:4] = x[1, 0] / 2                    # 63.5 steps
    codes, scale = lp.quant_rows_i8(x)
    assert scale[0] == 0 and not codes[0].any()
    for t in range(1, 9):
        s = Fraction(float(np.float32(np.abs(x[t]).max()) / np.float32(127)))
        assert Fraction(scale[t]) == s
        assert [nearest(Fraction(v) / s) for v in x[t]] == codes[t].astype(int).tolist()
        assert np.abs(codes[t]).max() == 127


def test_i8_rows_that_are_not_finite_are_nan_and_tiny_rows_zero():
    x = np.ones((4, 16))
    x[0, 3], x[1, 5] = np.nan, -np.inf
    x[2] = 1e-38
    codes, scale = lp.quant_rows_i8(x)
    assert np.isnan(scale[:2]).all() and scale[2] == 0 and scale[3] > 0
    y = lp.linear_i8(x, np.ones((8, 16)), np.ones(8))
    assert np.isnan(y[:2]).all() and (y[2] == 0).all()


def test_quant4_hand_worked_row():
    # range -1 .. 2: scale bf16(0.2) = 0.2001953125, zero = rint(4.995) = 5
    x = np.zeros(32)
    x[:6] = [-1.0, 2.0, 0.0, 0.31, -0.09, 1.7]
    codes, s, z = lp.quant4(x)
    assert s == 0.2001953125 and z == 5
    assert codes[:6].tolist() == [0, 15, 5, 7, 5, 13]
    assert (codes[6:] == 5).all()                                   # zero is exact
    assert lp.dequant4(codes, s, z)[6:].tolist() == [0.0] * 26


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_quant4_matches_exact_fractions_and_is_within_half_a_step(seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((7, 3, 64)).astype(np.float32) * 2 - (seed == 2)).bfloat16().double().numpy()
    if seed == 1:
        x = np.abs(x)
    codes, s, z = lp.quant4(x)
    for idx in np.ndindex(7, 3):
        fs = Fraction(float(s[idx]))
        lo = Fraction(min(0.0, x[idx].min()))
        fz = min(15, nearest(-lo / fs))
        assert fz == z[idx]
        want = [min(15, max(0, nearest(Fraction(v) / fs) + fz)) for v in x[idx]]
        assert want == codes[idx].tolist()
    err = np.abs(lp.dequant4(codes, s, z) - x)
    # half a step, and at the ends what the rounding of the scale (2^-8 of 15 steps) and of the zero point (half a
    # step) cut off
    assert (err <= s[..., None] * (0.5 + 15 * 2.0 ** -8 + 0.5)).all()


def test_quant4_special_rows():
    x = np.zeros((6, 32))
    x[1] = 5.0                      # constant rows are the top code
    x[2] = -5.0
    x[3, 1], x[4, 2] = np.inf, np.nan
    x[5] = 1e-38
    codes, s, z = lp.quant4(x)
    assert s[0] == 0 and s[5] == 0 and not codes[0].any() and not codes[5].any()
    assert (codes[1] == 15).all() and z[1] == 0 and (codes[2] == 0).all() and z[2] == 15
    assert np.isnan(s[3:5]).all() and not codes[3:5].any()
    assert np.isnan(lp.dequant4(codes, s, z)[3:5]).all()


def test_pack4_places_each_element():
    rng = np.random.default_rng(5)
    codes = rng.integers(0, 16, size=(3, 64)).astype(np.uint8)
    byte = lp.pack4(codes)
    assert byte.shape == (3, 32)
    for e in range(64):
        nib = (e % 8) // 2 + 4 * (e % 2)
        b = byte[:, 4 * (e // 8) + nib // 2]
        assert ((b >> (4 * (nib % 2))) & 15 == codes[:, e]).all()
    assert (lp.unpack4(byte) == codes).all()
