"""Pins of the oracle's MXFP4 (E2M1 codes, one power-of-two scale per block of
32): the format's values written out, roundings worked by hand (every midpoint
between two neighbouring values and its neighbours), the scale rule by brute
force over exponents, and the closed-form bound on the rounding error."""
import math

import numpy as np
import pytest

import oracle

MAGS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def test_code_values_follow_the_format():
    v = oracle.e2m1_values()
    assert v[:8].tolist() == MAGS
    assert np.array_equal(v[8:], -v[:8])
    assert np.array_equal(oracle.round_e2m1(v), np.arange(16))


# value -> code: each midpoint goes to the even code, and just off it to the nearer one
TIES = [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)]


@pytest.mark.parametrize("mid,code", TIES)
def test_hand_rounded_midpoints(mid, code):
    i = next(i for i in range(7) if (MAGS[i] + MAGS[i + 1]) / 2 == mid)
    below, above = math.nextafter(mid, 0.0), math.nextafter(mid, 9.0)
    assert oracle.round_e2m1([mid, below, above]).tolist() == [code, i, i + 1]
    assert oracle.round_e2m1([-mid, -below, -above]).tolist() == [code + 8, i + 8, i + 9]


def test_scale_exponent_by_brute_force():
    rng = np.random.default_rng(1)
    for a in list(rng.normal(size=200) * 2.0 ** rng.integers(-60, 60, 200)) + [6.0, 6.0001, 3.0, 0.75]:
        E = oracle.mx_scale_exponent([0.0, a])
        assert E == min(e for e in range(-127, 128) if abs(a) <= 6.0 * 2.0 ** e)
    assert oracle.mx_scale_exponent([0.0, -0.0]) == 0
    assert oracle.mx_scale_exponent([2.0 ** -149]) == -127
    assert oracle.mx_scale_exponent([float(np.finfo(np.float32).max)]) == 126


def test_rounding_error_bound_and_packing():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(20, 96)) * 2.0 ** rng.integers(-3, 4, (20, 96))
    codes, scales = oracle.quantize_mxfp4(x)
    back = oracle.dequantize_mxfp4(codes, scales)
    step = np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)
    # half a step: 1/4 below 2, 1/2 from 2 to 4, 1 from 4 to 6 (in units of the scale)
    a = np.abs(x) / step
    assert np.all(np.abs(back - x) <= step * np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0)))
    assert np.array_equal(oracle.unpack_mxfp4(oracle.pack_mxfp4(codes)), codes)
    assert oracle.pack_mxfp4(np.array([[1, 15]], dtype=np.uint8)).tolist() == [[0xF1]]
    # values of the format are left alone
    c2, s2 = oracle.quantize_mxfp4(back)
    assert np.array_equal(oracle.dequantize_mxfp4(c2, s2), back)


def test_blocks_that_are_not_finite():
    x = np.zeros((1, 96))
    x[0, 3], x[0, 40] = np.inf, np.nan
    codes, scales = oracle.quantize_mxfp4(x)
    assert scales.tolist() == [[255, 255, 127]] and not codes.any()
    assert np.isnan(oracle.dequantize_mxfp4(codes, scales)[0, :64]).all()


@pytest.mark.parametrize("mistake", ["ties away", "truncated", "scale one larger", "no scale"])
def test_a_planted_mistake_shows(mistake):
    rng = np.random.default_rng(3)
    x = np.round(rng.normal(size=(4, 64)) * 8) / 8       # many ties
    codes, scales = oracle.quantize_mxfp4(x)
    good = oracle.dequantize_mxfp4(codes, scales)
    E = scales.astype(float) - 127
    if mistake == "scale one larger":
        E = E + 1
    f = np.repeat(2.0 ** E, 32, axis=1)
    a, mags = np.abs(x) / f, np.array(MAGS)
    if mistake == "ties away":
        c = np.searchsorted((mags[1:] + mags[:-1]) / 2, a, side="right")
    elif mistake == "truncated":
        c = np.searchsorted(mags, a, side="right") - 1
    else:
        c = oracle.round_e2m1(a)
    bad = np.sign(x) * mags[c] * (1.0 if mistake == "no scale" else f)
    assert not np.array_equal(bad, good)
