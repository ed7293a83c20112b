"""Pins of the microscaled oracle (oracle/mx.py) by what the formats say of
themselves: every value a format holds restores to itself, rounding is at most
half a step, ties go to the even element, scales are the smallest that hold the
block."""
import numpy as np
import pytest

from oracle import mx

FORMATS = ("int8", "e4m3", "e2m1")
TOP = {"int8": 127 / 64, "e4m3": 448.0, "e2m1": 6.0}
HALF_STEP = {"int8": 2.0 ** -7, "e4m3": 2.0 ** -4, "e2m1": 2.0 ** -2}  # int8: absolute, before the scale


def test_element_tables():
    assert list(mx.TABLE["e2m1"]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = mx.TABLE["e4m3"]
    assert t[0] == 0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[126] == 448.0 and len(t) == 127
    for f in FORMATS:
        assert mx.TABLE[f][-1] == TOP[f] and (np.diff(mx.TABLE[f]) > 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_of_the_format_restore_exactly(fmt):
    tab = np.concatenate([mx.TABLE[fmt], -mx.TABLE[fmt][1:]])
    for exp in (-120, -3, 0, 5, 110):
        x = np.zeros((1, -(-len(tab) // 31) * 32))
        for b in range(x.shape[1] // 32):  # the largest value in each block fixes its scale
            part = tab[31 * b:31 * b + 31]
            x[0, 32 * b:32 * b + len(part)] = part
            x[0, 32 * b + 31] = TOP[fmt]
        x *= 2.0 ** exp
        codes, scales = mx.pack(x, fmt)
        assert (scales[0, :x.shape[1] // 32] == 127 + exp).all()
        assert (mx.unpack(codes, scales, fmt) == x).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_rounding_is_at_most_half_a_step_and_nothing_saturates(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 200)) * np.exp(rng.standard_normal((50, 1)) * 5)
    codes, scales = mx.pack(x, fmt)
    y = mx.unpack(codes, scales, fmt)
    s = 2.0 ** (np.repeat(scales.astype(float), 32, -1)[:, :200] - 127)
    assert (np.abs(x) <= TOP[fmt] * s).all()
    amax = np.abs(np.pad(x, ((0, 0), (0, 24))).reshape(50, 7, 32)).max(-1)
    assert (amax > TOP[fmt] * 2.0 ** (scales[:, :7].astype(float) - 128)).all()  # half the scale would not do
    if fmt == "int8":
        assert (np.abs(x - y) <= HALF_STEP[fmt] * s).all()
    else:
        low = {"e4m3": 2.0 ** -10, "e2m1": 0.25}[fmt]
        assert (np.abs(x - y) <= np.maximum(HALF_STEP[fmt] * np.abs(x), low * s)).all()


def test_ties_go_to_the_even_element():
    x = np.zeros((1, 32))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    y = mx.unpack(*mx.pack(x, "e2m1"), "e2m1")
    assert list(y[0, :8]) == [6, 0, 1, 1, 2, 2, 4, 4]
    x = np.zeros((1, 32))
    x[0, :5] = [1, 0.5 / 64, 1.5 / 64, -2.5 / 64, 3.5 / 64]
    y = mx.unpack(*mx.pack(x, "int8"), "int8")
    assert list(y[0, :5] * 64) == [64, 0, 2, -2, 4]


@pytest.mark.parametrize("fmt", FORMATS)
def test_special_blocks(fmt):
    x = np.ones((1, 160))
    x[0, 3] = np.inf
    x[0, 40] = np.nan
    x[0, 64:96] = 0
    x[0, 96:128] = 2.0 ** -133
    codes, scales = mx.pack(x, fmt)
    assert list(scales[0, :2]) == [255, 255] and scales[0, 2] == 0 and scales[0, 3] == 0
    assert scales.shape[1] == 8 and (scales[0, 5:] == 0).all()
    y = mx.unpack(codes, scales, fmt)
    assert np.isnan(y[0, :64]).all() and (y[0, 64:96] == 0).all() and (y[0, 96:128] == 2.0 ** -133).all() == (fmt != "e2m1")
    assert (y[0, 128:] == 1).all()
    half = codes[0, :64] if fmt != "e2m1" else codes[0, :32]
    assert (half == 0).all()
