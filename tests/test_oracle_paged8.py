"""Pins of the 8-bit part of oracle.paged: hand values, closed forms, and a second statement of the rounding."""
import numpy as np
import pytest
import torch

from oracle import paged


def test_e4m3_hand_values():
    x = [0.0, 1.0, 1.0625, 1.0626, 1.1875, 448.0, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 2.5 * 2.0 ** -9, -0.3]
    y = [0.0, 1.0, 1.0, 1.125, 1.25, 448.0, 2.0 ** -6, 2.0 ** -9, 0.0, 2.0 ** -8, 2.0 ** -8, -0.3125]
    np.testing.assert_array_equal(paged.e4m3(x), y)
    assert np.isnan(paged.e4m3([np.inf, -np.inf, np.nan])).all()


def test_e4m3_is_the_type_of_that_name():
    rng = np.random.default_rng(0)
    x = (rng.normal(size=20000) * np.exp(rng.normal(size=20000) * 4)).astype(np.float32)
    x = x[np.abs(x) <= 448]
    np.testing.assert_array_equal(paged.e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(paged.e4m3(every), every)


@pytest.mark.parametrize("top,e", [(0.0, -64), (448.0, 0), (448.0001, 1), (447.9, 0), (224.0, -1), (225.0, 0), (1.0, -8),
                                   (1.75, -8), (1.7500001, -7), (3.3e38, 120), (1e-30, -64)])
def test_exponent_hand_values(top, e):
    assert paged.exponent(top) == e
    assert top <= np.ldexp(448.0, e) and (e == -64 or top > np.ldexp(448.0, e - 1))


def test_append_keeps_four_significant_bits():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(40, 2, 128)) * np.exp(rng.normal(size=(40, 2, 1)))
    v, e = paged.append8(np.full((3, 2, 16, 128), 7.0), np.zeros((3, 2, 1)), x, np.arange(40) + 2)
    wide = paged.widened(v, e).transpose(0, 2, 1, 3).reshape(48, 2, 128)
    step = np.ldexp(1.0, np.repeat(e[:, :, 0], 16, 0)[2:42] - 9)
    assert (np.abs(wide[2:42] - x) <= np.maximum(2.0 ** -4 * np.abs(x), step[..., None] / 2)).all()
    assert (np.abs(v) <= 448).all()


def test_append_row_by_row_is_append_at_once():
    """But for what lies below 2^-6 of a group's scale, where rounding again may move it by half a step each time."""
    rng = np.random.default_rng(2)
    x = rng.normal(size=(16, 1, 128)) * np.exp(rng.normal(size=(16, 1, 1)))
    one = paged.append8(np.zeros((1, 1, 16, 128)), np.zeros((1, 1, 1)), x, np.arange(16))
    v, e = np.zeros((1, 1, 16, 128)), np.full((1, 1, 1), 99)
    for t in range(16):
        v, e = paged.append8(v, e, x[t:t + 1], [t])
    np.testing.assert_array_equal(e, one[1])
    big = np.abs(one[0]) >= 2.0 ** -6
    np.testing.assert_array_equal(v[big], one[0][big])
    assert (np.abs(v - one[0]) <= 2.0 ** -8).all()


def test_append_begins_a_group_anew_and_leaves_the_rest():
    v, e = np.full((2, 1, 16, 128), 3.0), np.full((2, 1, 1), 50)
    x = np.ones((2, 1, 128))
    v1, e1 = paged.append8(v, e, x, [16, 17])
    assert (v1[0] == 3).all() and e1[0] == 50 and e1[1] == -8 and (v1[1, 0, :2] == 256).all() and (v1[1, 0, 2:] == 3).all()
    v2, e2 = paged.append8(v1, e1, x * 4, [18])     # grows by two: the rows in front are rounded to a quarter
    assert e2[1] == -6 and (v2[1, 0, :3].T == [64, 64, 256]).all() and (v2[1, 0, 3:] == 3).all()
    v3, e3 = paged.append8(v2, e2, x * np.nan, [19])
    assert e3[1] == -6 and np.isnan(v3[1, 0, 3]).all() and (v3[1, 0, :3].T == [64, 64, 256]).all()
