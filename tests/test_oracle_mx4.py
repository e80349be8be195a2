"""The oracle's 4-bit matrices (CPU only): every rounding case by hand, and the
nearest of all values by brute force."""

import numpy as np
import pytest

from oracle import mx4 as Q


def one_block(v):
    codes, scales = Q.quantize(np.array([v], dtype=float))
    return Q.values(codes, scales, len(v))[0], int(scales[0, 0])


def test_halfway_cases():
    """With 4 in the block its scale is 1."""
    x = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 0.2500001, 0.7499999, 5.0000001, 7.9, -0.25, -5, -7.9]
    got, scale = one_block(x)
    assert scale == 127
    assert got.tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 0.5, 0.5, 6, 6, 0, -4, -6]


@pytest.mark.parametrize("top,s", [(1.0, -2), (1.99, -2), (2.0, -1), (3.0, -1), (4.0, 0), (7.99, 0), (8.0, 1), (448.0, 6),
                                   (2.0 ** -125, -127), (2.0 ** -126, -127), (2.0 ** -149, -127), (2.0 ** 127, 125)])
def test_scales(top, s):
    assert one_block([top, 0.0, -top / 3])[1] == s + 127


def test_zeros_nan_and_infinity():
    assert one_block([0.0] * 5)[1] == 0
    for v in (np.nan, np.inf, -np.inf):
        got, scale = one_block([1.0, v, 2.0])
        assert scale == 255 and np.isnan(got).all()
    codes, scales = Q.quantize(np.concatenate([np.ones((1, 32)), np.full((1, 3), np.nan)], axis=1))
    assert np.isfinite(Q.values(codes, scales, 35)[0, :32]).all() and scales[0, :3].tolist() == [125, 255, 0]


def test_nearest_by_brute_force():
    r = np.random.default_rng(3)
    x = r.standard_normal((40, 70)) * np.exp2(r.integers(-30, 30, (40, 1)))
    codes, scales = Q.quantize(x)
    assert codes.shape == (40, 48) and scales.shape == (40, 16)
    got = Q.values(codes, scales, 70)
    for i in range(40):
        for j in range(70):
            grid = Q.MAGNITUDES * 2.0 ** (int(scales[i, j // 32]) - 127)
            assert abs(abs(got[i, j]) - abs(x[i, j])) == np.abs(grid - abs(x[i, j])).min()
            assert got[i, j] * x[i, j] >= 0
    top = np.abs(x[:, :32]).max(axis=1) * 2.0 ** -(scales[:, 0].astype(float) - 127)
    assert (top >= 4).all() and (top < 8).all()


def test_layout():
    """Element 2i in the low half of byte i; zeros behind the end."""
    x = np.zeros((2, 34))
    x[0, 0], x[0, 1], x[0, 33], x[1, 32] = 4, -6, 1, 0.5
    codes, scales = Q.quantize(x)
    assert codes[0, 0] == 6 | (15 << 4) and codes[0, 16] == 6 << 4 and codes[1, 16] == 6
    assert scales[0].tolist() == [127, 125] + [0] * 14 and scales[1].tolist() == [0, 124] + [0] * 14
    assert not codes[:, 17:].any()
