"""The oracle's norms (CPU only): closed forms, and every gradient against
central differences of the forward formula in float64."""

import numpy as np
import pytest

from oracle import norm as ON


def test_a_row_of_two():
    """x = (a - d, a + d): mean a, variance d^2."""
    a, d = 3.0, 0.25
    y, mean, rstd = ON.forward(np.array([[a - d, a + d]]), np.array([2.0, 4.0]), np.array([1.0, -1.0]), eps=0.0)
    assert mean[0] == a and rstd[0] == 1 / d
    assert np.array_equal(y, [[-2.0 + 1.0, 4.0 - 1.0]])
    y, mean, rstd = ON.forward(np.array([[3.0, 4.0]]), eps=0.0, kind="rms")
    assert mean[0] == 0 and np.isclose(rstd[0], np.sqrt(2) / 5) and np.allclose(y, np.array([[3, 4]]) * np.sqrt(2) / 5)


def test_shift_and_scale():
    """The layer norm does not see a shift of the row, and (eps = 0) neither norm a factor."""
    x = np.random.default_rng(1).standard_normal((3, 17))
    assert np.allclose(ON.forward(x, eps=0)[0], ON.forward(5 * x + 7, eps=0)[0])
    assert np.allclose(ON.forward(x, eps=0, kind="rms")[0], ON.forward(5 * x, eps=0, kind="rms")[0])


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("affine", [False, True])
def test_gradients_by_differences(kind, affine):
    r = np.random.default_rng(2)
    m, n, eps, h = 4, 7, 1e-3, 1e-6
    x, dy = r.standard_normal((m, n)) + 0.5, r.standard_normal((m, n))
    w, b = (1 + 0.3 * r.standard_normal(n), r.standard_normal(n)) if affine else (None, None)

    def loss(x, w, b):
        return (ON.forward(x, w, b, eps, kind)[0] * dy).sum()

    _, mean, rstd = ON.forward(x, w, b, eps, kind)
    dx, dw, db = ON.backward(dy, x, mean, rstd, w, kind)
    # central differences: off by h^2 times a third derivative (under 100 here) and 2^-52 / h of the loss
    for i in range(m):
        for j in range(n):
            e = np.zeros((m, n))
            e[i, j] = h
            assert abs((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h) - dx[i, j]) < 1e-7
    if affine:
        for j in range(n):
            e = np.zeros(n)
            e[j] = h
            assert abs((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h) - dw[j]) < 1e-7
            assert abs((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h) - db[j]) < 1e-7
