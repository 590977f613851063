"""The oracle's balance where a row's sigmoids are all small beside the 1e-20 of their
sum: its gradient against differences, and what is left of it in closed form."""

import numpy as np
import pytest

from oracle import block as B


@pytest.mark.parametrize("level", [-36, -46, -50, -80])
def test_gradient_of_small_sigmoids(level):
    g = np.random.Generator(np.random.PCG64(-level))
    T, E, k = 6, 5, 2
    z = level + 0.3 * g.normal(size=(T, E))
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    r = B.balance(z, ids, True)
    f = E * r["counts"][0] / (k * T)
    h = 1e-5

    def value(z):
        return f @ B.balance(z, ids, True)["probs"][0]

    for t in range(T):
        for e in range(E):
            a, b = z.copy(), z.copy()
            a[t, e] += h
            b[t, e] -= h
            # (Second order: h^2 of the slope; the two losses' rounding over 2 h.)
            rounding = 2.0 ** -52 * max(r["loss"][0], 1e-300) / h * 8 + 2.0 ** -52 * abs(level) / h * abs(r["grad"][t, e])
            assert abs((value(a) - value(b)) / (2 * h) - r["grad"][t, e]) <= 2 * h * h * abs(f).max() + rounding


def test_what_is_left_far_down():
    """Where the sum is far below 1e-20, p is the sigmoid times 1e20 and the rest of
    f - sum f p is f."""
    z, ids = np.full((4, 4), -80.0), np.arange(4).reshape(4, 1)
    r = B.balance(z, ids, True)
    assert np.allclose(r["grad"], np.exp(-80.0) * 1e20 / 4, rtol=1e-12)
