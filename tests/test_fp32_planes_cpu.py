"""The bounds of plane_cases hold for products of whole planes and fail for products
that lack one, so that a test that uses them sees the difference."""
import numpy as np
import pytest

import plane_cases as P

U = P.U


def test_three_planes_hold_every_bit():
    x = P.numbers(4000, 1)
    assert np.array_equal(sum(P.planes(x, 3)), x)
    p = P.planes(x, 3)
    assert np.all(np.abs(p[1]) <= 2.0 ** -8 * np.abs(x)) and np.all(np.abs(p[2]) <= 2.0 ** -16 * np.abs(x))
    assert np.abs(p[2]).max() > 2.0 ** -18


@pytest.mark.parametrize("kind,units", [((3, 3), P.THREE_BY_THREE), ((3, 2), P.THREE_BY_TWO)])
def test_a_missing_plane_is_seen(kind, units):
    x, y = P.numbers(4000, 2), P.numbers(4000, 3)
    if kind[1] == 2:   # a weight of 4 bits: 8 bits of scale times 5
        y = P.planes(y, 1)[0] * (1 + np.arange(4000) % 15)
        assert np.array_equal(sum(P.planes(y, 2)), y)
    off = lambda **kw: (np.abs(P.product(x, y, kind, **kw) - x * y) / np.abs(x * y)).max() / U  # noqa: E731
    assert off() <= units
    assert off(missing_x=True) > 50
    if kind[1] == 3:
        assert off(missing_y=True) > 50
    # the widest bound that is made of these
    assert P.probability_bound(8000) < 30
