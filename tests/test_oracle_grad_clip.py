"""The clip factor of the oracle where the norm or the limit is infinite."""
import numpy as np
import pytest

from oracle import gradients as og

INF, NAN = np.inf, np.nan


@pytest.mark.parametrize("value", [1.0, INF, -INF, NAN])
def test_an_infinite_limit_is_the_norm_alone(value):
    x = np.array([0.5, value, -2.0])
    n, (y,) = og.clip([x], INF)
    assert np.array_equal(y, x, equal_nan=True)
    assert np.isnan(n) == np.isnan(value) and (np.isnan(value) or n == np.sqrt(4.25 + value * value))


def test_finite_limits():
    x = np.array([0.5, INF, -2.0])
    assert np.array_equal(og.clip([x], 3.0)[1][0], [0.0, NAN, -0.0], equal_nan=True)
    assert np.isnan(og.clip([np.array([1.0, NAN])], 3.0)[1][0]).all()
