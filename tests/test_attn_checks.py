"""The comparison that the GPU tests of attention use: what it has to reject, and what it accepts."""
import numpy as np
import pytest

from tests import attn_util as T

CANARY = np.full((1, 4), 9, np.float16)


def accepts(got, out, tol):
    got = np.array([got], np.float16)
    try:
        T.check_rows(got, {0: (np.array([out]), np.array([tol]))}, 1, CANARY, "case")
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("wrong", [0.0, 1.0, 65504.0, -np.inf, np.nan])
def test_an_infinity_has_to_arrive(wrong):
    """An infinite result has an infinite tolerance: no finite value, other sign or NaN passes for it."""
    want, tol = [1.0, np.inf, -np.inf, 0.5], [0.01, np.inf, np.inf, 0.01]
    assert accepts([1.0, np.inf, -np.inf, 0.5], want, tol)
    assert not accepts([1.0, wrong, -np.inf, 0.5], want, tol)
    assert not accepts([1.0, np.inf, -wrong, 0.5], want, tol)


@pytest.mark.parametrize("wrong", [0.0, np.inf, -np.inf])
def test_nan_has_to_arrive_and_to_stay_away(wrong):
    want, tol = [1.0, np.nan, 2.0, 0.5], [0.01, np.nan, 0.01, 0.01]
    assert accepts([1.0, np.nan, 2.0, 0.5], want, tol)
    assert not accepts([1.0, wrong, 2.0, 0.5], want, tol)
    assert not accepts([1.0, np.nan, np.nan, 0.5], want, tol)
    assert not accepts([1.0, np.nan, np.inf, 0.5], want, tol)


def test_finite_values_have_tolerances():
    want, tol = [1.0, 2.0, 3.0, 4.0], [0.25, 0.25, 0.0, 0.25]
    assert accepts([1.25, 1.75, 3.0, 4.0], want, tol)
    assert not accepts([1.25, 1.7, 3.0, 4.0], want, tol)
    assert not accepts([1.0, 2.0, 3.01, 4.0], want, tol)


def test_a_finite_value_without_a_tolerance_has_to_be_met():
    """No tolerance that is infinite or NaN lets a finite result through unseen."""
    want, tol = [1.0, 2.0, 3.0, 4.0], [np.inf, np.nan, 0.0, 0.0]
    assert accepts(want, want, tol)
    assert not accepts([1.5, 2.0, 3.0, 4.0], want, tol) and not accepts([1.0, 2.5, 3.0, 4.0], want, tol)


def test_rows_of_none_keep_what_they_held():
    T.check_rows(CANARY, {}, 1, CANARY, "case")
    with pytest.raises(AssertionError):
        T.check_rows(CANARY + 1, {}, 1, CANARY, "case")
