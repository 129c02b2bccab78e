"""The check that holds results with infinities, against planted mistakes (no GPU needed)."""
import numpy as np
import pytest
import torch

from tests import epilogue_reference as E
from tests import strict_reference as strict

WANT = np.array([[1.0, np.inf, -np.inf, 0.0, np.nan, -2.0]])


@pytest.mark.parametrize("at,value", [(0, 1.5), (1, 3.0), (1, -np.inf), (2, np.inf), (3, np.inf), (4, 0.0), (5, np.nan)])
def test_mistakes_beside_infinities_are_seen(at, value):
    got = torch.tensor(WANT, dtype=torch.float32)
    strict.check(got, WANT, 1e-6, "right")
    got[0, at] = value
    with pytest.raises(AssertionError):
        strict.check(got, WANT, 1e-6, "wrong")


def test_bounds_are_finite():
    with pytest.raises(AssertionError, match="anything"):
        strict.check(torch.zeros(1), np.zeros(1), np.inf, "any")
    h = np.array([np.inf, -np.inf, np.nan, 3e38, -3e38])
    for act in E.ACTS:
        for fast in (True, False):
            e = E.act_err(h, act, fast)
            assert np.isfinite(e[np.isfinite(E.act(h, act))]).all(), (act, fast)
