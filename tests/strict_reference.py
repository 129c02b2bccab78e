"""mx_reference.check for results that hold infinities: its largest excess is NaN where
one is wanted, and a NaN exceeds nothing, so it passes such results unseen."""
import numpy as np
import torch

from tests import mx_reference as R


def check(got, want, bound, what):
    """R.check, with wanted infinities equal in place and sign."""
    inf = np.isinf(want)
    g = R.f64(got).reshape(want.shape)
    assert np.array_equal(g[inf], want[inf]), f"{what}: infinities {g[inf]}, expected {want[inf]}"
    bound = np.where(inf, 0.0, np.broadcast_to(np.asarray(bound, dtype=np.float64), want.shape))
    assert np.isfinite(bound).all(), f"{what}: a bound that allows anything"
    at = torch.from_numpy(inf.copy()).to(got.device)
    R.check(got.reshape(want.shape).masked_fill(at, 0.0), np.where(inf, 0.0, want), bound, what)
