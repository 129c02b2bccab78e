"""Layer norm where its statistics are delicate: rows of one value, means far
from zero."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5
# one, four, eight and sixteen waves a row, one and two groups a lane, rows past the registers
COLS = [7, 100, 511, 700, 1000, 1500, 4001, 8100, 14333, 14336, 16640, 40001]


def forward(x, w=None, b=None, ckpt=None):
    rows, cols = x.shape
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    F.layer_norm_fwd(x, w, b, EPS, y, mean, rstd, ckpt)
    return y, mean, rstd


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_rows_of_one_value(cols, dtype):
    """Their variance is 0 and their deviations are 0, so the result is b, the
    mean that value and dx what is left of dy w without its mean.  The fp32 sum
    of the row may round (1000.1 times 14333), its mean may not."""
    t = R.DTYPES[dtype]
    values = torch.tensor([1000.0, 1000.1, -0.1, 3.0e4 / 7, 1 / 3, 2.0 ** -20, 0.0, 5.0]).to(t)
    x = values[:, None].expand(-1, cols).contiguous().to(DEV)
    w = torch.linspace(-2, 2, cols, device=DEV).to(t)
    b = torch.linspace(3, 5, cols, device=DEV).to(t)
    y, mean, rstd = forward(x, w, b, F.Act8(*x.shape))
    dx = torch.empty_like(x)
    F.layer_norm_bwd(torch.ones_like(x), x, None, mean, rstd, dx=dx)
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand_as(y))
    assert torch.equal(mean.cpu(), values.float())
    # dy = 1, w = 1: 1 - mean(1), with xh = 0
    assert not bool(dx.any())


@pytest.mark.parametrize("cols", COLS)
def test_a_mean_far_from_zero(cols):
    """Deviations of 1 around 5000, each within a few steps of its own size, not of
    the mean's (2^-11).  x and the first mean are multiples of 2^-11, so the
    deviations from it are exact, and below 8: the sum's error shifts them by
    depth U32 5000 < 0.1.  With depth = n / 64 + 24 additions in a chain, the mean's
    correction is then off by (depth + 2) U32 8, the variance by (depth + 4) U32
    (1 + 0.1^2) of itself and by 2 * 0.1 times the correction's error, so rstd by less
    than (2 depth + 8) U32 of itself; the result takes four more roundings."""
    g = torch.Generator().manual_seed(cols)
    # multiples of 2^-11 around 5000 are exact, and so are their deviations from any fp32 mean near them
    x = 5000 + (torch.randn(20, cols, generator=g) * 2048).round() / 2048
    x = x.to(DEV)
    y, mean, rstd = forward(x)
    torch.cuda.synchronize()
    v = R.f64(x)
    m = v.mean(axis=1, keepdims=True)
    c = v - m
    var = (c * c).mean(axis=1, keepdims=True)
    want = c / np.sqrt(var + EPS)
    depth = cols / 64 + 24
    mean_err = (depth + 2) * R.U32 * 8.0  # of the corrected mean, before it is rounded for the backward
    rel = (2 * depth + 8) * R.U32
    bound = (mean_err + np.abs(c) * rel) / np.sqrt(var + EPS) + 4 * R.U32 * np.abs(want)
    R.check(y, want, bound, "y")
    R.check(mean, m[:, 0], mean_err, "mean")
    R.check(rstd, 1 / np.sqrt(var + EPS)[:, 0], rel / np.sqrt(var + EPS)[:, 0], "rstd")
