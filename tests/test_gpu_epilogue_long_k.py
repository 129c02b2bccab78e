"""The products with an epilogue past K = 2^24, whose kernel has offsets of 64 bits: sparse
operands whose products are small whole numbers of sixteenths, so that every sum is exact
and a wrong offset, column, mask or row shows."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import epilogue_reference as E
from tests import mx_reference as R
from tests.test_gpu_epilogue import GUARD, tensors, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
K = (1 << 24) + 300
AT = [0, 1, 255, 256, 5000, 1 << 23, (1 << 24) - 1, 1 << 24, (1 << 24) + 257, K - 1]
VALUES = np.array([1, .5, 3, 1, 2, 1.5, 1, 4, 2, 6])
M, N = 19, 29  # two blocks of rows; the last four columns start at 4 mod 8 and are one


def operand(rows, skip, period):
    """(codes, values at AT): rows differ in sign, scale and in which positions are 0."""
    r, j = np.arange(rows)[:, None], np.arange(len(AT))[None]
    v = VALUES * np.where((r + j) % 2, -1.0, 1.0) * 2.0 ** (r % 3 - 1) * ((r + skip * j) % period != 0)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[:, AT] = torch.tensor(v, dtype=torch.bfloat16, device=DEV)
    q = F.Mxfp4(rows, K)
    F.mxfp4_quantize(x, q)
    return q, v


@pytest.fixture(scope="module")
def operands():
    (a, x), (b, w) = operand(M, 1, 3), operand(N, 2, 5)
    prod = x @ w.T
    assert (prod * 16 == np.round(prod * 16)).all() and (prod[:, :, None] != 0).sum() > M * N // 2
    tail = x[:, 7:] @ w[:, 7:].T  # what lies past 2^24 matters
    assert (tail != 0).sum() > M * N // 2
    return a, b, prod


def test_products_of_the_codes(operands):
    a, b, prod = operands
    y = torch.empty(M, N, device=DEV)
    F.mxfp4_gemm_epilogue(a, b, y)
    assert np.array_equal(R.f64(y), prod)


@pytest.mark.parametrize("act", E.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_every_part_of_the_epilogue(operands, dtype, act):
    a, b, prod = operands
    for p, bias in ((0.0, dtype), (0.25, "f32")):
        kw, ref = tensors(M, N, dtype, bias, True, p, act)
        wide = torch.full((M + 2, N + 6), GUARD, dtype=R.DTYPES[dtype], device=DEV)
        y, pre = wide[1:M + 1, 3:N + 3], torch.full((M, N), GUARD, dtype=wide.dtype, device=DEV)
        F.mxfp4_gemm_epilogue(a, b, y, act=act, pre=pre, **kw)
        verify(y.contiguous(), pre, prod, 0.0 * prod, act, ref, dtype != "f32", (dtype, act, p))
        first = y.clone()
        y.copy_(kw["residual"])
        F.mxfp4_gemm_epilogue(a, b, y, act=act, **{**kw, "residual": y})
        assert torch.equal(y, first)
        y.fill_(GUARD)
        assert (wide == GUARD).all()
