"""fp32 results of the FP8 products with an epilogue: activations in fp32's own accuracy,
in every tiling, and 16-bit results as before."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import epilogue_reference as E
from tests import mx_reference as R
from tests import strict_reference as strict
from tests.test_gpu_epilogue import fp8_product, points, rand, tensors, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
# tiles of 64, 128, 256 and 224; contractions that end inside a k-tile and that do not
FORMS = [(336, 528, 144), (2048, 2304, 144), (2880, 3104, 144), (2880, 3104, 128), (3584, 4096, 128), (3584, 4096, 144)]


def some_points(n, seed):
    """n of the fp32 points, every special value among them."""
    v = points("f32")
    at = torch.from_numpy(np.random.default_rng(seed).permutation(v.numel() - 5)[:n - 5]).to(DEV)
    return torch.cat([v[at], v[-5:]])


def check_act(y, bias, act, what):
    """Every row of y is act(bias), within the kernel's own bound for fp32."""
    assert torch.equal(y.view(torch.int32), y[:1].expand_as(y).contiguous().view(torch.int32)), what
    h = R.f64(bias)[None]
    strict.check(y[:1], E.act(h, act), E.act_err(h, act, False), what)


@pytest.mark.parametrize("act", [a for a in E.ACTS if a != E.NONE])
@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("rowwise", [False, True])
def test_products_of_zeros_leave_the_activation(M, N, K, act, rowwise):
    a, b = torch.zeros(M, K, dtype=torch.uint8, device=DEV), torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV)
    ia, ib = torch.ones(M, dtype=torch.float64, device=DEV), torch.ones(N, dtype=torch.float64, device=DEV)
    bias, y = some_points(N, act), torch.empty(M, N, device=DEV)
    if rowwise:
        F.fp8_gemm_rowwise_epilogue(a, b, ia, ib, y, bias=bias, act=act)
    else:
        F.fp8_gemm_epilogue(a, b, ia.data_ptr(), ib.data_ptr(), y, bias=bias, act=act)
    check_act(y, bias, act, (M, N, K, act, rowwise))


@pytest.mark.parametrize("act", [a for a in E.ACTS if a != E.NONE])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(64, 256, 128), (336, 528, 144)])
def test_layers_with_an_fp32_result(M, N, K, dtype, act):
    """(64 x 256 x 128: casts and product in one launch.)"""
    w, saved = rand((N, K), dtype, 2, 0.05), F.LinearSaved(M, N, K, transposed=False)
    y = torch.empty(M, N, device=DEV)
    for seed in range(8):
        bias = some_points(N, seed)
        F.fp8_scaled_linear_fwd_epilogue(torch.zeros(M, K, dtype=w.dtype, device=DEV), w, saved, y, bias=bias, act=act)
        check_act(y, bias, act, (M, N, K, dtype, act, seed))
    x, pre = rand((M, K), dtype, 1), torch.empty_like(y)
    kw, ref = tensors(M, N, "f32", "f32", True, 0.25, act)
    F.fp8_scaled_linear_fwd_epilogue(x, w, saved, y, act=act, pre=pre, **kw)
    verify(y, pre, *fp8_product(saved), act, ref, False, (M, N, K, dtype, act))
