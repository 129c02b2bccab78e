"""Every activation of every value, infinities included (the check that
test_gpu_epilogue's test of the same values uses passes whatever stands beside one)."""
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import epilogue_reference as E
from tests import mx_reference as R
from tests import strict_reference as strict
from tests.test_gpu_epilogue import points

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", E.ACTS)
@pytest.mark.parametrize("rows", [1, 700])  # one row; tiles of 64
def test_activation_of_every_value(act, dtype, rows):
    """An empty contraction leaves act(bias)."""
    b = points(dtype)
    b = b if rows == 1 else b[-20000:].contiguous()
    y = torch.empty(rows, b.numel(), dtype=b.dtype, device=DEV)
    F.mxfp4_gemm_epilogue(F.Mxfp4(rows, 0), F.Mxfp4(b.numel(), 0), y, bias=b, act=act)
    bits = y.view(torch.int16 if y.element_size() == 2 else torch.int32)
    assert (bits == bits[:1]).all()
    h = R.f64(b)[None]
    strict.check(y[:1], E.act(h, act), E.act_err(h, act, dtype != "f32"), (act, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", E.ACTS)
def test_fp8_activation_of_every_value(act, dtype):
    b = points(dtype)
    y = torch.empty(16, b.numel(), dtype=b.dtype, device=DEV)
    inv = torch.ones(1, dtype=torch.float64, device=DEV)
    e = torch.empty(16, 0, dtype=torch.uint8, device=DEV), torch.empty(b.numel(), 0, dtype=torch.uint8, device=DEV)
    F.fp8_gemm_epilogue(*e, inv.data_ptr(), inv.data_ptr(), y, bias=b, act=act)
    assert (y.view(torch.int16) == y[:1].view(torch.int16)).all()
    h = R.f64(b)[None]
    strict.check(y[:1], E.act(h, act), E.act_err(h, act, True), (act, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", E.ACTS)
def test_both_passes_at_infinities_and_nan(act, dtype):
    """At an infinity every slope has its limit; a NaN stays one, but under relu, whose
    slope there is 1 (it is not below 0)."""
    h = torch.tensor([[float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 1.0]], dtype=R.DTYPES[dtype], device=DEV)
    gh = torch.empty_like(h)
    F.epilogue_bwd(torch.full_like(h, 2.0), gh, pre=h, act=act)
    want = {E.NONE: [2, 2, 2, 2, 2, 2], E.RELU: [2, 0, 2, 0, 0, 2]}.get(act, [2, 0, float("nan"), 1, 1, None])
    for got, w in zip(gh[0].tolist(), want):
        assert w is None or got == w or (w != w and got != got), (act, gh, want)
