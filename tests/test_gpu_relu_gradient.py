"""relu's backward step selects: where h <= 0 the gradient is exactly 0, whatever comes
in, so infinities and NaN at inactive units reach neither gb, the FP8 scale nor a product."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import epilogue_reference as E
from tests import mx_reference as R
from tests.test_gpu_epilogue import rand, rng_words

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(M, N, dtype, seed):
    """(gy with an infinity or NaN at a third of the inactive units, the same with 0
    there, h, which holds zeros of both signs and infinities)."""
    gy, h = rand((M, N), dtype, seed, 0.1), rand((M, N), dtype, seed + 1, 2.0)
    h[::3, ::5], h[1::3, ::5], h[::4, 1::6], h[1::4, 1::6] = 0.0, -0.0, -np.inf, np.inf
    clean = torch.where(h <= 0, torch.zeros_like(gy), gy)
    at = torch.arange(M * N, device=DEV).view(M, N)
    for k, v in enumerate((np.inf, -np.inf, np.nan)):
        gy = torch.where((h <= 0) & (at % 9 == k), torch.full_like(gy, v), gy)
    assert not torch.isfinite(gy).all()
    return gy, clean, h


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", [(3, 7), (64, 256), (257, 1031), (2048, 2056)])
def test_the_step(M, N, dtype, p):
    gy, clean, h = case(M, N, dtype, M)
    rng, part = rng_words(1), torch.empty(F.epilogue_workspace_len(M, N), device=DEV)
    gh, gb, gh2, gb2 = torch.empty_like(gy), torch.empty(N, device=DEV), torch.empty_like(gy), torch.empty(N, device=DEV)
    kw = {"pre": h, "act": F.ACT_RELU, "p": p, "rng": rng, "part": part}
    F.epilogue_bwd(gy, gh, gb, **kw)
    F.epilogue_bwd(clean, gh2, gb2, **kw)
    assert torch.isfinite(gh).all() and torch.equal(gh, gh2) and torch.equal(gb, gb2)
    assert (gh[h <= 0] == 0).all() and not torch.signbit(gh[h <= 0]).any()
    want, err, _, _ = E.backward(R.f64(clean), R.f64(h), E.RELU, E.keep(rng.tolist(), M, N, p), dtype != "f32")
    R.check(gh, want, err, "gh")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(65, 130, 40), (600, 520, 72)])
def test_mx_backward(M, N, K, dtype):
    gy, clean, h = case(M, N, dtype, 5)
    ws, saved = F.Mxfp4LinearWs(M, N, K), F.Mxfp4LinearSaved(M, N, K)
    F.mxfp4_linear_fwd(rand((M, K), dtype, 1), rand((N, K), dtype, 2), ws, saved, torch.empty_like(gy))
    part, got = torch.empty(F.epilogue_workspace_len(M, N), device=DEV), []
    for g in (gy, clean):
        out = [torch.empty(s, dtype=gy.dtype, device=DEV) for s in ((M, N), (M, K), (N, K))] + [torch.empty(N, device=DEV)]
        F.mxfp4_linear_bwd_epilogue(g, ws, saved, out[1], out[2], gh=out[0], gb=out[3], pre=h, act=F.ACT_RELU, part=part)
        got.append(out)
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(64, 256, 128), (336, 528, 144)])  # one launch; launches of their own
def test_fp8_backward(M, N, K, dtype):
    gy, clean, h = case(M, N, dtype, 7)
    saved, ws = F.LinearSaved(M, N, K, transposed=False), F.LinearBwdWs(M, N, transposed=False)
    F.fp8_scaled_linear_fwd_epilogue(rand((M, K), dtype, 1), rand((N, K), dtype, 2, 0.05), saved, torch.empty_like(gy))
    part, got = torch.empty(F.epilogue_workspace_len(M, N), device=DEV), []
    for g in (gy, clean):
        out = [torch.empty(s, dtype=gy.dtype, device=DEV) for s in ((M, N), (M, K), (N, K))] + [torch.empty(N, device=DEV)]
        F.fp8_scaled_linear_bwd_epilogue(g, saved, ws, out[1], out[2], gh=out[0], gb=out[3], pre=h, act=F.ACT_RELU,
                                         part=part)
        got.append(out + [ws.gy_q.clone()])
        assert np.isfinite(ws.gy_sc.read()["inv"])
    for a, b in zip(*got):
        assert torch.equal(a, b) and (a.dtype == torch.uint8 or torch.isfinite(a).all())
