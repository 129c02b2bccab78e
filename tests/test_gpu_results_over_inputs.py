"""Results that lie over an input of their call, in the sizes whose casts otherwise
share the product's launch: what a call with buffers of its own gives, bit for bit.
Several workgroups each, so one that stored early would show in another's input."""
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R
from tests.test_gpu_epilogue import rand, rng_words

pytestmark = pytest.mark.gpu
DEV = "cuda"
S = 256  # x, W and y of S x S: the largest layer of one launch


def over(t, dtype, at=0):
    """A new S x S tensor of dtype that starts `at` bytes from the start of a copy of t:
    (the copy of t, the tensor)."""
    size = torch.empty((), dtype=dtype).element_size()
    raw = torch.zeros(max(t.nbytes, at + S * S * size), dtype=torch.uint8, device=DEV)
    copy = raw[:t.nbytes].view(t.dtype).view(t.shape)
    copy.copy_(t)
    return copy, raw[at:at + S * S * size].view(dtype).view(S, S)


# (result's type, its place in bytes behind the input's start)
PLACES = [("same", 0), ("same", 16), ("same", S * S), ("f32", 0)]


def kind(t, name):
    return torch.float32 if name == "f32" else t.dtype


@pytest.mark.parametrize("out,at", PLACES)
@pytest.mark.parametrize("which", ["x", "w"])
def test_fp8_forward(which, out, at):
    x, w = rand((S, S), "bf16", 1), rand((S, S), "bf16", 2, 0.05)
    y = torch.empty(S, S, dtype=kind(x, out), device=DEV)
    saved, saved2 = (F.LinearSaved(S, S, S, transposed=False) for _ in range(2))
    o = F.OUT_F32 if out == "f32" else F.OUT_BF16
    F.fp8_scaled_linear_fwd(x, w, saved, y, o)
    t, y2 = over(x if which == "x" else w, y.dtype, at)
    F.fp8_scaled_linear_fwd(t if which == "x" else x, t if which == "w" else w, saved2, y2, o)
    assert torch.equal(y, y2)
    assert torch.equal(saved.x_q, saved2.x_q) and torch.equal(saved.w_q, saved2.w_q)


@pytest.mark.parametrize("out,at", PLACES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("which", ["x", "w"])
def test_fp8_forward_with_an_epilogue(which, dtype, out, at):
    x, w = rand((S, S), dtype, 1), rand((S, S), dtype, 2, 0.05)
    y = torch.empty(S, S, dtype=kind(x, out), device=DEV)
    pre = torch.empty_like(y)
    saved, saved2 = (F.LinearSaved(S, S, S, transposed=False) for _ in range(2))
    kw = {"bias": rand((S,), "f32", 3), "act": F.ACT_RELU, "p": 0.25, "rng": rng_words(4)}
    F.fp8_scaled_linear_fwd_epilogue(x, w, saved, y, pre=pre, **kw)
    for result in ("y", "pre"):
        t, r = over(x if which == "x" else w, y.dtype, at)
        o = torch.empty_like(y)
        F.fp8_scaled_linear_fwd_epilogue(t if which == "x" else x, t if which == "w" else w, saved2,
                                         r if result == "y" else o, pre=r if result == "pre" else o, **kw)
        got = (r, o) if result == "y" else (o, r)
        assert torch.equal(got[0], y) and torch.equal(got[1], pre), result
        assert torch.equal(saved.x_q, saved2.x_q) and torch.equal(saved.w_q, saved2.w_q)
    if out == "same" and at == 0 and which == "x":  # a residual stream updated in place
        F.fp8_scaled_linear_fwd_epilogue(x, w, saved, y, residual=x, **kw)
        F.fp8_scaled_linear_fwd_epilogue(x, w, saved2, x, residual=x, **kw)
        assert torch.equal(x, y) and torch.equal(saved.x_q, saved2.x_q)


@pytest.mark.parametrize("out,at", PLACES)
@pytest.mark.parametrize("which", ["gx", "gw"])
@pytest.mark.parametrize("call", ["plain", "unscale"])
def test_fp8_backward(call, which, out, at):
    if call == "unscale" and out == "f32":
        pytest.skip("fp16 gradients only")
    x, w, gy = rand((S, S), "bf16", 1), rand((S, S), "bf16", 2, 0.05), rand((S, S), "bf16", 3, 1e-3)
    saved = F.LinearSaved(S, S, S, transposed=False)
    F.fp8_scaled_linear_fwd(x, w, saved, torch.empty_like(x), F.OUT_BF16)
    ws, ws2 = (F.LinearBwdWs(S, S, transposed=False) for _ in range(2))
    t = torch.float16 if call == "unscale" else kind(x, out)
    scale, found = torch.full((1,), 8.0, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(g, v, gx, gw):
        if call == "unscale":
            F.fp8_scaled_linear_bwd_unscale(g, saved, v, scale, found, gx, gw)
        else:
            F.fp8_scaled_linear_bwd(g, saved, v, gx, gw, F.OUT_F32 if out == "f32" else F.OUT_BF16)
    want = [torch.empty(S, S, dtype=t, device=DEV) for _ in range(2)]
    run(gy, ws, *want)
    g, r = over(gy, t, at)
    o = torch.empty(S, S, dtype=t, device=DEV)
    got = (r, o) if which == "gx" else (o, r)
    run(g, ws2, *got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(ws.gy_q, ws2.gy_q)


@pytest.mark.parametrize("M", [1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [512, 8192])  # 16 and 32 columns a workgroup
def test_mx_apply(M, N, dtype):
    """A quantised x and the product of the codes give the same bits as the call whose
    result lies over x; its sums in another order than the call that fuses the two."""
    K = N if N == 512 else 256
    w = F.Mxfp4(N, K)
    F.mxfp4_quantize(rand((N, K), dtype, 2, 0.05), w)
    bias = rand((N,), "f32", 3)
    raw = torch.zeros(M * max(N, K), dtype=R.DTYPES[dtype], device=DEV)
    x, y = raw[:M * K].view(M, K), raw[:M * N].view(M, N)
    x0, a, ws = rand((M, K), dtype, 1), F.Mxfp4(M, K), F.Mxfp4(M, K)
    F.mxfp4_quantize(x0, a)
    want, pre = torch.empty(M, N, dtype=x0.dtype, device=DEV), torch.empty(M, N, dtype=x0.dtype, device=DEV)
    F.mxfp4_gemm(a, w, want)
    x.copy_(x0)
    F.mxfp4_linear_apply(x, w, y, ws)
    assert torch.equal(y, want)
    F.mxfp4_gemm_epilogue(a, w, want, bias=bias, act=F.ACT_GELU, pre=pre)
    o = torch.empty_like(want)
    for result in ("y", "pre"):
        x.copy_(x0)
        F.mxfp4_linear_apply_epilogue(x, w, y if result == "y" else o, ws, bias=bias, act=F.ACT_GELU,
                                      pre=y if result == "pre" else o)
        got = (y, o) if result == "y" else (o, y)
        assert torch.equal(got[0], want) and torch.equal(got[1], pre), result
    if N == K:
        F.mxfp4_gemm_epilogue(a, w, want, bias=bias, residual=x0)
        x.copy_(x0)
        F.mxfp4_linear_apply_epilogue(x, w, x, ws, bias=bias, residual=x)
        assert torch.equal(x, want)
