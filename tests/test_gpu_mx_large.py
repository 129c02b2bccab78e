"""Tensors past 2^31 elements, wide rows past the register kernels, and calls
captured before they ever ran: the last rows against the definition."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def fill(rows, cols, dtype, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.empty(rows, cols, dtype=dtype, device=DEV)
    for r in range(0, rows, 1 << 14):  # (pieces: randn's fp32 copy stays small)
        x[r:r + (1 << 14)].normal_(generator=g)
    return x


def test_quantize_and_dequantize():
    rows, cols = 70001, 32768
    x = fill(rows, cols, torch.bfloat16, 1)
    q, qT = F.Mxfp4(rows, cols), F.Mxfp4(cols, rows)
    F.mxfp4_quantize(x, q, qT)
    y = torch.empty_like(x)
    F.mxfp4_dequantize(q, y)
    torch.cuda.synchronize()
    for at in (slice(0, 8), slice(rows - 40, rows)):
        assert np.array_equal(R.f64(y[at]), R.fp4_values(R.f64(x[at]), False))
    del y
    yT = torch.empty(cols, rows, dtype=torch.bfloat16, device=DEV)
    F.mxfp4_dequantize(qT, yT)
    torch.cuda.synchronize()
    for at in (slice(0, 4), slice(cols - 4, cols)):
        assert np.array_equal(R.f64(yT[at]), R.fp4_values(R.f64(x[:, at].t()), False))


@pytest.mark.parametrize("M,N,K", [(70001, 32800, 40), (20, 1 << 27, 33)])
def test_product(M, N, K):
    a, b = fill(M, K, torch.float32, 1), fill(N, K, torch.float32, 2)
    A, B = F.Mxfp4(M, K), F.Mxfp4(N, K)
    F.mxfp4_quantize(a, A)
    F.mxfp4_quantize(b, B)
    C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    F.mxfp4_gemm(A, B, C)
    torch.cuda.synchronize()
    for rows in (slice(0, 20), slice(M - 20, M)):
        for cols in (slice(0, 300), slice(N - 300, N)):
            want, bound = R.dot(R.fp4_values(R.f64(a[rows]), False), R.fp4_values(R.f64(b[cols]), False))
            R.check(C[rows, cols], want, bound, f"{rows} {cols}")


def test_empty_contraction_of_many_outputs():
    """2^34 outputs, all zero."""
    M, N = 1 << 28, 64
    C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    C[:100], C[-100:] = 7, 7
    F.mxfp4_gemm(F.Mxfp4(M, 0), F.Mxfp4(N, 0), C)
    torch.cuda.synchronize()
    for r in range(0, M, 1 << 25):
        assert not bool(C[r:r + (1 << 25)].any())


def test_swiglu():
    rows, cols = 70001, 32768
    g, u = fill(rows, cols, torch.bfloat16, 1), fill(rows, cols, torch.bfloat16, 2)
    a, cg, cu = torch.empty_like(g), F.Act8(rows, cols), F.Act8(rows, cols)
    F.swiglu_fwd(g, u, a, cg, cu)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    F.swiglu_bwd(a, cg, cu, dg, du)
    torch.cuda.synchronize()
    at = slice(rows - 5, rows)
    vg, vu = R.f64(g[at]), R.f64(u[at])
    R.check(a[at], *R.swiglu(vg, vu), "a")
    (wg, bg), (wu, bu) = R.swiglu_grad(R.f64(a[at]), R.act8_values(vg), R.act8_values(vu))
    R.check(dg[at], wg, bg, "dg")
    R.check(du[at], wu, bu, "du")


@pytest.mark.parametrize("rows,cols,ckpt", [(2200000, 1024, True), (130000, 16640, False)])
def test_layer_norm(rows, cols, ckpt):
    x, dy = fill(rows, cols, torch.bfloat16, 1), fill(rows, cols, torch.bfloat16, 2)
    w = torch.ones(cols, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    c = F.Act8(rows, cols) if ckpt else None
    ws = torch.empty(F.layer_norm_workspace_len(rows, cols), device=DEV)
    F.layer_norm_fwd(x, w, None, 1e-5, y, mean, rstd, c)
    F.layer_norm_bwd(dy, x if c is None else c, w, mean, rstd, dx, dw, db, ws)
    torch.cuda.synchronize()
    at = slice(rows - 20, rows)
    ref = R.LayerNorm(R.f64(x[at]), None, None, 1e-5)
    R.check(y[at], ref.y, ref.y_err, "y")
    xv = R.f64(x[at])
    (want, bound), _, _ = ref.grads(R.f64(dy[at]), R.act8_values(xv) if ckpt else xv)
    R.check(dx[at], want, bound, "dx")
    total = torch.zeros(cols, dtype=torch.float64, device=DEV)
    size = torch.zeros(cols, dtype=torch.float64, device=DEV)
    for r in range(0, rows, 1 << 15):
        total += dy[r:r + (1 << 15)].double().sum(0)
        size += dy[r:r + (1 << 15)].double().abs().sum(0)
    R.check(db, R.f64(total), rows * R.U32 * R.f64(size), "db")


def test_captured_before_it_ever_ran():
    """A call's first use inside a capture: nothing in it may need a warm-up."""
    A, B = F.Mxfp4(30, 260), F.Mxfp4(8200, 260)
    a, b = fill(30, 260, torch.float16, 1), fill(8200, 260, torch.float16, 2)
    C = torch.empty(30, 8200, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.mxfp4_quantize(a, A)
        F.mxfp4_quantize(b, B)
        F.mxfp4_gemm(A, B, C)
    for i in range(3):
        a.copy_(fill(30, 260, torch.float16, 10 + i))
        C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, bound = R.dot(R.fp4_values(R.f64(a), False), R.fp4_values(R.f64(b), False))
        R.check(C, want, bound, "replay")
