"""MXFP4 quantisation, products and linears against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
RULES = [F.MX_FLOOR, F.MX_FIT]


def rand(shape, dtype, seed, sigma=1.0, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * sigma
    if spread:
        x = x * torch.exp2(torch.randint(-spread, spread + 1, shape, generator=g).float())
    return x.to(R.DTYPES[dtype]).to(DEV)


def assert_same(m, x, fit):
    codes, s = R.fp4(R.f64(x), fit)
    got, gs = R.fp4_unpack(m)
    nb = codes.shape[1]
    assert np.array_equal(gs[:, :nb], s)
    assert np.array_equal(got[:, :nb], codes)
    assert (got[:, nb:] == 0).all() and (gs[:, nb:] == 127).all()  # past the last block


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (5, 33), (16, 256), (128, 256), (129, 257),
                                       (256, 128), (257, 512), (300, 1000), (64, 4096), (1000, 40), (513, 776)])
def test_codes_both_directions(rows, cols, rule, dtype):
    x = rand((rows, cols), dtype, rows * 1000 + cols, spread=3)
    q, qT = F.Mxfp4(rows, cols), F.Mxfp4(cols, rows)
    for m in (q, qT):
        m.q.fill_(0xA5)
        m.s.fill_(0xA5)
    F.mxfp4_quantize(x, q, qT, rule=rule)
    torch.cuda.synchronize()
    assert_same(q, x, rule == F.MX_FIT)
    assert_same(qT, x.t(), rule == F.MX_FIT)
    one, oneT = F.Mxfp4(rows, cols), F.Mxfp4(cols, rows)
    F.mxfp4_quantize(x, one, rule=rule)
    F.mxfp4_quantize(x, qT=oneT, rule=rule)
    torch.cuda.synchronize()
    assert_same(one, x, rule == F.MX_FIT)
    assert_same(oneT, x.t(), rule == F.MX_FIT)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rule", RULES)
def test_every_16_bit_value_and_every_rounding(rule, dtype):
    """Each value next to a block maximum that puts it anywhere in the block's range."""
    if dtype == "f32":
        bits = torch.arange(0, 1 << 32, 65537, dtype=torch.int64)
        v = (bits - (bits >= 1 << 31).long() * (1 << 32)).int().view(torch.float32)
        v = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    else:
        v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(R.DTYPES[dtype])
    v = v[:v.numel() // 256 * 256].reshape(-1, 256)
    blocks = v.view(-1, 8, 32).clone()
    scale = torch.exp2(torch.arange(8).float())
    top = blocks.float().abs().amax(dim=-1)
    top = torch.where(torch.isfinite(top), top * scale * 1.4, top)
    fits = top <= torch.finfo(v.dtype).max
    blocks[..., 7] = torch.where(fits, top, top / (scale * 1.4)).to(v.dtype)
    x = blocks.view(-1, 256).to(DEV)
    m, mT = F.Mxfp4(*x.shape), F.Mxfp4(*x.shape[::-1])
    F.mxfp4_quantize(x, m, mT, rule=rule)
    torch.cuda.synchronize()
    assert_same(m, x, rule == F.MX_FIT)
    assert_same(mT, x.t(), rule == F.MX_FIT)


@pytest.mark.parametrize("rule", RULES)
def test_ties_and_extremes(rule):
    big = torch.finfo(torch.float32).max
    rows = [[6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6],
            [7.99, 6.0001, 4.0], [8, 6, 1], [0.0], [-0.0, 0.0], [big, -big], [2.0 ** -149], [2.0 ** -126, 2.0 ** -130],
            [2.0 ** -124, 1.75 * 2.0 ** -125], [float("inf"), 1], [float("nan"), 1], [float("-inf"), 5], [1, 2, 3]]
    x = torch.zeros(len(rows), 64)
    for i, r in enumerate(rows):
        x[i, 3:3 + len(r)] = torch.tensor(r)
        x[i, 40] = 1.0  # the second block stays finite
    x = x.to(DEV)
    m, mT = F.Mxfp4(*x.shape), F.Mxfp4(x.shape[1], x.shape[0])
    F.mxfp4_quantize(x, m, mT, rule=rule)
    y = torch.empty_like(x)
    F.mxfp4_dequantize(m, y)
    torch.cuda.synchronize()
    assert_same(m, x, rule == F.MX_FIT)
    assert_same(mT, x.t(), rule == F.MX_FIT)
    want = R.fp4_values(R.f64(x), rule == F.MX_FIT)
    assert np.array_equal(R.f64(y), want, equal_nan=True)
    assert np.isfinite(want[:9]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (7, 33), (130, 255), (64, 512), (33, 1001)])
def test_dequantize(rows, k, dtype):
    x = rand((rows, k), "f32", 5)
    m = F.Mxfp4(rows, k)
    F.mxfp4_quantize(x, m)
    y = torch.empty((rows, k), dtype=R.DTYPES[dtype], device=DEV)
    F.mxfp4_dequantize(m, y)
    torch.cuda.synchronize()
    want = torch.from_numpy(R.fp4_values(R.f64(x), False)).to(y.dtype)  # one rounding
    assert torch.equal(y.cpu(), want)


def product(M, N, K, out, seed, spread=0):
    a, b = rand((M, K), "f32", seed, spread=spread), rand((N, K), "f32", seed + 1, 0.02)
    A, B = F.Mxfp4(M, K), F.Mxfp4(N, K)
    for m in (A, B):
        m.s.fill_(255)  # scales past the last row are not the product's business
    F.mxfp4_quantize(a, A)
    F.mxfp4_quantize(b, B)
    guard = torch.full((M * N + 64,), 7.0, dtype=R.DTYPES[out], device=DEV)
    C = guard[:M * N].view(M, N)
    F.mxfp4_gemm(A, B, C)
    torch.cuda.synchronize()
    assert (guard[M * N:] == 7).all()
    want, bound = R.dot(R.fp4_values(R.f64(a), False), R.fp4_values(R.f64(b), False))
    R.check(C, want, bound, f"{M}x{N}x{K} {out}")
    return A, B, C


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 7, 33), (3, 5, 256), (16, 16, 128), (17, 33, 300), (1, 1000, 512),
                                   (48, 100, 1000), (64, 256, 128), (65, 64, 64), (128, 128, 2048), (130, 127, 513),
                                   (300, 500, 700), (1000, 24, 640), (256, 1024, 1500)])
def test_product(M, N, K, out):
    product(M, N, K, out, M + N + K, spread=2)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(4096, 2048, 512), (4000, 2100, 1000), (2049, 4097, 300), (14336, 512, 256)])
def test_large_product(M, N, K, out):
    product(M, N, K, out, M + N + K)


@pytest.mark.parametrize("M,N,K", [(200, 300, 3000), (1000, 40, 700), (500, 64, 260), (2500, 1500, 600), (1500, 1400, 130),
                                   (70, 14336, 256), (40, 14000, 512), (20, 9000, 300), (15, 20, 20000)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_product_of_every_shape_of_tile(M, N, K, out):
    product(M, N, K, out, M + N + K, spread=2)


def test_a_contraction_past_the_tiled_kernels_offsets():
    """K above 2^24: sparse operands, so that the sum is known."""
    M, N, K = 2, 3, (1 << 24) + 300
    a, b = torch.zeros(M, K), torch.zeros(N, K)
    at = torch.tensor([0, 1, 255, 256, 1 << 23, (1 << 24) - 1, 1 << 24, K - 1])
    a[:, at] = torch.tensor([[1.0], [2.0]]) * torch.tensor([1.0, .5, 3, 1, 2, 1, 4, 6])
    b[:, at] = torch.tensor([[1.0], [-1.0], [3.0]])
    A, B, C = F.Mxfp4(M, K), F.Mxfp4(N, K), torch.empty(M, N, device=DEV)
    F.mxfp4_quantize(a.to(DEV), A)
    F.mxfp4_quantize(b.to(DEV), B)
    F.mxfp4_gemm(A, B, C)
    torch.cuda.synchronize()
    assert torch.equal(C.cpu(), torch.tensor([[18.5], [37.0]]) * torch.tensor([1.0, -1.0, 3.0]))


@pytest.mark.parametrize("M,N", [(1, 5), (40, 300), (200, 200)])
def test_empty_contraction_gives_zeros(M, N):
    A, B = F.Mxfp4(M, 0), F.Mxfp4(N, 0)
    C = torch.full((M, N), 3.0, device=DEV)
    F.mxfp4_gemm(A, B, C)
    torch.cuda.synchronize()
    assert (C == 0).all()


def test_empty_outputs():
    F.mxfp4_gemm(F.Mxfp4(0, 64), F.Mxfp4(5, 64), torch.empty(0, 5, device=DEV))
    F.mxfp4_quantize(torch.empty(0, 40, device=DEV), F.Mxfp4(0, 40), F.Mxfp4(40, 0))
    F.mxfp4_dequantize(F.Mxfp4(3, 0), torch.empty(3, 0, device=DEV))
    torch.cuda.synchronize()


@pytest.mark.parametrize("M,N,K", [(5, 40, 300), (70, 200, 600), (2048, 4096, 512)])
def test_nan_block_reaches_its_row_only(M, N, K):
    a, b = rand((M, K), "f32", 1), rand((N, K), "f32", 2)
    a[M // 2, K // 2] = float("nan")
    b[N // 3, 0] = float("inf")
    A, B, C = F.Mxfp4(M, K), F.Mxfp4(N, K), torch.empty(M, N, device=DEV)
    F.mxfp4_quantize(a, A)
    F.mxfp4_quantize(b, B)
    F.mxfp4_gemm(A, B, C)
    torch.cuda.synchronize()
    bad = torch.isnan(C).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M // 2] = True
    want[:, N // 3] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 512, 4096), (1, 100, 14336), (2, 77, 999), (7, 300, 64), (16, 4096, 512),
                                   (17, 130, 2050), (33, 64, 300), (64, 1000, 1024), (100, 96, 500)])
def test_apply(M, N, K, dtype, rule):
    x, w = rand((M, K), dtype, 3, spread=2), rand((N, K), dtype, 4, 0.02)
    W, ws = F.Mxfp4(N, K), F.Mxfp4(M, K)
    F.mxfp4_quantize(w, W, rule=rule)
    y = torch.empty((M, N), dtype=x.dtype, device=DEV)
    F.mxfp4_linear_apply(x, W, y, ws, rule=rule)
    torch.cuda.synchronize()
    fit = rule == F.MX_FIT
    want, bound = R.dot(R.fp4_values(R.f64(x), fit), R.fp4_values(R.f64(w), fit))
    R.check(y, want, bound, "y")


def test_apply_with_nan_zeros_and_padded_rows():
    """A padded batch: rows of zeros give zeros, a row with an inf gives NaN."""
    M, N, K = 6, 200, 1000
    x, w = rand((M, K), "bf16", 3), rand((N, K), "bf16", 4)
    x[2:4] = 0
    x[5, 999] = float("inf")
    W, ws, y = F.Mxfp4(N, K), F.Mxfp4(M, K), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    F.mxfp4_quantize(w, W)
    F.mxfp4_linear_apply(x, W, y, ws)
    torch.cuda.synchronize()
    assert (y[2:4] == 0).all() and torch.isnan(y[5]).all() and torch.isfinite(y[:5]).all()


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (64, 256, 128), (33, 70, 301), (300, 513, 258), (2048, 4096, 256)])
def test_linear(M, N, K, dtype, rule):
    x, w, gy = rand((M, K), dtype, 1), rand((N, K), dtype, 2, 0.02), rand((M, N), dtype, 3, 0.1)
    ws, saved = F.Mxfp4LinearWs(M, N, K), F.Mxfp4LinearSaved(M, N, K)
    y, gx, gw = (torch.empty(s, dtype=x.dtype, device=DEV) for s in ((M, N), (M, K), (N, K)))
    F.mxfp4_linear_fwd(x, w, ws, saved, y, rule=rule)
    F.mxfp4_linear_bwd(gy, ws, saved, gx, gw, rule=rule)
    y2 = torch.empty_like(y)
    F.mxfp4_linear_fwd(x, w, F.Mxfp4LinearWs(M, N, K, backward=False), None, y2, rule=rule)
    torch.cuda.synchronize()
    fit = rule == F.MX_FIT

    def val(t):
        return R.fp4_values(R.f64(t), fit)
    R.check(y, *R.dot(val(x), val(w)), "y")
    R.check(gx, *R.dot(val(gy), val(w.t())), "gx")
    R.check(gw, *R.dot(val(gy.t()), val(x.t())), "gw")
    assert torch.equal(y, y2)


def test_unaligned_input_and_output():
    """Tensors that start in the middle of another one, aligned to their element only."""
    M, N, K = 40, 64, 512
    buf = rand((M * K + 1,), "bf16", 9)
    x = buf[1:].view(M, K)
    q, qT = F.Mxfp4(M, K), F.Mxfp4(K, M)
    F.mxfp4_quantize(x, q, qT)
    out = torch.zeros(M * K + 1, dtype=torch.bfloat16, device=DEV)
    F.mxfp4_dequantize(q, out[1:].view(M, K))
    w = rand((N, K), "bf16", 10)
    W = F.Mxfp4(N, K)
    F.mxfp4_quantize(w, W)
    c = torch.zeros(M * N + 1, dtype=torch.bfloat16, device=DEV)
    F.mxfp4_gemm(q, W, c[1:].view(M, N))
    torch.cuda.synchronize()
    assert_same(q, x, False)
    assert_same(qT, x.t(), False)
    assert out[0] == 0 and c[0] == 0
    want = R.fp4_values(R.f64(x), False)
    assert np.array_equal(R.f64(out[1:]).reshape(M, K), want)
    R.check(c[1:].view(M, N), *R.dot(want, R.fp4_values(R.f64(w), False)), "c")


def test_two_streams_and_a_replayed_graph():
    M, N, K = 64, 256, 512
    w = rand((N, K), "bf16", 1, 0.02)
    W = F.Mxfp4(N, K)
    F.mxfp4_quantize(w, W)
    xs = [rand((M, K), "bf16", 10 + i) for i in range(2)]
    ys = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    wss = [F.Mxfp4(M, K) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, x, y, ws in zip(streams, xs, ys, wss):
        with torch.cuda.stream(s):
            F.mxfp4_linear_apply(x, W, y, ws)
    torch.cuda.synchronize()
    want = [R.dot(R.fp4_values(R.f64(x), False), R.fp4_values(R.f64(w), False)) for x in xs]
    for y, (v, b) in zip(ys, want):
        R.check(y, v, b, "stream")
    # a captured training step, replayed on new inputs
    ws, saved = F.Mxfp4LinearWs(M, N, K), F.Mxfp4LinearSaved(M, N, K)
    x, gy = xs[0].clone(), rand((M, N), "bf16", 5, 0.1)
    y, gx, gw = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((M, N), (M, K), (N, K)))

    def step():
        F.mxfp4_linear_fwd(x, w, ws, saved, y)
        F.mxfp4_linear_bwd(gy, ws, saved, gx, gw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(rand((M, K), "bf16", 50 + i))
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (y, gx, gw)]
        for t in (y, gx, gw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (y, gx, gw)):
            assert torch.equal(a, b)
