"""MXFP4 kernels for large matrices at sizes that give them several k-tiles,
ragged edges and every type: the 256 x 256 product tiles, the 256-column cast."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R
from tests.test_gpu_mxfp4 import RULES, product, rand

pytestmark = pytest.mark.gpu
DEV = "cuda"


def full_chip(off_rows, off_cols):
    """Ragged M x N with more tiles of 256 x 256 than compute units: the large
    tiles are for products that fill the chip."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    a = int(np.ceil(np.sqrt(cus)))
    assert a * (a + 1) > cus
    return 256 * (a + 1) - off_rows, 256 * a - off_cols


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("off,K", [((100, 71), K) for K in (256, 512, 700, 1000, 1300, 1536)] +  # 1 to 6 k-tiles
                         [((0, 0), 700), ((255, 252), 700)])
def test_product_that_fills_the_chip(off, K, out):
    M, N = full_chip(*off)
    product(M, N, K, out, K)


@pytest.mark.parametrize("K", [300, 800])
def test_nan_blocks_in_large_tiles(K):
    M, N = full_chip(3, 5)
    a, b = rand((M, K), "f32", 1), rand((N, K), "f32", 2)
    a[M - 1, K - 1] = float("nan")
    a[300, 0] = float("-inf")
    b[N - 2, 17] = float("inf")
    A, B, C = F.Mxfp4(M, K), F.Mxfp4(N, K), torch.empty(M, N, device=DEV)
    F.mxfp4_quantize(a, A)
    F.mxfp4_quantize(b, B)
    F.mxfp4_gemm(A, B, C)
    torch.cuda.synchronize()
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[[300, M - 1]] = True
    want[:, N - 2] = True
    assert torch.equal(torch.isnan(C), want)


@pytest.mark.parametrize("dtype,rule", [("bf16", F.MX_FLOOR), ("f16", F.MX_FIT), ("f32", F.MX_FLOOR)])
def test_linear_that_fills_the_chip(dtype, rule):
    """All three products: K has as many tiles as N."""
    M, N = full_chip(37, 90)
    K = N + 13
    x, w, gy = rand((M, K), dtype, 1), rand((N, K), dtype, 2, 0.02), rand((M, N), dtype, 3, 0.1)
    ws, saved = F.Mxfp4LinearWs(M, N, K), F.Mxfp4LinearSaved(M, N, K)
    y, gx, gw = (torch.empty(s, dtype=x.dtype, device=DEV) for s in ((M, N), (M, K), (N, K)))
    F.mxfp4_linear_fwd(x, w, ws, saved, y, rule=rule)
    F.mxfp4_linear_bwd(gy, ws, saved, gx, gw, rule=rule)
    torch.cuda.synchronize()
    fit = rule == F.MX_FIT

    def val(t):
        return R.fp4_values(R.f64(t), fit)
    for name, got, a, b in (("y", y, val(x), val(w)), ("gx", gx, val(gy), val(w.t())), ("gw", gw, val(gy.t()), val(x.t()))):
        # a spread of rows, every tile row and both of its halves among them
        at = np.unique(np.concatenate([np.arange(0, got.shape[0], 61), np.arange(got.shape[0] - 5, got.shape[0])]))
        R.check(got[torch.from_numpy(at).to(DEV)], *R.dot(a[at], b), name)


def check_codes(m, x, fit, what):
    """The codes and scales of some rows of x: the first, ones across the tiles'
    borders, the last."""
    rows = x.shape[0]
    codes, s = R.fp4_unpack(m)
    for lo in (0, 250, rows // 2 + 3, rows - 40):
        at = slice(max(lo, 0), min(lo + 40, rows))
        want, ws = R.fp4(R.f64(x[at]), fit)
        nb = want.shape[1]
        assert np.array_equal(s[at, :nb], ws), (what, at)
        assert np.array_equal(codes[at, :nb], want), (what, at)
        assert (codes[at, nb:] == 0).all() and (s[at, nb:] == 127).all(), (what, at)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(4100, 4099), (4352, 4096), (12345, 1500)])
def test_wide_cast_both_directions(rows, cols, dtype, rule):
    """More tiles of 256 x 256 than compute units."""
    assert -(-rows // 256) * -(-cols // 256) > torch.cuda.get_device_properties(0).multi_processor_count
    x = rand((rows, cols), dtype, rows + cols, spread=3)
    q, qT = F.Mxfp4(rows, cols), F.Mxfp4(cols, rows)
    for m in (q, qT):
        m.q.fill_(0xA5)
        m.s.fill_(0xA5)
    F.mxfp4_quantize(x, q, qT, rule=rule)
    torch.cuda.synchronize()
    fit = rule == F.MX_FIT
    check_codes(q, x, fit, "rows")
    check_codes(qT, x.t(), fit, "columns")
    one = F.Mxfp4(cols, rows)
    one.q.fill_(0x5A)
    F.mxfp4_quantize(x, qT=one, rule=rule)
    torch.cuda.synchronize()
    assert torch.equal(one.q, qT.q)


@pytest.mark.parametrize("rows,cols,dtype", [(7001, 9003, "f32"), (11001, 9003, "f16"), (11001, 9003, "bf16")])
def test_streaming_cast(rows, cols, dtype):
    """Past the caches, where loads and stores are non-temporal: ragged columns."""
    g = torch.Generator(DEV).manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device=DEV).to(R.DTYPES[dtype])
    assert rows * cols * (5 if dtype == "f32" else 3) >= 256 << 20
    q, qT = F.Mxfp4(rows, cols), F.Mxfp4(cols, rows)
    F.mxfp4_quantize(x, q, qT, rule=F.MX_FIT)
    torch.cuda.synchronize()
    check_codes(q, x, True, "rows")
    check_codes(qT, x.t(), True, "columns")


def test_values_past_fp16():
    """The largest fp16 value rounds up to 2^16 by FIT and in an 8-bit checkpoint,
    which is an infinity as fp16 and a number as fp32; FLOOR saturates below."""
    x = torch.full((3, 40), 65504.0, dtype=torch.float16, device=DEV)
    m, c = F.Mxfp4(3, 40), F.Act8(3, 40)
    y16, y32 = torch.empty_like(x), torch.empty(3, 40, device=DEV)
    for rule, value in ((F.MX_FLOOR, 6 * 2.0 ** 13), (F.MX_FIT, 2.0 ** 16)):
        F.mxfp4_quantize(x, m, rule=rule)
        F.mxfp4_dequantize(m, y16)
        F.mxfp4_dequantize(m, y32)
        torch.cuda.synchronize()
        assert (y32 == value).all() and (y16 == (value if value < 65504 else float("inf"))).all()
    F.act8_quantize(x, c)
    F.act8_dequantize(c, y16)
    F.act8_dequantize(c, y32)
    torch.cuda.synchronize()
    assert (y32 == 2.0 ** 16).all() and torch.isinf(y16).all()
