"""Dropout with a counter-based generator against its definition."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import epilogue_reference as E
from tests import mx_reference as R
from tests.test_gpu_epilogue import GUARD, rand, rng_words

pytestmark = pytest.mark.gpu
DEV = "cuda"


def want(x, factor, residual):
    """drop(x) (+ residual) and its bound: the scale's rounding and the product's, then the sum's."""
    v = np.where(factor == 0, 0.0, x * factor)
    err = 2 * E.U32 * np.abs(v)
    if residual is not None:
        v = v + residual
        err = err + E.U32 * np.abs(v)
    return v, err


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0, 2.0 ** -18, 2.0 ** -16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (5, 1027), (300, 7), (64, 256), (33, 4097), (1000, 1)])
def test_forward_and_backward(rows, cols, p, dtype):
    x, res, gy = rand((rows, cols), dtype, 1), rand((rows, cols), dtype, 2), rand((rows, cols), dtype, 3)
    rng = rng_words(rows + cols)
    factor = E.keep(rng.tolist(), rows, cols, p)
    y, y2, gx = (torch.full_like(x, GUARD) for _ in range(3))
    F.dropout_fwd(x, p, rng, y, residual=res)
    F.dropout_fwd(x, p, rng, y2)
    F.dropout_bwd(gy, p, rng, gx)
    R.check(y, *want(R.f64(x), factor, R.f64(res)), "y")
    R.check(y2, *want(R.f64(x), factor, None), "y alone")
    R.check(gx, *want(R.f64(gy), factor, None), "gx")


def test_gradient_against_differences():
    """The map is linear: f(x + d) - f(x) is f's gradient along d."""
    x, rng = rand((40, 100), "f32", 1), rng_words(3)
    d = torch.zeros_like(x)
    d[::3, ::5] = 1
    y0, y1, g = (torch.empty_like(x) for _ in range(3))
    F.dropout_fwd(x, 0.25, rng, y0)
    F.dropout_fwd(x + d, 0.25, rng, y1)
    F.dropout_bwd(d, 0.25, rng, g)
    assert torch.allclose(y1 - y0, g, rtol=0, atol=float(8 * 2.0 ** -24 * (x.abs().max() + 1) * 4 / 3))


def test_rows_apart_in_place_and_guards():
    rows, cols = 50, 93
    x, res, rng = rand((rows, cols), "bf16", 1), rand((rows, cols), "bf16", 2), rng_words(1)
    base = torch.empty_like(x)
    F.dropout_fwd(x, 0.5, rng, base, residual=res)
    wide = torch.full((rows + 2, 2 * cols + 9), GUARD, dtype=x.dtype, device=DEV)
    for off in (0, 1, 8):
        xs, ys = wide[1:rows + 1, off:off + cols], wide[1:rows + 1, off + cols:off + 2 * cols]
        xs.copy_(x)
        F.dropout_fwd(xs, 0.5, rng, ys, residual=res)
        assert torch.equal(ys, base)
        F.dropout_fwd(xs, 0.5, rng, xs, residual=res)
        assert torch.equal(xs, base)
        ys.copy_(res)
        xs.copy_(x)
        F.dropout_fwd(xs, 0.5, rng, ys, residual=ys)
        assert torch.equal(ys, base)
        xs.fill_(GUARD)
        ys.fill_(GUARD)
        assert (wide == GUARD).all()


def test_infinities_and_nan_where_nothing_is_kept():
    x = torch.full((30, 77), float("nan"), device=DEV)
    x[1::2] = float("-inf")
    rng = rng_words(2)
    y = torch.empty_like(x)
    F.dropout_fwd(x, 0.5, rng, y)
    factor, v = E.keep(rng.tolist(), 30, 77, 0.5), R.f64(y)
    assert (v[factor == 0] == 0).all()
    assert np.isnan(v[::2][factor[::2] > 0]).all() and np.isneginf(v[1::2][factor[1::2] > 0]).all()


def test_empty_and_more_dimensions():
    rng = rng_words(2)
    for shape in ((0, 5), (4, 0), (0,)):
        F.dropout_fwd(torch.empty(shape, device=DEV), 0.5, rng, torch.empty(shape, device=DEV))
    x = rand((2, 3, 5, 24), "bf16", 1)
    y, flat = torch.empty_like(x), torch.empty(30, 24, dtype=x.dtype, device=DEV)
    F.dropout_fwd(x, 0.5, rng, y)
    F.dropout_fwd(x.view(30, 24), 0.5, rng, flat)
    assert torch.equal(y.view(30, 24), flat)
    v, out = x[0, 0, 0], torch.empty(24, dtype=x.dtype, device=DEV)
    F.dropout_fwd(v, 0.5, rng, out)
    assert torch.equal(out, flat[0])


def test_past_2_to_31_elements():
    """Group numbers and byte offsets past 32 bits' signed range; the last rows against
    their definition."""
    rows, cols = 33000, 65544
    x = torch.full((rows, cols), 1.0, dtype=torch.bfloat16, device=DEV)
    rng = rng_words(8)
    F.dropout_fwd(x, 0.5, rng, x)
    g = cols // 8
    n = np.arange((rows - 2) * g, rows * g, dtype=np.uint64)
    seed, off = (v % 2 ** 64 for v in rng.tolist())
    m = 0xFFFFFFFF
    ctr = np.stack([n & np.uint64(m), n >> np.uint64(32), np.full_like(n, off & m), np.full_like(n, off >> 32)], -1)
    w = E.philox(ctr, (seed & m, seed >> 32))
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(2, cols)
    assert np.array_equal(R.f64(x[-2:]), np.where(u >= 32768, 2.0, 0.0))


def test_a_captured_dropout_reads_its_words_when_it_runs():
    x, rng = rand((100, 300), "bf16", 1), rng_words(1)
    y, want_y = torch.empty_like(x), torch.empty_like(x)
    F.dropout_fwd(x, 0.5, rng, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.dropout_fwd(x, 0.5, rng, y)
    for k in range(4):
        rng.copy_(rng_words(20 + k))
        F.dropout_fwd(x, 0.5, rng, want_y)
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(y, want_y)
