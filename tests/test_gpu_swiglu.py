"""8-bit checkpoints and the gated activation against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHAPES = [(1, 1), (1, 8), (3, 31), (5, 33), (64, 128), (17, 1000), (37, 1001), (200, 40), (1, 14336), (300, 2048)]


def rand(shape, dtype, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(R.DTYPES[dtype]).to(DEV)


def act8_same(c, x):
    codes, s = R.act8(R.f64(x))
    rows, n = s.shape
    assert np.array_equal(c.s.cpu().numpy().astype(np.int64), s)
    assert np.array_equal(c.q.cpu().numpy().astype(np.int64).reshape(rows, n, 32), codes)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_checkpoint(rows, cols, dtype):
    x = rand((rows, cols), dtype, rows + cols)
    x = x * torch.exp2(torch.arange(cols, device=DEV) % 13 - 6).to(x.dtype)
    c = F.Act8(rows, cols)
    F.act8_quantize(x, c)
    y = torch.empty((rows, cols), device=DEV)
    F.act8_dequantize(c, y)
    z = torch.empty_like(x)
    F.act8_dequantize(c, z)
    torch.cuda.synchronize()
    act8_same(c, x)
    want = R.act8_values(R.f64(x))
    assert np.array_equal(R.f64(y), want)
    assert torch.equal(z.cpu(), torch.from_numpy(want).to(z.dtype))
    # the documented distance: 2^-4 of the value, or 2^-10 of the scale
    scale = np.repeat(2.0 ** (c.s.cpu().numpy().astype(np.float64) - 127), 32, axis=1)[:, :cols]
    v = R.f64(x)
    assert (np.abs(want - v) <= np.maximum(np.abs(v) * 2.0 ** -4, scale * 2.0 ** -10)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_checkpoint_of_every_16_bit_value(dtype):
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(R.DTYPES[dtype])
    # one value a block, next to a larger one
    v = torch.zeros(65536, 32, dtype=x.dtype)
    v[:, 5] = x
    v[:, 9] = torch.where(x.float().abs() * 100 <= torch.finfo(x.dtype).max, x.float() * 100, x.float()).to(x.dtype)
    v = v.view(2048, 1024).to(DEV)
    c = F.Act8(*v.shape)
    F.act8_quantize(v, c)
    torch.cuda.synchronize()
    act8_same(c, v)


def test_checkpoint_extremes():
    big = torch.finfo(torch.float32).max
    x = torch.zeros(8, 64)
    for i, v in enumerate([big, 2.0 ** -149, 448.0, 449.0, float("inf"), float("nan"), 2.0 ** -126, 0.0]):
        x[i, 1], x[i, 2], x[i, 40] = v, -v / 3, 1.0
    x = x.to(DEV)
    c = F.Act8(8, 64)
    F.act8_quantize(x, c)
    y = torch.empty_like(x)
    F.act8_dequantize(c, y)
    torch.cuda.synchronize()
    act8_same(c, x)
    assert np.array_equal(R.f64(y), R.act8_values(R.f64(x)), equal_nan=True)
    assert torch.isnan(y[4:6, :32]).all() and torch.isfinite(y[4:6, 32:]).all() and torch.isfinite(y[:4]).all()


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(rows, cols, dtype, ckpt):
    g, u, da = rand((rows, cols), dtype, 1, 3.0), rand((rows, cols), dtype, 2), rand((rows, cols), dtype, 3)
    a, dg, du = (torch.empty_like(g) for _ in range(3))
    cg, cu = (F.Act8(rows, cols), F.Act8(rows, cols)) if ckpt else (None, None)
    F.swiglu_fwd(g, u, a, cg, cu)
    F.swiglu_bwd(da, cg if ckpt else g, cu if ckpt else u, dg, du)
    torch.cuda.synchronize()
    vg, vu = R.f64(g), R.f64(u)
    R.check(a, *R.swiglu(vg, vu), "a")
    if ckpt:
        act8_same(cg, g)
        act8_same(cu, u)
        vg, vu = R.act8_values(vg), R.act8_values(vu)
    (wg, bg), (wu, bu) = R.swiglu_grad(R.f64(da), vg, vu)
    R.check(dg, wg, bg, "dg")
    R.check(du, wu, bu, "du")


def test_gradient_against_differences():
    """The formula's gradient is the slope of the formula (64 bits)."""
    g, u, h = np.linspace(-8, 8, 161), np.linspace(-2, 2, 161), 1e-6
    (dg, _), (du, _) = R.swiglu_grad(np.ones(161), g, u)
    assert np.abs(dg - (R.swiglu(g + h, u)[0] - R.swiglu(g - h, u)[0]) / (2 * h)).max() < 1e-8
    assert np.abs(du - (R.swiglu(g, u + h)[0] - R.swiglu(g, u - h)[0]) / (2 * h)).max() < 1e-8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(33, 64), (20, 100), (7, 31)])
def test_halves_of_one_matrix(rows, cols, dtype):
    """g and u as the two halves of one product's output, gradients into the
    halves of one matrix; what lies around them is left alone."""
    both = rand((rows, 2 * cols + 3), dtype, 1)
    g, u = both[:, 1:cols + 1], both[:, cols + 2:2 * cols + 2]
    da = rand((rows, cols), dtype, 2)
    a = torch.empty_like(da)
    cg, cu = F.Act8(rows, cols), F.Act8(rows, cols)
    F.swiglu_fwd(g, u, a, cg, cu)
    d = torch.full_like(both, 9.0)
    F.swiglu_bwd(da, g, u, d[:, 1:cols + 1], d[:, cols + 2:2 * cols + 2])
    torch.cuda.synchronize()
    act8_same(cg, g)
    act8_same(cu, u)
    R.check(a, *R.swiglu(R.f64(g), R.f64(u)), "a")
    (wg, bg), (wu, bu) = R.swiglu_grad(R.f64(da), R.f64(g), R.f64(u))
    R.check(d[:, 1:cols + 1], wg, bg, "dg")
    R.check(d[:, cols + 2:2 * cols + 2], wu, bu, "du")
    assert (d[:, 0] == 9).all() and (d[:, cols + 1] == 9).all() and (d[:, -1] == 9).all()


def test_gradients_in_place():
    g, u, da = rand((50, 96), "bf16", 1), rand((50, 96), "bf16", 2), rand((50, 96), "bf16", 3)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    F.swiglu_bwd(da, g, u, dg, du)
    F.swiglu_bwd(da, g, u, g, u)
    torch.cuda.synchronize()
    assert torch.equal(g, dg) and torch.equal(u, du)


def test_far_arguments():
    """Saturated gates: exact zeros and pass-through, never NaN from finite inputs."""
    g = torch.tensor([[-3e38, -1e4, -200.0, -100.0, -88.0, 0.0, 88.0, 200.0, 1e4, 3e38]], device=DEV)
    u, da = torch.full_like(g, 0.5), torch.ones_like(g)
    a, dg, du = (torch.empty_like(g) for _ in range(3))
    F.swiglu_fwd(g, u, a)
    F.swiglu_bwd(da, g, u, dg, du)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        R.check(a, *R.swiglu(R.f64(g), R.f64(u)), "a")
        (wg, bg), (wu, bu) = R.swiglu_grad(R.f64(da), R.f64(g), R.f64(u))
    assert torch.isfinite(dg).all() and torch.isfinite(du).all()
    R.check(du, wu, bu, "du")
    R.check(dg, wg, bg, "dg")


def test_a_nan_stays_in_its_block():
    g, u, da = rand((4, 96), "bf16", 1), rand((4, 96), "bf16", 2), rand((4, 96), "bf16", 3)
    g[1, 40] = float("inf")
    a, dg, du = (torch.empty_like(g) for _ in range(3))
    cg, cu = F.Act8(4, 96), F.Act8(4, 96)
    F.swiglu_fwd(g, u, a, cg, cu)
    F.swiglu_bwd(da, cg, cu, dg, du)
    torch.cuda.synchronize()
    for t in (dg, du):
        bad = torch.isnan(t)
        assert bad[1, 32:64].all() and bad.sum() == 32


def test_empty():
    for shape in ((0, 8), (3, 0)):
        t = torch.empty(shape, device=DEV)
        F.swiglu_fwd(t, t, t.clone(), F.Act8(*shape), F.Act8(*shape))
        F.swiglu_bwd(t, F.Act8(*shape), F.Act8(*shape), t.clone(), t.clone())
    torch.cuda.synchronize()


@pytest.mark.parametrize("ckpt", [False, True])
def test_fp32_keeps_its_precision_over_the_whole_range(ckpt):
    """fp32 values in and out: errors in half steps of fp32 (U), whatever |g|.  t =
    exp(-|g|) is off by a step (2 U), 1 + t by 2, r = 1 / (1 + t) by 3, t r by 6;
    sigmoid is one of r and t r, 1 - sigmoid the other.  Two products more each
    for a and du (8 U); dg's factor 1 + g (1 - sigmoid) is off by 7 U of |g| (1 -
    sigmoid) and U of itself, and three more products follow (10 U)."""
    g = torch.linspace(-86, 86, 64 * 500, device=DEV).view(64, 500)
    u, da = rand((64, 500), "f32", 1), rand((64, 500), "f32", 2)
    a, dg, du = (torch.empty_like(g) for _ in range(3))
    cg, cu = (F.Act8(64, 500), F.Act8(64, 500)) if ckpt else (None, None)
    F.swiglu_fwd(g, u, a, cg, cu)
    F.swiglu_bwd(da, cg if ckpt else g, cu if ckpt else u, dg, du)
    torch.cuda.synchronize()
    vg, vu, vda = R.f64(g), R.f64(u), R.f64(da)

    def parts(v):  # sigmoid(v) and 1 - sigmoid(v), both to 64 bits
        return 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
    s, _ = parts(vg)
    want = vg * s * vu
    R.check(a, want, 8 * R.U32 * np.abs(want) + np.abs(vu) * 2.0 ** -140, "a")
    if ckpt:
        vg, vu = R.act8_values(vg), R.act8_values(vu)
    s, c = parts(vg)
    tiny = np.abs(vda) * (1 + np.abs(vu)) * 2.0 ** -140
    R.check(du, vda * vg * s, 8 * R.U32 * np.abs(vda * vg * s) + tiny, "du")
    f = 1 + vg * c
    bound = np.abs(vda * vu) * s * (7 * np.abs(vg) * c + 11 * np.abs(f)) * R.U32 + tiny
    R.check(dg, vda * vu * s * f, bound, "dg")


def test_gates_below_the_exponentials_range():
    """exp(90) is past fp32, silu(-90) is not: -90 exp(-90) is a normal number."""
    g = torch.full((1, 8), -87.5, device=DEV) - torch.arange(8, device=DEV) * 0.5
    u, da = torch.full_like(g, 1e10), torch.full_like(g, 1e10)
    a, dg, du = (torch.empty_like(g) for _ in range(3))
    F.swiglu_fwd(g, u, a)
    F.swiglu_bwd(da, g, u / 1e10, dg, du)
    torch.cuda.synchronize()
    v = R.f64(g)
    s = 1 / (1 + np.exp(-v))
    # exp(g) is subnormal here: off by half of 2^-149, times what it is multiplied by, and the roundings above
    step = 2.0 ** -149
    R.check(a, v * s * R.f64(u), np.abs(v) * R.f64(u) * (step + 8 * R.U32 * s) + R.f64(u) * step, "a")
    R.check(du, v * s * R.f64(da), np.abs(v) * R.f64(da) * (step + 8 * R.U32 * s) + R.f64(da) * step, "du")
    want = R.f64(da) * s * (1 + v / (1 + np.exp(v)))
    R.check(dg, want, np.abs(v) * R.f64(da) * (2 * step + 20 * R.U32 * s), "dg")
    assert bool((a < 0).all()) and bool((dg < 0).all())
