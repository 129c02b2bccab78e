"""Products with an epilogue and their backward pass against the definition in 64
bits."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import epilogue_reference as E
from tests import mx_reference as R
from tests.parity import GROUP_ALIGN, gamma

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 77.0


def rand(shape, dtype, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(R.DTYPES[dtype]).to(DEV)


def rng_words(seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=g).to(DEV)


def tensors(M, N, dtype, bias, residual, p, seed):
    """(keyword arguments, the same in 64 bits) of an epilogue."""
    kw, ref = {"p": p}, {"factor": np.ones((M, N)), "bias": None, "residual": None}
    if bias:
        kw["bias"] = rand((N,), bias, seed + 1, 0.5)
        ref["bias"] = R.f64(kw["bias"])
    if residual:
        kw["residual"] = rand((M, N), dtype, seed + 2)
        ref["residual"] = R.f64(kw["residual"])
    if p:
        kw["rng"] = rng_words(seed + 3)
        ref["factor"] = E.keep(kw["rng"].tolist(), M, N, p)
    return kw, ref


def verify(y, pre, prod, prod_err, act, ref, fast, what):
    h, h_err, v, v_err = E.forward(prod, prod_err, ref["bias"], act, ref["residual"], ref["factor"], fast)
    R.check(y, v, v_err, f"{what} y")
    if pre is not None:
        R.check(pre, h, h_err, f"{what} h")


def mx_operands(M, N, K, seed, rule=F.MX_FLOOR, dtype="f32"):
    x, w = rand((M, K), dtype, seed), rand((N, K), dtype, seed + 9, 0.05)
    a, b = F.Mxfp4(M, K), F.Mxfp4(N, K)
    F.mxfp4_quantize(x, a, rule=rule)
    F.mxfp4_quantize(w, b, rule=rule)
    fit = rule == F.MX_FIT
    return x, w, a, b, R.dot(R.fp4_values(R.f64(x), fit), R.fp4_values(R.f64(w), fit))


# one workgroup's waves, joined or alone; tiles of 16, 32, 64; 128; 256; a contraction of nothing
SHAPES = [(1, 1, 1), (1, 300, 700), (3, 33, 300), (24, 512, 1000), (40, 200, 96), (100, 96, 3000), (200, 200, 2000),
          (300, 1031, 500), (1000, 1031, 333), (2600, 4100, 96), (17, 70, 0)]


@pytest.mark.parametrize("act", E.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_mx_product(M, N, K, dtype, act):
    seed = M * 7 + N + K + act
    _, _, a, b, (prod, err) = mx_operands(M, N, K, seed)
    kw, ref = tensors(M, N, dtype, dtype if act % 2 else "f32", act != 2, 0.25 if act != 3 else 0.0, seed)
    y = torch.full((M, N), GUARD, dtype=R.DTYPES[dtype], device=DEV)
    pre = torch.full_like(y, GUARD)
    F.mxfp4_gemm_epilogue(a, b, y, act=act, pre=pre, **kw)
    verify(y, pre, prod, err, act, ref, dtype != "f32", (M, N, K, dtype, act))


@pytest.mark.parametrize("M,N,K", [(1, 600, 1000), (200, 200, 512), (300, 1031, 500), (2600, 4100, 64)])
def test_an_empty_epilogue_is_the_plain_product(M, N, K):
    _, _, a, b, _ = mx_operands(M, N, K, 5)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        want, got = torch.empty(M, N, dtype=dtype, device=DEV), torch.empty(M, N, dtype=dtype, device=DEV)
        F.mxfp4_gemm(a, b, want)
        F.mxfp4_gemm_epilogue(a, b, got)
        assert torch.equal(want, got)


@pytest.mark.parametrize("M,N,K", [(5, 37, 300), (300, 1031, 200), (2600, 4100, 64)])
def test_strided_rows_in_place_and_what_lies_around(M, N, K):
    """Output and residual in column ranges of wider matrices, at any alignment; the
    residual as the output itself; nothing else is written."""
    _, _, a, b, (prod, err) = mx_operands(M, N, K, 11)
    kw, ref = tensors(M, N, "bf16", "bf16", True, 0.25, 3)
    for off, ld in ((0, N + 8), (1, N + 3), (3, 2 * N + 5)):
        wide = torch.full((M + 2, ld + 4), GUARD, dtype=torch.bfloat16, device=DEV)
        y = wide[1:M + 1, off:off + N]
        res = torch.zeros(M, ld, dtype=torch.bfloat16, device=DEV)[:, off:off + N]
        res.copy_(kw["residual"])
        F.mxfp4_gemm_epilogue(a, b, y, act=F.ACT_SILU, **{**kw, "residual": res})
        verify(y, None, prod, err, F.ACT_SILU, ref, True, "strided")
        first = y.clone()
        y.copy_(kw["residual"])
        F.mxfp4_gemm_epilogue(a, b, y, act=F.ACT_SILU, **{**kw, "residual": y})
        assert torch.equal(y, first)
        y.fill_(GUARD)
        assert (wide == GUARD).all()


@pytest.mark.parametrize("M", [1, 2, 4, 5, 24, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rule", [F.MX_FLOOR, F.MX_FIT])
def test_mx_apply_and_training_forward(M, dtype, rule):
    N, K = 333, 1500
    x, w, _, b, (prod, err) = mx_operands(M, N, K, M, rule, dtype)
    for act, p, out in ((F.ACT_GELU, 0.0, dtype), (F.ACT_NONE, 0.5, dtype), (F.ACT_GELU_TANH, 0.0, "f32")):
        kw, ref = tensors(M, N, out, dtype, True, p, M + act)
        y = torch.empty(M, N, dtype=R.DTYPES[out], device=DEV)
        F.mxfp4_linear_apply_epilogue(x, b, y, F.Mxfp4(M, K), act=act, rule=rule, **kw)
        verify(y, None, prod, err, act, ref, out != "f32", (M, dtype, "apply"))
        ws, saved, saved2 = F.Mxfp4LinearWs(M, N, K), F.Mxfp4LinearSaved(M, N, K), F.Mxfp4LinearSaved(M, N, K)
        pre = torch.empty_like(y)
        F.mxfp4_linear_fwd_epilogue(x, w, ws, saved, y, act=act, pre=pre, rule=rule, **kw)
        verify(y, pre, prod, err, act, ref, out != "f32", (M, dtype, "forward"))
        F.mxfp4_linear_fwd(x, w, ws, saved2, torch.empty_like(y), rule=rule)
        for m, m2 in ((saved.x_qT, saved2.x_qT), (saved.w_qT, saved2.w_qT)):
            assert all(np.array_equal(u, v) for u, v in zip(R.fp4_unpack(m), R.fp4_unpack(m2)))


def test_leading_dimensions_are_rows():
    x, w, _, b, (prod, err) = mx_operands(6, 40, 100, 2, dtype="bf16")
    kw, ref = tensors(6, 40, "bf16", "bf16", True, 0.25, 8)
    y = torch.empty(2, 3, 40, dtype=torch.bfloat16, device=DEV)
    kw["residual"] = kw["residual"].view(2, 3, 40)
    F.mxfp4_linear_apply_epilogue(x.view(2, 3, 100), b, y, F.Mxfp4(6, 100), act=F.ACT_RELU, **kw)
    verify(y.view(6, 40), None, prod, err, F.ACT_RELU, ref, True, "3-D")


def test_contractions_past_32_bit_offsets():
    M, N, K = 3, 5, (1 << 24) + 40
    a, b = F.Mxfp4(M, K), F.Mxfp4(N, K)
    x, w = torch.ones(M, K, dtype=torch.bfloat16, device=DEV), torch.full((N, K), 0.5, dtype=torch.bfloat16, device=DEV)
    x[1] = -1
    F.mxfp4_quantize(x, a)
    F.mxfp4_quantize(w, b)
    y = torch.empty(M, N, dtype=torch.float32, device=DEV)
    F.mxfp4_gemm_epilogue(a, b, y, act=F.ACT_RELU, bias=torch.arange(N, dtype=torch.float32, device=DEV))
    want = np.maximum(np.array([1, -1, 1])[:, None] * (K / 2) + np.arange(N)[None], 0)
    R.check(y, want, 64 * E.U32 * K, "long")  # sums of powers of two and multiples of 64: few roundings


# ------------------------------------------------------- activations, point by point

def points(dtype):
    """Every finite 16-bit value, or fp32 values over the whole range; then infinities and NaN."""
    if dtype == "f32":
        g = np.random.default_rng(1)
        v = np.concatenate([np.linspace(-20, 20, 60001), g.normal(size=40000) * 3, np.exp(g.uniform(-90, 88, 20000)),
                            -np.exp(g.uniform(-90, 88, 20000)), [0.0, -0.0, np.inf, -np.inf, np.nan]])
        return torch.tensor(v, dtype=torch.float32, device=DEV)
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(R.DTYPES[dtype])
    return v.to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", E.ACTS)
def test_activation_of_every_value(act, dtype):
    """An empty contraction leaves act(bias)."""
    b = points(dtype)
    y = torch.empty(1, b.numel(), dtype=b.dtype, device=DEV)
    F.mxfp4_gemm_epilogue(F.Mxfp4(1, 0), F.Mxfp4(b.numel(), 0), y, bias=b, act=act)
    h = R.f64(b)[None]
    R.check(y, E.act(h, act), E.act_err(h, act, dtype != "f32"), (act, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", E.ACTS)
def test_slope_of_every_value(act, dtype):
    h = points(dtype)[None].contiguous()
    gy = torch.ones_like(h)
    gh = torch.empty_like(h)
    F.epilogue_bwd(gy, gh, pre=h, act=act)
    v = R.f64(h)
    want = np.where(np.isnan(v) & (act not in (E.NONE, E.RELU)), np.nan, E.slope(np.nan_to_num(v, nan=1.0), act))
    R.check(gh, want, E.slope_err(np.nan_to_num(v, nan=1.0), act, dtype != "f32"), (act, dtype))


@pytest.mark.parametrize("act", [a for a in E.ACTS if a not in (E.NONE, E.RELU)])
def test_slope_against_differences_of_the_forward(act):
    """fp32: (act(h + d) - act(h - d)) / 2 d from the forward kernel, d a power of two:
    off by the forward's errors over d and by d^2 / 6 of the third derivative (below 4)."""
    d = 2.0 ** -7
    h = torch.arange(-640, 641, dtype=torch.float32, device=DEV)[None] / 64

    def fwd(b):
        y = torch.empty(1, b.numel(), device=DEV)
        F.mxfp4_gemm_epilogue(F.Mxfp4(1, 0), F.Mxfp4(b.numel(), 0), y, bias=b[0].contiguous(), act=act)
        return R.f64(y)
    diff = (fwd(h + d) - fwd(h - d)) / (2 * d)
    gh = torch.empty_like(h)
    F.epilogue_bwd(torch.ones_like(h), gh, pre=h, act=act)
    v = np.abs(R.f64(h)) + d
    err = (E.act_err(v, act, False) + E.act_err(-v, act, False)) / d + 4 * d * d / 6 + 2 * E.slope_err(R.f64(h), act, False)
    assert (np.abs(diff - R.f64(gh)) <= err).all()


# ------------------------------------------------------------------------------ FP8

def fp8_product(saved):
    """The product of the saved codes and its bound (the matrix instruction's
    alignment inside groups of 8, tests/parity.py)."""
    def val(q, rec):
        return q.view(torch.float8_e4m3fn).float().cpu().double().numpy(), rec.read()["inv"]
    (x, xi), (w, wi) = val(saved.x_q, saved.x_sc), val(saved.w_q, saved.w_sc)
    alpha = float(np.float32(xi * wi))
    K = x.shape[1]
    return alpha * (x @ w.T), (GROUP_ALIGN + 2 * gamma(K)) * alpha * (np.abs(x) @ np.abs(w).T) + \
        E.U32 * np.abs(alpha * (x @ w.T))


@pytest.mark.parametrize("act", E.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(16, 16, 16), (64, 256, 128), (48, 400, 272), (336, 528, 144), (2880, 3104, 144),
                                   (2880, 3104, 128), (3584, 4096, 128)])
def test_fp8_forward(M, N, K, dtype, act):
    x, w = rand((M, K), dtype, M + act), rand((N, K), dtype, N, 0.05)
    saved = F.LinearSaved(M, N, K, transposed=act % 2 == 1)
    out = dtype if act else "f32"
    kw, ref = tensors(M, N, out, dtype if act != 2 else "f32", act != 1, 0.25 if act != 3 else 0.0, act)
    y = torch.full((M, N), GUARD, dtype=R.DTYPES[out], device=DEV)
    pre = torch.full_like(y, GUARD)
    F.fp8_scaled_linear_fwd_epilogue(x, w, saved, y, act=act, pre=pre, **kw)
    prod, err = fp8_product(saved)
    verify(y, pre, prod, err, act, ref, True, (M, N, K, dtype, act))
    # the codes and records are those of the layer without an epilogue
    plain = F.LinearSaved(M, N, K, transposed=act % 2 == 1)
    if dtype == "bf16":
        F.fp8_scaled_linear_fwd(x, w, plain, torch.empty(M, N, dtype=torch.bfloat16, device=DEV))
    else:
        for t, sc, q, qT in ((x, plain.x_sc, plain.x_q, plain.x_qT), (w, plain.w_sc, plain.w_q, plain.w_qT)):
            F.fp8_amax_f16(t, sc)
            F.fp8_quantize_f16(t, F.E4M3FN, sc, q, qT)
    for u, v in zip(saved.tensors()[:4], plain.tensors()[:4]):
        assert (u is None and v is None) or torch.equal(u, v)
    assert saved.x_sc.read()["inv"] == plain.x_sc.read()["inv"]
    # the product alone, from the codes
    y2 = torch.empty_like(y)
    F.fp8_gemm_epilogue(saved.x_q, saved.w_q, saved.x_sc.inv_ptr(), saved.w_sc.inv_ptr(), y2, act=act, **kw)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("M,N,K", [(48, 400, 272), (2880, 3104, 144), (2880, 3104, 128)])
def test_fp8_rowwise_product(M, N, K):
    x, w = rand((M, K), "bf16", 1), rand((N, K), "bf16", 2, 0.05)
    x *= torch.exp2(torch.arange(M, device=DEV) % 7 - 3.0)[:, None].bfloat16()
    xq, wq = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(N, K, dtype=torch.uint8, device=DEV)
    xs, ws = F.RowScalesDev(M), F.RowScalesDev(N)
    F.fp8_quantize_rowwise(x, F.E4M3FN, xs, xq)
    F.fp8_quantize_rowwise(w, F.E4M3FN, ws, wq)
    kw, ref = tensors(M, N, "bf16", "f32", True, 0.25, 4)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    pre = torch.empty_like(y)
    F.fp8_gemm_rowwise_epilogue(xq, wq, xs.inv, ws.inv, y, act=F.ACT_GELU, pre=pre, **kw)
    a, b = (q.view(torch.float8_e4m3fn).float().cpu().double().numpy() for q in (xq, wq))
    alpha = np.outer(R.f64(xs.inv), R.f64(ws.inv)).astype(np.float32).astype(np.float64)
    prod = alpha * (a @ b.T)
    err = (GROUP_ALIGN + 2 * gamma(K)) * alpha * (np.abs(a) @ np.abs(b).T) + E.U32 * np.abs(prod)
    verify(y, pre, prod, err, F.ACT_GELU, ref, True, "rowwise")


def test_fp8_empty_contraction():
    y = torch.empty(16, 32, dtype=torch.bfloat16, device=DEV)
    inv = torch.ones(1, dtype=torch.float64, device=DEV)
    e = torch.empty(16, 0, dtype=torch.uint8, device=DEV), torch.empty(32, 0, dtype=torch.uint8, device=DEV)
    bias = rand((32,), "bf16", 1)
    F.fp8_gemm_epilogue(*e, inv.data_ptr(), inv.data_ptr(), y, bias=bias, act=F.ACT_RELU, residual=torch.ones_like(y))
    assert torch.equal(y, (bias.clamp(min=0).float() + 1).bfloat16().expand(16, 32))


# ------------------------------------------------------------- the backward step

BWD = [(1, 1), (3, 7), (5, 1027), (64, 256), (130, 8), (257, 64), (1000, 513), (4100, 96), (37, 9000), (2048, 2056)]


@pytest.mark.parametrize("act", E.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", BWD)
def test_backward_step(M, N, dtype, act):
    gy, pre = rand((M, N), dtype, M, 0.1), rand((M, N), dtype, N, 2.0)
    p = 0.25 if act != 4 else 0.0
    rng = rng_words(M + N)
    factor = E.keep(rng.tolist(), M, N, p)
    gh, gh_err, gb, gb_err = E.backward(R.f64(gy), R.f64(pre), act, factor, dtype != "f32")
    part = torch.full((F.epilogue_workspace_len(M, N) + 3,), GUARD, device=DEV)
    for gtype in ("f32", dtype):
        g, b = torch.full_like(gy, GUARD), torch.full((N,), GUARD, dtype=R.DTYPES[gtype], device=DEV)
        F.epilogue_bwd(gy, g, b, pre=pre, act=act, p=p, rng=rng, part=part)
        R.check(g, gh, gh_err, "gh")
        R.check(b, gb, gb_err, "gb")
        assert (part[F.epilogue_workspace_len(M, N):] == GUARD).all()
        again, inplace = torch.empty_like(b), gy.clone()
        F.epilogue_bwd(inplace, inplace, again, pre=pre, act=act, p=p, rng=rng, part=part)
        assert torch.equal(again, b) and torch.equal(inplace, g)
        F.epilogue_bwd(gy, None, again, pre=pre, act=act, p=p, rng=rng, part=part)
        assert torch.equal(again, b)
        g2 = torch.empty_like(g)
        F.epilogue_bwd(gy, g2, pre=pre, act=act, p=p, rng=rng)
        assert torch.equal(g2, g)


def test_backward_of_no_rows():
    b = torch.full((40,), GUARD, device=DEV)
    F.epilogue_bwd(torch.empty(0, 40, device=DEV), None, b)
    assert (b == 0).all()
    F.epilogue_bwd(torch.empty(4, 0, device=DEV), torch.empty(4, 0, device=DEV), torch.empty(0, device=DEV))


def test_dropped_gradients_are_zero_whatever_they_were():
    M, N = 40, 200
    rng = rng_words(5)
    factor = E.keep(rng.tolist(), M, N, 0.5)
    gy = torch.full((M, N), float("nan"), device=DEV)
    gy[::2] = float("inf")
    pre = torch.full_like(gy, float("nan"))
    gh = torch.empty_like(gy)
    F.epilogue_bwd(gy, gh, pre=pre, act=F.ACT_SILU, p=0.5, rng=rng)
    g = R.f64(gh)
    assert (g[factor == 0] == 0).all() and np.isnan(g[factor > 0]).all()
    _, _, a, b, _ = mx_operands(M, N, 64, 1)
    bias = torch.full((N,), float("inf"), device=DEV)
    y = torch.empty(M, N, device=DEV)
    F.mxfp4_gemm_epilogue(a, b, y, bias=bias, p=0.5, rng=rng, residual=torch.ones(M, N, device=DEV))
    v = R.f64(y)
    assert (v[factor == 0] == 1).all() and np.isposinf(v[factor > 0]).all()
    F.mxfp4_gemm_epilogue(a, b, y, bias=bias, p=1.0, rng=rng, residual=torch.ones(M, N, device=DEV))
    assert (y == 1).all()


def e5m2(x):
    """The values of a tensor's e5m2 codes and the inverse scale, from the definition."""
    s = 57344.0 / max(np.abs(x).max(), 1e-12)
    v = (x.astype(np.float32) * np.float32(s)).astype(np.float64)
    ulp = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -14))) - 2)
    return np.clip(np.round(v / ulp) * ulp, -57344, 57344), 1 / s


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(16, 16, 16), (64, 256, 128), (336, 528, 144), (1024, 1040, 96)])
@pytest.mark.parametrize("transposed", [False, True])
def test_fp8_backward(M, N, K, dtype, transposed):
    """gx and gw from the codes of the device's own gh, which is held to its definition."""
    x, w = rand((M, K), dtype, 1), rand((N, K), dtype, 2, 0.05)
    gy, pre = rand((M, N), dtype, 3, 0.1), rand((M, N), dtype, 4, 2.0)
    rng = rng_words(7)
    saved, ws = F.LinearSaved(M, N, K, transposed=transposed), F.LinearBwdWs(M, N, transposed=transposed)
    F.fp8_scaled_linear_fwd_epilogue(x, w, saved, torch.empty(M, N, dtype=gy.dtype, device=DEV))

    def val(q, rec):
        return q.view(torch.float8_e4m3fn).float().cpu().double().numpy(), rec.read()["inv"]
    (xv, xi), (wv, wi) = val(saved.x_q, saved.x_sc), val(saved.w_q, saved.w_sc)
    part = torch.empty(F.epilogue_workspace_len(M, N), device=DEV)
    for act, p, with_gb in ((F.ACT_GELU, 0.25, True), (F.ACT_NONE, 0.0, True), (F.ACT_NONE, 0.5, False), (F.ACT_NONE, 0.0, False)):
        factor = E.keep(rng.tolist(), M, N, p)
        want, want_err, gb, gb_err = E.backward(R.f64(gy), R.f64(pre), act, factor, True)
        same = act == F.ACT_NONE and p == 0
        gh = None if same else torch.full_like(gy, GUARD)
        b = torch.full((N,), GUARD, device=DEV) if with_gb else None
        gx, gw = torch.empty(M, K, dtype=gy.dtype, device=DEV), torch.empty(N, K, dtype=gy.dtype, device=DEV)
        F.fp8_scaled_linear_bwd_epilogue(gy, saved, ws, gx, gw, gh=gh, gb=b, pre=pre if act else None, act=act, p=p,
                                         rng=rng, part=part)
        if not same:
            R.check(gh, want, want_err, "gh")
        if with_gb:
            R.check(b, gb, gb_err, "gb")
        g, gi = e5m2(R.f64(gy if same else gh))
        assert np.array_equal(ws.gy_q.view(torch.float8_e5m2).float().cpu().double().numpy(), g)
        assert ws.gy_sc.read()["inv"] == gi
        for got, a, c, inv, what in ((gx, g, wv, wi, "gx"), (gw, g.T, xv, xi, "gw")):
            alpha, n = float(np.float32(gi * inv)), a.shape[1]
            ref = alpha * (a @ c)
            R.check(got, ref, (GROUP_ALIGN + 2 * gamma(n)) * alpha * (np.abs(a) @ np.abs(c)) + 2 * E.U32 * np.abs(ref), what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 70), (65, 130, 300), (600, 520, 200)])
def test_mx_backward(M, N, K, dtype):
    x, w = rand((M, K), dtype, 1), rand((N, K), dtype, 2, 0.05)
    gy, pre = rand((M, N), dtype, 3, 0.1), rand((M, N), dtype, 4, 2.0)
    rng = rng_words(9)
    ws, saved = F.Mxfp4LinearWs(M, N, K), F.Mxfp4LinearSaved(M, N, K)
    F.mxfp4_linear_fwd_epilogue(x, w, ws, saved, torch.empty(M, N, dtype=gy.dtype, device=DEV))
    part = torch.empty(F.epilogue_workspace_len(M, N), device=DEV)
    for act, p, kinds in ((F.ACT_GELU_TANH, 0.25, "xwb"), (F.ACT_NONE, 0.0, "xwb"), (F.ACT_SILU, 0.0, "x"),
                          (F.ACT_RELU, 0.5, "wb"), (F.ACT_RELU, 0.5, "b"), (F.ACT_NONE, 0.0, "b")):
        factor = E.keep(rng.tolist(), M, N, p)
        want, want_err, gb, gb_err = E.backward(R.f64(gy), R.f64(pre), act, factor, dtype != "f32")
        same = act == F.ACT_NONE and p == 0
        gh = None if same or kinds == "b" else torch.full_like(gy, GUARD)
        gx = torch.empty(M, K, dtype=gy.dtype, device=DEV) if "x" in kinds else None
        gw = torch.empty(N, K, dtype=gy.dtype, device=DEV) if "w" in kinds else None
        b = torch.empty(N, dtype=gy.dtype, device=DEV) if "b" in kinds else None
        F.mxfp4_linear_bwd_epilogue(gy, ws, saved, gx, gw, gh=gh, gb=b, pre=pre if act else None, act=act, p=p, rng=rng,
                                    part=part)
        if gh is not None:
            R.check(gh, want, want_err, "gh")
        if b is not None:
            R.check(b, gb, gb_err, "gb")
        g = gy if same else gh
        ex, ew = (torch.empty_like(t) if t is not None else None for t in (gx, gw))
        if gx is not None or gw is not None:  # the plain backward of the same gradient
            F.mxfp4_linear_bwd(g, ws, saved, ex, ew)
        assert gx is None or torch.equal(gx, ex)
        assert gw is None or torch.equal(gw, ew)


# ------------------------------------------------------------------ streams and graphs

def test_a_captured_step_draws_new_masks_when_its_words_change():
    """Forward and backward of two layers in one graph, replayed with eager work and
    other words between; every replay equals the eager result for its words."""
    M, H, I = 96, 144, 272
    x, w1, w2 = rand((M, H), "bf16", 1), rand((I, H), "bf16", 2, 0.05), rand((H, I), "bf16", 3, 0.05)
    b1, b2, gy = rand((I,), "bf16", 4), rand((H,), "bf16", 5), rand((M, H), "bf16", 6, 0.1)
    rng = rng_words(1)

    class Step:
        def __init__(self):
            bf = dict(dtype=torch.bfloat16, device=DEV)
            self.s1, self.s2 = F.LinearSaved(M, I, H), F.LinearSaved(M, H, I)
            self.ws1, self.ws2 = F.LinearBwdWs(M, I), F.LinearBwdWs(M, H)
            self.h, self.a, self.y = torch.empty(M, I, **bf), torch.empty(M, I, **bf), torch.empty(M, H, **bf)
            self.ga, self.gx, self.g1, self.g2 = (torch.empty(M, I, **bf), torch.empty(M, H, **bf),
                                                  torch.empty(I, H, **bf), torch.empty(H, I, **bf))
            self.gh1, self.gh2 = torch.empty(M, I, **bf), torch.empty(M, H, **bf)
            self.gb1, self.gb2 = torch.empty(I, **bf), torch.empty(H, **bf)
            self.part = torch.empty(max(F.epilogue_workspace_len(M, n) for n in (H, I)), device=DEV)

        def run(self):
            F.fp8_scaled_linear_fwd_epilogue(x, w1, self.s1, self.a, bias=b1, act=F.ACT_GELU, pre=self.h)
            F.fp8_scaled_linear_fwd_epilogue(self.a, w2, self.s2, self.y, bias=b2, residual=x, p=0.25, rng=rng)
            F.fp8_scaled_linear_bwd_epilogue(gy, self.s2, self.ws2, self.ga, self.g2, gh=self.gh2, gb=self.gb2, p=0.25,
                                             rng=rng, part=self.part)
            F.fp8_scaled_linear_bwd_epilogue(self.ga, self.s1, self.ws1, self.gx, self.g1, gh=self.gh1, gb=self.gb1,
                                             pre=self.h, act=F.ACT_GELU, part=self.part)

        def results(self):
            return [t.clone() for t in (self.y, self.gx, self.g1, self.g2, self.gb1, self.gb2)]
    cap, eager = Step(), Step()
    cap.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            cap.run()
    seen = []
    for k in range(4):
        rng.copy_(rng_words(10 + k))
        eager.run()
        want = eager.results()
        torch.cuda.synchronize()
        graph.replay()
        got = cap.results()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])


def test_calls_on_another_stream():
    M, N, K = 200, 300, 500
    _, _, a, b, (prod, err) = mx_operands(M, N, K, 3)
    kw, ref = tensors(M, N, "bf16", "bf16", True, 0.25, 6)
    y = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        F.mxfp4_gemm_epilogue(a, b, y, act=F.ACT_GELU, **kw)
    s.synchronize()
    verify(y, None, prod, err, F.ACT_GELU, ref, True, "side stream")
    y.zero_()
    torch.cuda.synchronize()
    F.mxfp4_gemm_epilogue(a, b, y, act=F.ACT_GELU, stream=s, **kw)
    s.synchronize()
    verify(y, None, prod, err, F.ACT_GELU, ref, True, "given stream")
