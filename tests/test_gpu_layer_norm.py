"""Layer norm, forward and backward, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5
SHAPES = [(1, 1), (1, 64), (2, 7), (5, 1027), (33, 128), (3, 31), (17, 768), (300, 40), (64, 1000), (40, 4096),
          (9, 14336), (3, 20000), (2, 40001), (2000, 256)]


def rand(shape, dtype, seed, sigma=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma + shift).to(R.DTYPES[dtype]).to(DEV)


def v64(t):
    return None if t is None else R.f64(t)


def run(x, w, b, dy, ckpt, eps=EPS, pdtype=None):
    rows, cols = x.shape
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw = torch.empty(cols, dtype=pdtype or x.dtype, device=DEV)
    db = torch.empty_like(dw)
    c = F.Act8(rows, cols) if ckpt else None
    ws = torch.full((F.layer_norm_workspace_len(rows, cols),), float("nan"), device=DEV)
    F.layer_norm_fwd(x, w, b, eps, y, mean, rstd, c)
    F.layer_norm_bwd(dy, c if ckpt else x, w, mean, rstd, dx, dw, db, ws)
    torch.cuda.synchronize()
    return y, mean, rstd, c, dx, dw, db


def check_all(x, w, b, dy, ckpt, eps=EPS, pdtype=None):
    y, mean, rstd, c, dx, dw, db = run(x, w, b, dy, ckpt, eps, pdtype)
    ref = R.LayerNorm(v64(x), v64(w), v64(b), eps)
    R.check(y, ref.y, ref.y_err, "y")
    R.check(mean, ref.mean[:, 0], ref.mean_err[:, 0], "mean")
    R.check(rstd, ref.rstd[:, 0], (ref.rstd * ref.rstd_rel)[:, 0], "rstd")
    xv = v64(x)
    if ckpt:
        codes, s = R.act8(xv)
        assert np.array_equal(c.s.cpu().numpy().astype(np.int64), s)
        assert np.array_equal(c.q.cpu().numpy().astype(np.int64).reshape(codes.shape), codes)
        xv = R.act8_values(xv)
    for name, got, (want, bound) in zip(("dx", "dw", "db"), (dx, dw, db), ref.grads(v64(dy), xv)):
        R.check(got, want, bound, name)


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype,pdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(rows, cols, dtype, pdtype, ckpt):
    x, dy = rand((rows, cols), dtype, 1, 2.0, 0.5), rand((rows, cols), dtype, 2, 0.1)
    w, b = rand((cols,), pdtype, 3, 0.2, 1.0), rand((cols,), pdtype, 4, 0.2)
    check_all(x, w, b, dy, ckpt, pdtype=R.DTYPES[pdtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("has_w,has_b", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("cols", [100, 4096])
def test_without_parameters(cols, has_w, has_b, dtype):
    x, dy = rand((20, cols), dtype, 1), rand((20, cols), dtype, 2)
    w, b = (rand((cols,), dtype, 3) if f else None for f in (has_w, has_b))
    check_all(x, w, b, dy, False)


@pytest.mark.parametrize("cols", [64, 1001, 4096])
def test_constant_rows_and_a_far_mean(cols):
    """A row of one value has variance 0 (a padded row: all zeros); a mean far
    from zero must not swallow the deviations."""
    x = rand((6, cols), "f32", 1)
    x[1] = 0
    x[2] = 5.0
    x[3] += 1000.0
    dy = rand((6, cols), "f32", 2)
    check_all(x, rand((cols,), "f32", 3), rand((cols,), "f32", 4), dy, False)


@pytest.mark.parametrize("cols", [128, 5000])
def test_a_nan_stays_in_its_row(cols):
    x, dy = rand((7, cols), "bf16", 1), rand((7, cols), "bf16", 2)
    x[3, cols // 2] = float("nan")
    w = rand((cols,), "bf16", 3)
    y, _, _, _, dx, dw, db = run(x, w, w, dy, False)
    for t in (y, dx):
        bad = torch.isnan(t)
        assert bad[3].all() and bad.sum() == cols
    assert torch.isnan(dw).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("rows,cols", [(50, 300), (200, 4096), (2, 20000)])
def test_parts_and_repeats(rows, cols):
    """Each gradient on its own is the one computed with the others, a repeated
    call gives the same bits, and nothing past the outputs is written."""
    x, dy, w = rand((rows, cols), "bf16", 1), rand((rows, cols), "bf16", 2), rand((cols,), "f32", 3)
    y, mean, rstd, _, dx, dw, db = run(x, w, None, dy, False, pdtype=torch.float32)
    y2 = torch.empty_like(y)
    F.layer_norm_fwd(x, w, None, EPS, y2)
    n = F.layer_norm_workspace_len(rows, cols)
    guard = [torch.full((rows * cols + 8,), 3.0, dtype=x.dtype, device=DEV)] + \
        [torch.full((cols + 8,), 3.0, device=DEV) for _ in range(2)] + [torch.full((n + 8,), 3.0, device=DEV)]
    dx2, dw2, db2, ws = guard[0][:-8].view(rows, cols), guard[1][:-8], guard[2][:-8], guard[3][:-8]
    for kw in ({"dx": dx2}, {"dw": dw2, "ws": ws}, {"db": db2, "ws": ws}):
        F.layer_norm_bwd(dy, x, w, mean, rstd, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    for g in guard:
        assert (g[-8:] == 3).all()
    again = run(x, w, None, dy, False, pdtype=torch.float32)
    for a, b in zip((y, dx, dw, db), (again[0], again[4], again[5], again[6])):
        assert torch.equal(a, b)


def test_no_rows():
    x, w = torch.empty(0, 40, device=DEV), torch.ones(40, device=DEV)
    _, _, _, _, _, dw, db = run(x, w, w, x, True)
    assert (dw == 0).all() and (db == 0).all()


def test_unaligned_rows():
    """Rows aligned to their element only, and a tensor that starts off 16 bytes."""
    for cols in (64, 1000, 4096):
        buf = rand((10 * cols + 1,), "bf16", 1)
        x, dy = buf[1:].view(10, cols), rand((10 * cols + 3,), "bf16", 2)[3:].view(10, cols)
        w = rand((cols + 1,), "f32", 3)[1:]
        check_all(x, w, None, dy, True, pdtype=torch.float32)


def test_gradients_against_differences():
    """The formula's gradients are the slope of the formula (64 bits)."""
    rng = np.random.default_rng(0)
    x, dy, w, b = rng.normal(size=(3, 11)), rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=11)
    (dx, _), (dw, _), (db, _) = R.LayerNorm(x, w, b, EPS).grads(dy, x)

    def loss(x, w, b):
        return (R.LayerNorm(x, w, b, EPS).y * dy).sum()
    h = 1e-6
    for name, p, grad in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        for i in np.ndindex(p.shape):
            args = {"x": x, "w": w, "b": b}
            hi, lo = p.copy(), p.copy()
            hi[i] += h
            lo[i] -= h
            slope = (loss(**{**args, name: hi}) - loss(**{**args, name: lo})) / (2 * h)
            assert abs(slope - grad[i]) < 1e-7


def test_captured_step():
    rows, cols = 64, 512
    x, dy = rand((rows, cols), "bf16", 1), rand((rows, cols), "bf16", 2)
    w, b = rand((cols,), "f32", 3), rand((cols,), "f32", 4)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    c, ws = F.Act8(rows, cols), torch.empty(F.layer_norm_workspace_len(rows, cols), device=DEV)

    def step():
        F.layer_norm_fwd(x, w, b, EPS, y, mean, rstd, c)
        F.layer_norm_bwd(dy, c, w, mean, rstd, dx, dw, db, ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(rand((rows, cols), "bf16", 10 + i))
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (y, dx, dw, db)]
        for t in (y, dx, dw, db):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip((y, dx, dw, db), eager):
            assert torch.equal(a, e)
