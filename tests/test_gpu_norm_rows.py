"""Layer norm where its statistics are delicate: rows of one value, means far
from zero."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests import mx_reference as R
from tests.test_gpu_layer_norm import rand, run

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5
# one, four, eight and sixteen waves a row, one and two groups a lane, rows past the registers
COLS = [7, 100, 511, 700, 1000, 1500, 4001, 8100, 14333, 14336, 16640, 40001]


def forward(x, w=None, b=None, ckpt=None):
    rows, cols = x.shape
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    F.layer_norm_fwd(x, w, b, EPS, y, mean, rstd, ckpt)
    return y, mean, rstd


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_rows_of_one_value(cols, dtype):
    """Their variance is 0 and their deviations are 0, so the result is b, the
    mean that value and dx what is left of dy w without its mean.  The fp32 sum
    of the row may round (1000.1 times 14333), its mean may not."""
    t = R.DTYPES[dtype]
    values = torch.tensor([1000.0, 1000.1, -0.1, 3.0e4 / 7, 1 / 3, 2.0 ** -20, 0.0, 5.0]).to(t)
    x = values[:, None].expand(-1, cols).contiguous().to(DEV)
    w = torch.linspace(-2, 2, cols, device=DEV).to(t)
    b = torch.linspace(3, 5, cols, device=DEV).to(t)
    y, mean, rstd = forward(x, w, b, F.Act8(*x.shape))
    dx = torch.empty_like(x)
    F.layer_norm_bwd(torch.ones_like(x), x, None, mean, rstd, dx=dx)
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand_as(y))
    assert torch.equal(mean.cpu(), values.float())
    # dy = 1, w = 1: 1 - mean(1), with xh = 0
    assert not bool(dx.any())


@pytest.mark.parametrize("cols", COLS)
def test_a_mean_far_from_zero(cols):
    """Deviations of 1 around 5000, each within a few steps of its own size, not of
    the mean's (2^-11).  x and the first mean are multiples of 2^-11, so the
    deviations from it are exact, and below 8: the sum's error shifts them by
    depth U32 5000 < 0.1.  With depth = n / 64 + 24 additions in a chain, the mean's
    correction is then off by (depth + 2) U32 8, the variance by (depth + 4) U32
    (1 + 0.1^2) of itself and by 2 * 0.1 times the correction's error, so rstd by less
    than (2 depth + 8) U32 of itself; the result takes four more roundings."""
    g = torch.Generator().manual_seed(cols)
    # multiples of 2^-11 around 5000 are exact, and so are their deviations from any fp32 mean near them
    x = 5000 + (torch.randn(20, cols, generator=g) * 2048).round() / 2048
    x = x.to(DEV)
    y, mean, rstd = forward(x)
    torch.cuda.synchronize()
    v = R.f64(x)
    m = v.mean(axis=1, keepdims=True)
    c = v - m
    var = (c * c).mean(axis=1, keepdims=True)
    want = c / np.sqrt(var + EPS)
    depth = cols / 64 + 24
    mean_err = (depth + 2) * R.U32 * 8.0  # of the corrected mean, before it is rounded for the backward
    rel = (2 * depth + 8) * R.U32
    bound = (mean_err + np.abs(c) * rel) / np.sqrt(var + EPS) + 4 * R.U32 * np.abs(want)
    R.check(y, want, bound, "y")
    R.check(mean, m[:, 0], mean_err, "mean")
    R.check(rstd, 1 / np.sqrt(var + EPS)[:, 0], rel / np.sqrt(var + EPS)[:, 0], "rstd")


UNEVEN = [(1100, 4090), (1300, 8100), (700, 14333), (17000, 2000), (5000, 700), (20001, 300)]


@pytest.mark.parametrize("rows,cols,dtype,pdtype,ckpt", [(*s, *t, False) for s in UNEVEN
                                                         for t in (("bf16", "f32"), ("f16", "f16"), ("f32", "f32"))] +
                         [(*s, *t, True) for s, t in zip(UNEVEN, [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")] * 2)])
def test_several_rows_a_block(rows, cols, dtype, pdtype, ckpt):
    """More rows than blocks, unevenly: statistics of one row after the other in the
    same block, loads ahead across rows, and hundreds of partial rows of dw and db.
    The bounds on dw and db are those of the sums' own chains (long ones would
    hide a missing part)."""
    x, dy = rand((rows, cols), dtype, 1, 2.0, 0.5), rand((rows, cols), dtype, 2, 0.1)
    w, b = rand((cols,), pdtype, 3, 0.2, 1.0), rand((cols,), pdtype, 4, 0.2)
    y, mean, rstd, c, dx, dw, db = run(x, w, b, dy, ckpt, pdtype=R.DTYPES[pdtype])
    chain = chain_of(rows, cols)
    assert chain < rows / 20
    wsum = None
    for lo in range(0, rows, 2500):  # (in pieces: 64-bit copies of the whole take long)
        at = slice(lo, min(lo + 2500, rows))
        ref = R.LayerNorm(R.f64(x[at]), R.f64(w), R.f64(b), EPS)
        R.check(y[at], ref.y, ref.y_err, "y")
        R.check(mean[at], ref.mean[:, 0], ref.mean_err[:, 0], "mean")
        R.check(rstd[at], ref.rstd[:, 0], (ref.rstd * ref.rstd_rel)[:, 0], "rstd")
        xv, vdy = R.f64(x[at]), R.f64(dy[at])
        if ckpt:
            codes, s = R.act8(xv)
            assert np.array_equal(c.s[at].cpu().numpy().astype(np.int64), s)
            assert np.array_equal(c.q[at].cpu().numpy().astype(np.int64).reshape(codes.shape), codes)
            xv = R.act8_values(xv)
        (want, bound), _, _ = ref.grads(vdy, xv)
        R.check(dx[at], want, bound, "dx")
        xh = (xv - ref.mean) * ref.rstd
        xh_err = ref.rstd * ref.mean_err + np.abs(xh) * (ref.rstd_rel + 3 * R.U32)
        sums = np.stack([(vdy * xh).sum(0), np.abs(vdy * xh).sum(0), (np.abs(vdy) * xh_err).sum(0), vdy.sum(0), np.abs(vdy).sum(0)])
        wsum = sums if wsum is None else wsum + sums
    R.check(dw, wsum[0], chain * R.U32 * wsum[1] + wsum[2], "dw")
    R.check(db, wsum[3], chain * R.U32 * wsum[4], "db")
    assert (np.abs(wsum[3]) > 10 * chain * R.U32 * wsum[4]).mean() > 0.9  # (the bounds tell db from 0)


def chain_of(rows, cols):
    """Additions in a chain behind an element of dw or db: a wave's rows, four waves
    of a block, every 32nd part (eight at a time), a tree of 32, and the product.
    A block has rows / parts of them or one more; where a row takes one wave, it
    has four rows at a time."""
    parts = F.layer_norm_workspace_len(rows, cols) // (2 * cols)
    return -(-rows // parts) + 4 + -(-parts // 32) + 8 + 5 + 2


@pytest.mark.parametrize("rows,cols", [(1500, 2048), (2048, 4096), (5000, 1024), (2100, 5000), (30000, 40), (600, 20000),
                                       (2200000, 1024), (130000, 16640)])
def test_parts_add_up(rows, cols):
    """db of whole numbers is exact whatever the order, every partial row in it (up
    to 512); dw likewise where xh is made whole: mean 0 and rstd 1 handed in."""
    g = torch.Generator(DEV).manual_seed(rows)
    x, dy = (torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sums = torch.zeros(2, cols, dtype=torch.int64, device=DEV)
    for r in range(0, rows, 1 << 14):
        at = slice(r, min(r + (1 << 14), rows))
        n = at.stop - r
        vx = torch.randint(-2, 3, (n, cols), generator=g, device=DEV, dtype=torch.int32)
        vdy = torch.randint(-2, 4, (n, cols), generator=g, device=DEV, dtype=torch.int32)  # (not balanced: db grows)
        x[at], dy[at] = vx, vdy
        sums[0] += (vx * vdy).sum(0)
        sums[1] += vdy.sum(0)
    assert 6 * rows < 1 << 24  # every partial sum is a whole number below 2^24
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    n = F.layer_norm_workspace_len(rows, cols)
    ws = torch.full((n,), float("nan"), device=DEV)
    F.layer_norm_bwd(dy, x, None, mean, rstd, dw=dw, db=db, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(db.long(), sums[1]) and torch.equal(dw.long(), sums[0])
    assert torch.equal(db, db.round()) and torch.equal(dw, dw.round())
    del x, dy
    torch.cuda.empty_cache()
