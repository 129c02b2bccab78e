"""The microscaled formats, the gated activation and the layer norm from their
definitions, in 64 bits on the CPU, and the error bounds that the GPU tests
hold the kernels to.  Written apart from the kernels: codes are found by
comparing against the list of representable magnitudes."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U32 = 2.0 ** -24  # half a step of fp32, relative
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f64(t):
    return t.detach().to("cpu").double().numpy()


def _nearest(a, mags):
    """Index of the magnitude nearest to a (a <= mags[-1]); ties to the even index."""
    hi = np.minimum(np.searchsorted(mags, a), len(mags) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = mags[hi] - a, a - mags[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def _scales(blocks, largest, emax, fit):
    """Exponent of each block (last axis) and whether it holds an inf or a NaN."""
    bad = ~np.isfinite(blocks).all(axis=-1)
    amax = np.abs(np.where(bad[..., None], 0.0, blocks)).max(axis=-1)
    m, ex = np.frexp(amax)  # amax = m 2^ex, m in [1/2, 1)
    e = ex - 1 - emax
    if fit:
        e = np.minimum(np.where(amax > largest * 2.0 ** e, e + 1, e), 127 - emax)
    return np.maximum(np.where(amax > 0, e, -127), -127), bad


def _blocks(x):
    rows, cols = x.shape
    n = -(-cols // 32)
    v = np.zeros((rows, 32 * n))
    v[:, :cols] = x
    return v.reshape(rows, n, 32)


def fp4(x, fit):
    """(codes [rows, n, 32], scale bytes [rows, n]) of x's rows."""
    v = _blocks(x)
    e, bad = _scales(v, 6.0, 2, fit)
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(v / 2.0 ** e[..., None]), 6.0)
    codes = _nearest(np.where(bad[..., None], 0.0, a), E2M1) | (np.signbit(v) * 8)
    return np.where(bad[..., None], 0, codes), np.where(bad, 255, e + 127)


def fp4_values(x, fit):
    c, s = fp4(x, fit)
    return fp4_decode(c, s)[:, :x.shape[1]]


def fp4_decode(codes, s):
    p = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7] * p[..., None]
    return v.reshape(codes.shape[0], -1)


def fp4_unpack(m):
    """(codes [rows, 8 nk, 32], scale bytes [rows, 8 nk]) of an Mxfp4's buffers, by
    the layout the C header states."""
    rows, k = m.rows, m.k
    nk = -(-k // 256)
    q = m.q.cpu().numpy().reshape(rows, 128 * nk)
    codes = np.stack([q & 15, q >> 4], axis=-1).reshape(rows, 8 * nk, 32).astype(np.int64)
    s = m.s.cpu().numpy()
    r, b = np.meshgrid(np.arange(rows), np.arange(8 * nk), indexing="ij")
    at = (r // 32 * nk + b // 8) * 256 + ((b % 8) // 2 * 16 + r % 16) * 4 + (r % 32) // 16 * 2 + b % 2
    return codes, s[at].astype(np.int64)


def _e4m3_mags():
    m = [i * 2.0 ** -9 for i in range(8)]
    m += [(1 + i / 8) * 2.0 ** e for e in range(-6, 9) for i in range(8)]
    return np.array(m[:-1])  # the last one is NaN's code


E4M3 = _e4m3_mags()


def act8(x):
    """(codes, scale bytes) of x's rows."""
    v = _blocks(x)
    e, bad = _scales(v, 448.0, 8, True)
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(v / 2.0 ** e[..., None]), 448.0)
    codes = _nearest(np.where(bad[..., None], 0.0, a), E4M3) | (np.signbit(v) * 128)
    return np.where(bad[..., None], 0, codes), np.where(bad, 255, e + 127)


def act8_values(x):
    c, s = act8(x)
    p = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    v = np.where(c & 128, -1.0, 1.0) * E4M3[c & 127] * p[..., None]
    return v.reshape(x.shape[0], -1)[:, :x.shape[1]]


def check(got, want, bound, what):
    """|got - want| <= bound + half a step of got's dtype at the largest value the
    bound allows; NaN where want has NaN."""
    fi = torch.finfo(got.dtype)
    g = f64(got).reshape(want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN in {np.isnan(g).sum()} places, expected {nan.sum()}"
    bound = np.broadcast_to(np.asarray(bound, dtype=np.float64), want.shape)
    tol = bound + (np.abs(want) + bound) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2
    off = np.where(nan, -1.0, np.abs(g - want) - tol)
    if off.size and off.max() > 0:
        i = np.unravel_index(np.argmax(off), off.shape)
        raise AssertionError(f"{what}: {(off > 0).sum()} of {off.size} beyond the bound; at {i} got {g[i]!r}, "
                             f"expected {want[i]!r} +- {tol[i]!r}")


def dot(a, b):
    """a b^T in 64 bits and the bound of an fp32 sum of its exact products in any
    order: at most k additions, each off by a step (matrix cores may cut where
    they align) of a partial sum that sum|a b| bounds, and by the smallest
    subnormal."""
    k = a.shape[1]
    with np.errstate(invalid="ignore"):
        return a @ b.T, 2 * k * U32 * (np.abs(a) @ np.abs(b).T) + (k + 1) * 2.0 ** -149


def swiglu(g, u):
    """silu(g) u and its bound: exp2(-g log2 e) has the rounding of the product and
    of the constant (|g| U32 each) and the instruction's own step (2 U32); then
    an addition, a division and two products, half a step each.  Below 2^-126
    the exponential's reciprocal may be flushed."""
    s = 1 / (1 + np.exp(-g))
    a = g * s * u
    return a, (2 * np.abs(g) + 8) * U32 * np.abs(a) + np.abs(g * u) * 2.0 ** -126


def swiglu_grad(da, g, u):
    """(dg, du) and their bounds; dg's factor 1 + g (1 - s) may cancel, so its
    error counts against 1 + |g|."""
    s = 1 / (1 + np.exp(-g))
    rel = (2 * np.abs(g) + 12) * U32
    dg, du = da * u * s * (1 + g * (1 - s)), da * g * s
    tiny = np.abs(da) * (1 + np.abs(g)) * 2.0 ** -126 + 2.0 ** -148
    return (dg, 2 * rel * np.abs(da * u) * s * (1 + np.abs(g)) + np.abs(u) * tiny + tiny), (du, rel * np.abs(du) + tiny)


class LayerNorm:
    """y and the statistics of rows of x, with bounds.  A sum of n terms adds along
    chains of at most n / 64 + 24 (a wave's lanes, then a tree)."""

    def __init__(self, x, w, b, eps):
        n = x.shape[1]
        self.depth = d = n / 64 + 24
        self.w = np.ones(n) if w is None else w
        self.b = np.zeros(n) if b is None else b
        self.mean = x.mean(axis=1, keepdims=True)
        c = x - self.mean
        var = (c * c).mean(axis=1, keepdims=True)
        self.rstd = 1 / np.sqrt(var + eps)
        self.mean_err = (d + 2) * U32 * np.abs(x).mean(axis=1, keepdims=True) + 2.0 ** -149
        var_err = (d + 6) * U32 * var + 2 * self.mean_err * np.abs(c).mean(axis=1, keepdims=True) + self.mean_err ** 2
        self.rstd_rel = 0.5 * var_err / (var + eps) + 4 * U32
        self.y = c * self.rstd * self.w + self.b
        self.y_err = (np.abs(self.w) * self.rstd * (self.mean_err + np.abs(c) * (self.rstd_rel + 6 * U32)) +
                      2 * U32 * (np.abs(self.y) + np.abs(self.b)))

    def grads(self, dy, x):
        """((dx, bound), (dw, bound), (db, bound)) with x the input or its checkpoint's
        values.  dw and db add along at most `rows` terms."""
        d, rows = self.depth, dy.shape[0]
        xh = (x - self.mean) * self.rstd
        xh_err = self.rstd * self.mean_err + np.abs(xh) * (self.rstd_rel + 3 * U32)
        q = dy * self.w
        c1, c2 = q.mean(axis=1, keepdims=True), (q * xh).mean(axis=1, keepdims=True)
        c1_err = (d + 3) * U32 * np.abs(q).mean(axis=1, keepdims=True)
        c2_err = ((d + 4) * U32 * np.abs(q * xh) + np.abs(q) * xh_err).mean(axis=1, keepdims=True)
        dx = self.rstd * (q - c1 - xh * c2)
        parts = np.abs(q) + np.abs(c1) + np.abs(xh * c2)
        dx_err = self.rstd * (parts * (self.rstd_rel + 6 * U32) + c1_err + np.abs(xh) * c2_err + np.abs(c2) * xh_err)
        dw, db = (dy * xh).sum(axis=0), dy.sum(axis=0)
        dw_err = ((rows + 2) * U32 * np.abs(dy * xh) + np.abs(dy) * xh_err).sum(axis=0)
        db_err = rows * U32 * np.abs(dy).sum(axis=0)
        return (dx, dx_err), (dw, dw_err), (db, db_err)
