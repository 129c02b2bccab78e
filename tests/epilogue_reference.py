"""A product's epilogue, its backward step and dropout from their definitions, in
64 bits on the CPU, with the error bounds that the GPU tests hold the kernels to.
Written apart from the kernels."""
import math

import numpy as np
from scipy.special import erfc

U32 = 2.0 ** -24  # half a step of fp32, relative
NONE, RELU, SILU, GELU, GELU_TANH = range(5)
ACTS = (NONE, RELU, SILU, GELU, GELU_TANH)


def philox(counter, key, rounds=10):
    """Philox 4x32: counter [..., 4] and key [2] of 32-bit words (uint64 arrays)."""
    m32 = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & m32]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return np.stack(c, axis=-1)


def keep(rng, rows, cols, p):
    """The factor of each element: 0 or 65536 / (65536 - t)."""
    t = int(65536 * float(np.float32(p)) + 0.5)
    if t == 0:
        return np.ones((rows, cols))
    g = -(-cols // 8)
    n = np.arange(rows * g, dtype=np.uint64)
    seed, off = (int(v) % 2 ** 64 for v in rng)
    m = 0xFFFFFFFF
    ctr = np.stack([n & np.uint64(m), n >> np.uint64(32), np.full_like(n, off & m), np.full_like(n, off >> 32)], axis=-1)
    w = philox(ctr, (seed & m, seed >> 32))
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], axis=-1).reshape(rows, 8 * g)[:, :cols]
    return np.where(u >= t, 65536 / (65536 - t) if t < 65536 else 0.0, 0.0)


def _sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def _tanh_arg(h):
    return 2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)


def act(h, a):
    """act(h); at -inf the limit."""
    with np.errstate(invalid="ignore", over="ignore"):
        if a == RELU:
            y = np.where(h <= 0, 0.0, h)
        elif a == SILU:
            y = h * _sigmoid(h)
        elif a == GELU:
            y = h * erfc(-h / math.sqrt(2)) / 2
        elif a == GELU_TANH:
            y = h * _sigmoid(_tanh_arg(h))
        else:
            return h
    return np.where(h == -np.inf, 0.0, y)


def slope(h, a):
    """act'(h); at an infinity the limit."""
    h = np.clip(h, -200, 200)
    if a == RELU:
        return np.where(h <= 0, 0.0, 1.0)
    if a == SILU:
        s = _sigmoid(h)
        return s + h * s * _sigmoid(-h)
    if a == GELU:
        return erfc(-h / math.sqrt(2)) / 2 + h * np.exp(-h * h / 2) / math.sqrt(2 * math.pi)
    if a == GELU_TANH:
        s = _sigmoid(_tanh_arg(h))
        return s + h * s * _sigmoid(-_tanh_arg(h)) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * h * h)
    return np.ones_like(h)


def _rel(h, a, fast):
    """Relative error of the part of act(h) and act'(h) that goes to 0 with h's
    exponential: its argument x carries 2 |x| roundings of half a step (the product
    and the constant; `fast`: log2 e in one part) or about one, its own step 2; then a
    reciprocal and up to 8 products and sums.  gelu: the series' fit, and Horner's
    rule over terms whose magnitudes add up to twice its value (9 terms, 2 roundings
    each)."""
    h = np.clip(np.abs(h), 0, 200)
    x = {SILU: h, GELU: h * h / 2, GELU_TANH: np.abs(_tanh_arg(h))}.get(a, 0 * h)
    base = (2 * x if fast else 1.0) + 16
    if a == GELU:
        base = base + (x if fast else 0.0) + 36
        return base * U32 + (8.7e-6 if fast else 4e-8)
    if a == GELU_TANH:
        base = base + 6 * x  # the argument's own roundings: two constants, four operations
    return base * U32


TINY = 2.0 ** -126  # an exponential below this may be flushed


def act_err(h, a, fast):
    if a in (NONE, RELU):
        return np.zeros_like(h)
    y = act(h, a)
    # gelu of a positive h is h minus the tail's part
    with np.errstate(invalid="ignore"):
        part = np.where(h > 0, h - y, np.abs(y)) if a == GELU else np.abs(y)
    part = np.where(np.isfinite(part), part, 0.0)
    h = np.where(np.isfinite(h), np.abs(h), 0.0)
    return part * _rel(h, a, fast) + 2 * U32 * np.where(np.isfinite(y), np.abs(y), 0.0) + (1 + h) * TINY


def slope_err(h, a, fast):
    if a in (NONE, RELU):
        return np.zeros_like(h)
    h = np.clip(h, -200, 200)
    d = 1.0
    if a == GELU:
        size = erfc(np.abs(h) / math.sqrt(2)) / 2 + np.abs(h) * np.exp(-h * h / 2) * 0.4
    else:
        s = _sigmoid(h if a == SILU else _tanh_arg(h))
        d = 1.0 if a == SILU else 1.6 * (1 + 0.135 * h * h)
        size = s * (1 + np.abs(h) * (1 - s) * d)
    # A flushed exponential e < TINY takes s (1 + h (1 - s) d') with it, s <= e: that is
    # up to e (1 + |h| d), d' = 2 sqrt(2 / pi) (1 + 3 0.044715 h^2) <= d for gelu_tanh.
    return 2 * size * _rel(h, a, fast) + 2 * U32 * np.abs(slope(h, a)) + (1 + np.abs(h) * d) * TINY


def forward(prod, prod_err, bias, a, residual, factor, fast):
    """(h, its bound, y, its bound) of a product with bound prod_err.  No activation's
    slope exceeds 1.2.  A factor of 0 gives 0 whatever it meets."""
    b = 0.0 if bias is None else bias
    with np.errstate(invalid="ignore"):
        h = prod + b
        h_err = prod_err + U32 * np.where(np.isfinite(h), np.abs(h), 0.0)
        v = act(h, a)
        v_err = 1.2 * h_err + act_err(h, a, fast)
        y = np.where(factor == 0, 0.0, v * factor)
        size = np.where(np.isfinite(y), np.abs(y), 0.0)
        y_err = np.where(factor == 0, 0.0, v_err * factor + 3 * U32 * size)
        if residual is not None:
            y = y + residual
            y_err = y_err + U32 * np.where(np.isfinite(y), np.abs(y), 0.0)
    y_err = np.where(np.isfinite(y_err), y_err, 0.0)
    return h, h_err, y, y_err


def backward(gy, h, a, factor, fast):
    """(gh, its bound, gb, its bound); a column's fp32 sum of n terms adds at most n
    times."""
    with np.errstate(invalid="ignore"):
        s = slope(h, a) if a != NONE else 1.0
        gh = np.where(factor == 0, 0.0, gy * factor * s)
        e = slope_err(h, a, fast) if a != NONE else 0.0
        err = np.where(factor == 0, 0.0, np.abs(gy) * factor * e + 4 * U32 * np.abs(gh) + 2.0 ** -148)
    return gh, err, gh.sum(axis=0), err.sum(axis=0) + gy.shape[0] * U32 * np.abs(gh).sum(axis=0)
