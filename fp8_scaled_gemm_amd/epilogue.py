"""Binding of the products with an epilogue (bias, activation, dropout, residual),
their backward pass and dropout: include/fp8sg.h's entry points of the same names,
on the current torch stream.  Its names are those of the package
(`import fp8_scaled_gemm_amd as F; F.fp8_scaled_linear_fwd_epilogue(...)`).

Argument marshalling only, as in the package itself: every buffer's dtype, shape,
strides and device are checked here, before the library is called.

The epilogue's arguments, by keyword in every call:
  bias      N values, of the input's dtype or float32, or None
  act       ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU or ACT_GELU_TANH
  residual  M x N of the output's dtype, or None; its rows may be apart, and it may
            be the output itself
  pre       receives h = product + bias for the backward pass (M x N of the output's
            dtype), or None
  p, rng    dropout's probability, in steps of 2^-16, and the two int64 words in
            device memory that its generator starts from (None where p is 0)
The output and pre may lie over a linear's x or w (with the residual the output
itself too: a residual stream updated in place), over no other buffer of a call.
"""
import ctypes
import struct

import torch

from . import LinearBwdWs, LinearSaved, _check, _need, _need_2d, lib
from .mx import (_TYPE, MX_FLOOR, Mxfp4, Mxfp4LinearSaved, Mxfp4LinearWs, _apart, _bytes, _here, _linear, _matrix,
                 _need_codes, _ptr, _rows, _rule, _same, _stream, _type)

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = range(5)


# fp8sg_epilogue, packed anew for each call: bias, residual, pre, rng, ld_residual,
# ld_out, p, act, bias_type
_pack = struct.Struct("=4Q2qfii4x").pack
_SIZE = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4}


def bind(L):
    """Argument types of this module's entry points."""
    P, i64, i, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.fp8_gemm_epilogue.argtypes = L.fp8_gemm_rowwise_epilogue.argtypes = [P, P, P, P, P, P, i, i64, i64, i64, P]
    L.fp8_scaled_linear_fwd_epilogue.argtypes = [P, P, i, i64, i64, i64, P, P, P, i, P]
    L.fp8_scaled_linear_bwd_epilogue.argtypes = [P, i, P, i64, i64, i64, P, P, P, P, P, i64, P, P, i, P]
    L.epilogue_workspace_len.argtypes = [i64, i64]
    L.epilogue_workspace_len.restype = i64
    L.epilogue_bwd.argtypes = [P, i, P, i64, i64, P, P, P, i64, P]
    L.mxfp4_gemm_epilogue.argtypes = [P, P, P, P, i, i64, i64, i64, P]
    L.mxfp4_linear_fwd_epilogue.argtypes = [P, P, i, i64, i64, i64, i, P, P, P, P, i, P]
    L.mxfp4_linear_apply_epilogue.argtypes = [P, i, P, i64, i64, i64, i, P, P, P, i, P]
    L.mxfp4_linear_bwd_epilogue.argtypes = [P, i, i64, i64, i64, i, P, P, P, P, P, P, i64, P, P, i, P]
    L.dropout_fwd.argtypes = [P, i64, P, i64, i, i64, i64, f32, P, P, i64, P]
    L.dropout_bwd.argtypes = [P, i64, i, i64, i64, f32, P, P, i64, P]


def _row_stride(t, name, dtype, shape, rows, cols):
    """Row distance of a matrix of contiguous rows; beyond two dimensions it is contiguous."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return cols
    except AttributeError:
        pass
    _type(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return cols
    if t.dim() != 2 or (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return t.stride(0) if rows > 1 else cols


def _span(t):
    """First and last byte address + 1 of what a tensor's elements lie in."""
    at = t.data_ptr()
    if t.is_contiguous():
        return at, at + t.nbytes
    return at, at + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _clear(a, name_a, b, name_b):
    """Two tensors that do not share memory (their spans, or column ranges of one matrix)."""
    if a is None or b is None or not a.numel() or not b.numel():
        return
    (a0, a1), (b0, b1) = _span(a), _span(b)
    if a1 <= b0 or b1 <= a0:
        return
    if a.element_size() == b.element_size() and a.shape == b.shape and a.dim() == 2:
        return _apart(a, name_a, a.stride(0), b, name_b, b.stride(0))
    raise ValueError(f"{name_a} and {name_b} overlap")


def _all_clear(outputs, inputs):
    """No output shares memory with another output or with an input; each is a
    (tensor or None, name)."""
    for i, (t, name) in enumerate(outputs):
        for u, other in outputs[i + 1:] + inputs:
            _clear(t, name, u, other)


def _off_codes(C, pre, *codes):
    """C and pre lie over none of a product's operands, which it reads as it stores."""
    for t, name in ((C, "C"), (pre, "pre")):
        if t is not None and t.numel():
            a0, a1 = _span(t)
            for q in codes:
                if q.numel() and a0 < q.data_ptr() + q.nbytes and q.data_ptr() < a1:
                    raise ValueError(f"{name} and an operand overlap")


def _drop(p, rng):
    """Address of rng (0: nothing is dropped), whose device _here checks."""
    if rng is None:
        if p and not 0.0 <= p < 2.0 ** -17:
            if not 0.0 <= p <= 1.0:
                raise ValueError(f"p: {p} is not a probability")
            raise ValueError("rng is needed where p is not 0")
        return 0
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p: {p} is not a probability")
    if rng.__class__ is not torch.Tensor or rng.dtype is not torch.int64 or rng.numel() != 2 or not rng.is_contiguous():
        _need(rng, "rng", torch.int64, numel=2)
    return rng.data_ptr()


def _act(act):
    if act.__class__ is not int or not 0 <= act <= 4:
        raise ValueError(f"act must be one of ACT_NONE .. ACT_GELU_TANH, not {act!r}")
    return act


def _epilogue(y, shape, M, N, in_dtype, bias, act, residual, pre, p, rng, *others, clear=()):
    """The packed struct of a forward epilogue.  in_dtype: the linear's input's, or
    None.  others: the call's other tensors, for their device.  clear: those that
    neither y nor pre may lie over."""
    dt = y.dtype
    ldy = N if y.shape == shape and y.is_contiguous() else _row_stride(y, "y", dt, shape, M, N)
    at = y.data_ptr()
    end = at + (M * ldy if M else 0) * _SIZE[dt]  # (or a little past the last row)
    pb = pr = pp = bt = ldr = 0
    near = False  # whether an output comes near another tensor: looked at more closely then
    if bias is not None:
        bt = _TYPE.get(bias.dtype) if isinstance(bias, torch.Tensor) else None
        if bt is None:
            _type(bias, "bias")  # (says what it is)
        if in_dtype is not None and bt != 2 and bias.dtype is not in_dtype:
            raise TypeError(f"bias: dtype {bias.dtype}, expected {in_dtype} or float32")
        if bias.shape != (N,) or not bias.is_contiguous():
            _need(bias, "bias", None, shape=(N,))
        pb = bias.data_ptr()
        near = at < pb + 4 * N and pb < end
    if residual is not None:
        ldr = _row_stride(residual, "residual", dt, shape, M, N)
        pr = residual.data_ptr()
        if pr == at and ldr == ldy:  # the output itself is allowed
            residual = y
        elif at < pr + M * ldr * _SIZE[dt] and pr < end:
            near = True
    if pre is not None:
        _same(pre, "pre", dt, shape)
        pp = pre.data_ptr()
        pe = pp + M * N * _SIZE[dt]
        if (at < pe and pp < end) or (pb and pb < pe and pp < pb + 4 * N) or \
                (pr and pr < pe and pp < pr + M * ldr * _SIZE[dt]):
            near = True
    if near:
        _all_clear([(y, "y"), (pre, "pre")], [(bias, "bias"), (residual if residual is not y else None, "residual")])
        if residual is y:
            _clear(pre, "pre", y, "residual")
    if clear:
        _off_codes(y, pre, *clear)
    e = _pack(pb, pr, pp, _drop(p, rng) if rng is not None or p else 0, ldr, ldy, p, _act(act), bt)
    _here(y, bias, residual, pre, rng, *others)
    return e


def _backward(gy, gh, gb, pre, act, p, rng, part, M, N, alone, *out):
    """The packed struct of a backward step, and the workspace's length.  out: the
    call's other outputs, (tensor or None, name)."""
    dt, shape = gy.dtype, gy.shape
    size = M * N * _SIZE[dt]
    pg, n, bt, pp = gy.data_ptr(), 0, 0, 0
    words = _drop(p, rng)
    changes = _act(act) != ACT_NONE or p >= 2.0 ** -17
    spans, outputs, inputs = [(pg, pg + size)], [], [(gy, "gy")]
    if gh is not None:
        _same(gh, "gh", dt, shape)
        at = gh.data_ptr()
        if at != pg:  # (gy itself is allowed)
            spans.append((at, at + size))
            outputs.append((gh, "gh"))
    elif changes and not alone:
        raise ValueError("gh is needed where the epilogue has an activation or drops")
    if act != ACT_NONE:
        if pre is None:
            raise ValueError("pre is needed where the epilogue has an activation")
        _same(pre, "pre", dt, shape)
        pp = pre.data_ptr()
        if pp != pg or gh is not None and gh.data_ptr() == pg:
            spans.append((pp, pp + size))
        inputs.append((pre, "pre"))
    else:
        pre = None
    if gb is not None:
        gd = gb.dtype if isinstance(gb, torch.Tensor) else _type(gb, "gb")
        if gd is not dt and gd is not torch.float32:
            raise TypeError(f"gb: dtype {gd}, expected {dt} or float32")
        _same(gb, "gb", gd, (N,))
        at, bt = gb.data_ptr(), _TYPE[gd]
        spans.append((at, at + N * _SIZE[gd]))
        outputs.append((gb, "gb"))
        if part is not None:
            if part.__class__ is not torch.Tensor or part.dtype is not torch.float32 or not part.is_contiguous():
                _need(part, "part", torch.float32)
            n, at = part.numel(), part.data_ptr()
            spans.append((at, at + 4 * n))
            outputs.append((part, "part"))
    else:
        part = None
    for t, name in out:
        if t is not None:
            at = t.data_ptr()
            spans.append((at, at + t.nbytes))
            outputs.append((t, name))
    spans.sort()
    at = 0
    for lo, hi in spans:
        if lo < at:  # two come near each other: looked at more closely
            if gh is not None and gh.data_ptr() == pg:
                inputs[0] = (None, "gy")
                outputs.append((gh, "gh"))
            _all_clear(outputs, inputs)
            break
        at = hi
    _here(gy, gh, gb, pre, part, rng)
    return _pack(0, 0, pp, words, 0, 0, p, act, bt), n


def _lead(shape, n):
    return shape[:-1] + (n,)


# ------------------------------------------------------------------------- FP8

def _fp8_gemm(fn, A, B, ia, ib, C, bias, act, residual, pre, p, rng, stream):
    M, K = _need_2d(A, "A")
    N, _ = _need_2d(B, "B")
    _need(A, "A", torch.uint8)
    _need(B, "B", torch.uint8, shape=(N, K))
    ct = _type(C, "C")
    e = _epilogue(C, (M, N), M, N, None, bias, act, residual, pre, p, rng, A, B, clear=(A, B))
    _check(getattr(lib(), fn)(_ptr(A), _ptr(B), ia, ib, e, _ptr(C), ct, M, N, K, _stream(stream)), fn)


def fp8_gemm_epilogue(A: torch.Tensor, B: torch.Tensor, inv_a_ptr: int, inv_b_ptr: int, C: torch.Tensor, *, bias=None,
                      act: int = ACT_NONE, residual=None, pre=None, p: float = 0.0, rng=None, stream=None):
    """C[M,N] = residual + drop(act(A[M,K] B[N,K]^T * fl32(inv_a * inv_b) + bias)) of
    e4m3 codes; inv_*_ptr are device double addresses."""
    _fp8_gemm("fp8_gemm_epilogue", A, B, inv_a_ptr, inv_b_ptr, C, bias, act, residual, pre, p, rng, stream)


def fp8_gemm_rowwise_epilogue(A: torch.Tensor, B: torch.Tensor, inv_a: torch.Tensor, inv_b: torch.Tensor,
                              C: torch.Tensor, *, bias=None, act: int = ACT_NONE, residual=None, pre=None,
                              p: float = 0.0, rng=None, stream=None):
    """The same with an inverse scale for each row of A and of B (float64 vectors)."""
    _need(inv_a, "inv_a", torch.float64, numel=_need_2d(A, "A")[0])
    _need(inv_b, "inv_b", torch.float64, numel=_need_2d(B, "B")[0])
    _here(inv_a, inv_b)
    _fp8_gemm("fp8_gemm_rowwise_epilogue", A, B, inv_a.data_ptr(), inv_b.data_ptr(), C, bias, act, residual, pre, p,
              rng, stream)


def _saved(saved, M, N, K):
    if not isinstance(saved, LinearSaved):
        raise TypeError(f"saved: expected LinearSaved, got {type(saved).__name__}")
    saved.check(M, N, K)
    return ctypes.addressof(saved.struct())


def fp8_scaled_linear_fwd_epilogue(x: torch.Tensor, w: torch.Tensor, saved: LinearSaved, y: torch.Tensor, *, bias=None,
                                   act: int = ACT_NONE, residual=None, pre=None, p: float = 0.0, rng=None,
                                   stream=None):
    """y[M,N] = residual + drop(act(x[M,K] w[N,K]^T + bias)) through the FP8 path with
    dynamic scaling; x and w bf16 or fp16.  saved receives the codes and scale records."""
    M, K = _need_2d(x, "x")
    N, _ = _need_2d(w, "w")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x: dtype {x.dtype}, expected bfloat16 or float16")
    _need(x, "x", x.dtype)
    _need(w, "w", x.dtype, shape=(N, K))
    yt = _type(y, "y")
    sv = _saved(saved, M, N, K)
    e = _epilogue(y, (M, N), M, N, x.dtype, bias, act, residual, pre, p, rng, x, w, saved.x_q, saved.w_q,
                  saved.x_sc.buf, saved.w_sc.buf)
    _check(lib().fp8_scaled_linear_fwd_epilogue(x.data_ptr(), w.data_ptr(), _TYPE[x.dtype], M, N, K, sv,
                                                e, _ptr(y), yt, _stream(stream)),
           "fp8_scaled_linear_fwd_epilogue")


def fp8_scaled_linear_bwd_epilogue(gy: torch.Tensor, saved: LinearSaved, ws: LinearBwdWs, gx: torch.Tensor,
                                   gw: torch.Tensor, *, gh=None, gb=None, pre=None, act: int = ACT_NONE,
                                   p: float = 0.0, rng=None, part=None, stream=None):
    """The gradients gx, gw (of one dtype) and gb (or None) of
    fp8_scaled_linear_fwd_epilogue from gy and the forward's saved, pre, act, p and rng.
    gh: scratch like gy, or gy itself; None where the epilogue leaves gy as it is.
    part: float32, epilogue_workspace_len(M, N) of them, where gb is wanted (up to 256
    rows optional, though mxfp4_linear_bwd_epilogue takes a pass less with it)."""
    M, N = _need_2d(gy, "gy")
    if gy.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"gy: dtype {gy.dtype}, expected bfloat16 or float16")
    _need(gy, "gy", gy.dtype)
    K = _need_2d(getattr(saved, "x_q", None), "saved.x_q")[1]
    ot = _type(gx, "gx")
    _same(gx, "gx", gx.dtype, (M, K))
    _same(gw, "gw", gx.dtype, (N, K))
    sv = _saved(saved, M, N, K)
    if not isinstance(ws, LinearBwdWs):
        raise TypeError(f"ws: expected LinearBwdWs, got {type(ws).__name__}")
    ws.check(M, N)
    wc = ctypes.addressof(ws.struct())
    e, n = _backward(gy, gh, gb, pre, act, p, rng, part, M, N, False, (gx, "gx"), (gw, "gw"))
    _here(gx, gw, saved.x_q, saved.w_q, saved.x_sc.buf, saved.w_sc.buf, ws.gy_q, ws.gy_sc.buf)
    _check(lib().fp8_scaled_linear_bwd_epilogue(_ptr(gy), _TYPE[gy.dtype], sv, M, N, K, wc,
                                                e, _ptr(gh), _ptr(gb), _ptr(part), n, _ptr(gx), _ptr(gw),
                                                ot, _stream(stream)), "fp8_scaled_linear_bwd_epilogue")


# ----------------------------------------------------------------- backward step

def epilogue_workspace_len(M: int, N: int) -> int:
    """Floats of workspace that the backward step of an M x N epilogue needs for gb."""
    return _bytes(M, N, "epilogue_workspace_len", lib().epilogue_workspace_len)


def epilogue_bwd(gy: torch.Tensor, gh=None, gb=None, *, pre=None, act: int = ACT_NONE, p: float = 0.0, rng=None,
                 part=None, stream=None):
    """gh = drop(gy) * act'(pre) and gb = the sum of its (unrounded) rows; either may
    be None, and gh may be gy.  part: see fp8_scaled_linear_bwd_epilogue."""
    M, N = _matrix(gy, "gy")
    if gh is None and gb is None:
        raise ValueError("epilogue_bwd: gh or gb is needed")
    e, n = _backward(gy, gh, gb, pre, act, p, rng, part, M, N, True)
    _check(lib().epilogue_bwd(_ptr(gy), _TYPE[gy.dtype], e, M, N, _ptr(gh), _ptr(gb), _ptr(part), n,
                              _stream(stream)), "epilogue_bwd")


# ------------------------------------------------------------------------- MXFP4

def mxfp4_gemm_epilogue(A: Mxfp4, B: Mxfp4, C: torch.Tensor, *, bias=None, act: int = ACT_NONE, residual=None,
                        pre=None, p: float = 0.0, rng=None, stream=None):
    """C[M,N] = residual + drop(act(A[M,K] B[N,K]^T + bias)) in C's dtype."""
    for m, name in ((A, "A"), (B, "B")):
        if not isinstance(m, Mxfp4):
            raise TypeError(f"{name}: expected Mxfp4, got {type(m).__name__}")
    M, N = A.rows, B.rows
    _need_codes(B, "B", Mxfp4, N, A.k)
    ct = _type(C, "C")
    if C.dim() < 1 or C.shape[-1] != N or _rows(C) != M:
        raise ValueError(f"C: shape {tuple(C.shape)}, expected {M} x {N}")
    e = _epilogue(C, C.shape, M, N, None, bias, act, residual, pre, p, rng, A.q, A.s, B.q, B.s,
                  clear=(A.q, A.s, B.q, B.s))
    _check(lib().mxfp4_gemm_epilogue(A.c(), B.c(), e, _ptr(C), ct, M, N, A.k, _stream(stream)),
           "mxfp4_gemm_epilogue")


def mxfp4_linear_fwd_epilogue(x: torch.Tensor, w: torch.Tensor, ws: Mxfp4LinearWs, saved: Mxfp4LinearSaved,
                              y: torch.Tensor, *, bias=None, act: int = ACT_NONE, residual=None, pre=None,
                              p: float = 0.0, rng=None, rule: int = MX_FLOOR, stream=None):
    """mxfp4_linear_fwd with an epilogue: y = residual + drop(act(x w^T + bias))."""
    M, K = _matrix(x, "x")
    N, K2 = _matrix(w, "w")
    if w.dtype != x.dtype:
        raise TypeError(f"w: dtype {w.dtype}, expected x's {x.dtype}")
    if K2 != K:
        raise ValueError(f"w: {K2} columns, expected {K}")
    yt = _type(y, "y")
    e = _epilogue(y, _lead(x.shape, N), M, N, x.dtype, bias, act, residual, pre, p, rng, x, w)
    _linear(ws, Mxfp4LinearWs, "ws", (M, N, K), ("x_q", "w_q"))
    sv = None
    if saved is not None:
        _linear(saved, Mxfp4LinearSaved, "saved", (M, N, K), ("x_qT", "w_qT"))
        sv = saved.c()
    _check(lib().mxfp4_linear_fwd_epilogue(_ptr(x), _ptr(w), _TYPE[x.dtype], M, N, K, _rule(rule), ws.c(), sv,
                                           e, _ptr(y), yt, _stream(stream)), "mxfp4_linear_fwd_epilogue")


def mxfp4_linear_apply_epilogue(x: torch.Tensor, w: Mxfp4, y: torch.Tensor, ws: Mxfp4, *, bias=None,
                                act: int = ACT_NONE, residual=None, pre=None, p: float = 0.0, rng=None,
                                rule: int = MX_FLOOR, stream=None):
    """mxfp4_linear_apply with an epilogue: y = residual + drop(act(x w^T + bias))."""
    M, K = _matrix(x, "x")
    if not isinstance(w, Mxfp4):
        raise TypeError(f"w: expected Mxfp4, got {type(w).__name__}")
    N = w.rows
    _need_codes(w, "w", Mxfp4, N, K)
    _need_codes(ws, "ws", Mxfp4, M, K)
    yt = _type(y, "y")
    e = _epilogue(y, (M, N) if x.dim() == 2 else _lead(x.shape, N), M, N, x.dtype, bias, act, residual, pre, p, rng,
                  x, w.q, w.s, ws.q, ws.s)
    _check(lib().mxfp4_linear_apply_epilogue(_ptr(x), _TYPE[x.dtype], w.c(), M, N, K, _rule(rule), ws.c(),
                                             e, _ptr(y), yt, _stream(stream)),
           "mxfp4_linear_apply_epilogue")


def mxfp4_linear_bwd_epilogue(gy: torch.Tensor, ws: Mxfp4LinearWs, saved: Mxfp4LinearSaved, gx, gw, *, gh=None,
                              gb=None, pre=None, act: int = ACT_NONE, p: float = 0.0, rng=None, part=None,
                              rule: int = MX_FLOOR, stream=None):
    """The gradients gx, gw and gb (each may be None) of mxfp4_linear_fwd_epilogue;
    gh and part as in fp8_scaled_linear_bwd_epilogue."""
    M, N = _matrix(gy, "gy")
    if not isinstance(saved, Mxfp4LinearSaved):
        raise TypeError(f"saved: expected Mxfp4LinearSaved, got {type(saved).__name__}")
    K = saved.dims[2]
    if gx is None and gw is None and gb is None:
        raise ValueError("mxfp4_linear_bwd_epilogue: gx, gw or gb is needed")
    out = gw if gx is None else gx
    need, ot = (), 0
    if out is not None:
        ot = _type(out, "gw" if gx is None else "gx")
    if gx is not None:
        _same(gx, "gx", out.dtype, _lead(gy.shape, K))
        need += ("gy_q",)
    if gw is not None:
        _same(gw, "gw", out.dtype, (N, K))
        need += ("gy_qT",)
    e, n = _backward(gy, gh, gb, pre, act, p, rng, part, M, N, out is None, (gx, "gx"), (gw, "gw"))
    _here(gx, gw)
    _linear(ws, Mxfp4LinearWs, "ws", (M, N, K), need)
    _linear(saved, Mxfp4LinearSaved, "saved", (M, N, K), ("x_qT", "w_qT"))
    _check(lib().mxfp4_linear_bwd_epilogue(_ptr(gy), _TYPE[gy.dtype], M, N, K, _rule(rule), ws.c(), saved.c(),
                                           e, _ptr(gh), _ptr(gb), _ptr(part), n, _ptr(gx), _ptr(gw), ot,
                                           _stream(stream)), "mxfp4_linear_bwd_epilogue")


# ------------------------------------------------------------------------- dropout

def _dropout(x, name_x, p, rng, y, name_y, residual):
    """(x, ldx, residual, ldr, type, rows, cols, p, rng, y, ldy), checked."""
    xt = _TYPE.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if xt is None:
        _type(x, name_x)  # (says what it is)
    dt, shape = x.dtype, x.shape
    if not shape:
        raise ValueError(f"{name_x}: expected at least one dimension")
    cols = shape[-1]
    rows = shape[0] if len(shape) == 2 else _rows(x)
    ldx = cols if x.is_contiguous() else _row_stride(x, name_x, dt, shape, rows, cols)
    ldy = _row_stride(y, name_y, dt, shape, rows, cols)
    px, py, size = x.data_ptr(), y.data_ptr(), rows * _SIZE[dt]
    end = py + ldy * size
    # in place is allowed; what comes near in another way is looked at more closely
    if py < px + ldx * size and px < end and (px != py or ldx != ldy) and cols:
        _clear(y, name_y, x, name_x)
    pr = ldr = 0
    if residual is not None:
        ldr = _row_stride(residual, "residual", dt, shape, rows, cols)
        pr = residual.data_ptr()
        if py < pr + ldr * size and pr < end and (pr != py or ldr != ldy) and cols:
            _clear(y, name_y, residual, "residual")
    words = _drop(p, rng)
    _here(x, y, residual, rng)
    return px, ldx, pr, ldr, xt, rows, cols, p, words, py, ldy


def dropout_fwd(x: torch.Tensor, p: float, rng, y: torch.Tensor, residual=None, stream=None):
    """y = residual + drop(x): an element is kept with probability 1 - p and then
    scaled by its inverse.  rng: the generator's two int64 words on the device (None
    where p is 0).  Rows of the last dimension may be apart; y may be x or residual."""
    _check(lib().dropout_fwd(*_dropout(x, "x", p, rng, y, "y", residual), _stream(stream)), "dropout_fwd")


def dropout_bwd(gy: torch.Tensor, p: float, rng, gx: torch.Tensor, stream=None):
    """gx = drop(gy) with the forward's p and rng; gx may be gy."""
    g, ld, _, _, t, rows, cols, p, words, gx, ldx = _dropout(gy, "gy", p, rng, gx, "gx", None)
    _check(lib().dropout_bwd(g, ld, t, rows, cols, p, words, gx, ldx, _stream(stream)), "dropout_bwd")
