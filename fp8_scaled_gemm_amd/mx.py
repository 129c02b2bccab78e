"""Binding of the microscaled formats (MXFP4 matrices, 8-bit activation
checkpoints), the gated activation and the layer norm: include/fp8sg.h's entry
points of the same names, on the current torch stream.  Its names are those of
the package (`import fp8_scaled_gemm_amd as F; F.mxfp4_gemm(...)`).

Argument marshalling only, as in the package itself: every buffer's dtype,
shape, strides and device are checked here, before the library is called (the
two buffers of an operand where they are put into it, their device on each call).
"""
import ctypes

import torch

from . import _check, _cur_device, _need, _raw_stream, lib

MX_FLOOR, MX_FIT = 0, 1

_TYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class _Pair(ctypes.Structure):  # mxfp4_operand and fp8sg_act8
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p)]


class _LinSaved(ctypes.Structure):
    _fields_ = [("x_qT", _Pair), ("w_qT", _Pair)]


class _LinWs(ctypes.Structure):
    _fields_ = [("x_q", _Pair), ("w_q", _Pair), ("gy_q", _Pair), ("gy_qT", _Pair)]


def bind(L):
    """Argument types of this module's entry points."""
    P, i64, i, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.mxfp4_code_bytes.argtypes = L.mxfp4_scale_bytes.argtypes = [i64, i64]
    L.mxfp4_quantize.argtypes = [P, i, i64, i64, i, P, P, P]
    L.mxfp4_dequantize.argtypes = [P, i64, i64, P, i, P]
    L.mxfp4_gemm.argtypes = [P, P, P, i, i64, i64, i64, P]
    L.mxfp4_linear_fwd.argtypes = [P, P, i, i64, i64, i64, i, P, P, P, i, P]
    L.mxfp4_linear_bwd.argtypes = [P, i, i64, i64, i64, i, P, P, P, P, i, P]
    L.mxfp4_linear_apply.argtypes = [P, i, P, i64, i64, i64, i, P, P, i, P]
    L.act8_quantize.argtypes = [P, i, i64, i64, P, P]
    L.act8_dequantize.argtypes = [P, i64, i64, P, i, P]
    L.swiglu_fwd.argtypes = [P, i64, P, i64, i, i64, i64, P, P, P, P]
    L.swiglu_bwd.argtypes = [P, P, i64, P, i64, P, P, i, i64, i64, P, i64, P, i64, P]
    L.layer_norm_fwd.argtypes = [P, i, P, P, i, i64, i64, f32, P, P, P, P, P]
    L.layer_norm_workspace_len.argtypes = [i64, i64]
    L.layer_norm_bwd.argtypes = [P, P, P, i, P, i, P, P, i64, i64, P, P, P, P, i64, P]
    for name in ("mxfp4_code_bytes", "mxfp4_scale_bytes", "layer_norm_workspace_len"):
        getattr(L, name).restype = i64


def _here(*tensors):
    """Every tensor is on the current device, whose stream the call uses."""
    dev = _device()
    for t in tensors:
        if t is not None and t.get_device() != dev:  # (-1: not on a device)
            if not t.is_cuda:
                raise ValueError("tensor arguments must be device tensors")
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}: "
                             "call under torch.cuda.device(...)")


# The calls are short: their host time is kept down by passing addresses as
# plain integers and by one struct per buffer pair, filled again on each call.
_device = _cur_device if _cur_device is not None else torch.cuda.current_device


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(stream):
    """hipStream_t of `stream`, or of torch's current stream on the current device."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(_device()) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _type(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    ty = _TYPE.get(t.dtype)  # (c_int of the C ABI's fp8sg_out)
    if ty is None:
        raise TypeError(f"{name}: dtype {t.dtype}, expected bfloat16, float16 or float32")
    return ty


def _same(t, name, dtype, shape):
    """t is a contiguous tensor of this dtype and shape (_need names what differs)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    _need(t, name, dtype, shape=shape)


def _rule(rule):
    if rule not in (MX_FLOOR, MX_FIT):
        raise ValueError(f"rule must be MX_FLOOR or MX_FIT, not {rule!r}")
    return rule


def _matrix(t, name):
    """(rows, cols) of a contiguous matrix; leading dimensions count as rows."""
    _type(t, name)
    shape = t.shape
    if not shape:
        raise ValueError(f"{name}: expected at least one dimension")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if len(shape) == 2:
        return shape
    cols = shape[-1]
    return (t.numel() // cols if cols else _rows(t)), cols


def _rows(t):
    n = 1
    for d in t.shape[:-1]:
        n *= d
    return n


def _bytes(rows, k, what, fn):
    n = fn(rows, k)
    if n < 0:
        raise ValueError(f"{what}: {rows} x {k} is outside the size limits")
    return n


class _Codes:
    """Codes q and scales s of a matrix of fixed size (_fixed).  Either buffer may
    be exchanged for another that fits."""

    def _place(self):
        """The C struct, for c()."""
        d = self.__dict__
        d["_pair"] = p = _Pair()
        d["_at"] = ctypes.addressof(p)

    def __getstate__(self):  # for copies and pickles: all but the struct of addresses
        return {n: self.__dict__[n] for n in self._fixed + ("q", "s")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._place()

    def __setattr__(self, name, value):
        if name in self._fixed:
            raise AttributeError(f"{name}: the size of a {type(self).__name__} is fixed")
        if name in ("q", "s"):
            self._fits(value, name)
        super().__setattr__(name, value)

    def tensors(self):
        return self.q, self.s

    def c(self):
        """Address of the C struct, holding the buffers' present addresses."""
        p = self._pair
        p.q, p.s = self.q.data_ptr(), self.s.data_ptr()
        return self._at


class Mxfp4(_Codes):
    """An MXFP4 matrix, rows x k (mxfp4_operand): codes q and scales s, two
    uint8 device tensors, uninitialised until a call writes them."""
    _fixed = ("rows", "k")

    def __init__(self, rows: int, k: int, device="cuda", tensors=None):
        d = self.__dict__  # (past __setattr__: the buffers are checked or made here)
        d["rows"], d["k"] = rows, k
        L = lib()
        nq = _bytes(rows, k, "Mxfp4", L.mxfp4_code_bytes)
        ns = _bytes(rows, k, "Mxfp4", L.mxfp4_scale_bytes)
        if tensors is None:
            d["q"] = torch.empty(nq, dtype=torch.uint8, device=device)
            d["s"] = torch.empty(ns, dtype=torch.uint8, device=device)
        else:  # the two buffers of another Mxfp4 of the same size
            d["q"], d["s"] = tensors
            _need(self.q, "q", torch.uint8, numel=nq)
            _need(self.s, "s", torch.uint8, numel=ns)

        self._place()

    def _fits(self, t, name):
        L = lib()
        _need(t, name, torch.uint8, numel=(L.mxfp4_code_bytes if name == "q" else L.mxfp4_scale_bytes)(self.rows, self.k))


class Act8(_Codes):
    """An 8-bit checkpoint of a rows x cols activation (fp8sg_act8)."""
    _fixed = ("rows", "cols")

    def __init__(self, rows: int, cols: int, device="cuda", tensors=None):
        if rows < 0 or cols < 0:
            raise ValueError(f"Act8: {rows} x {cols}")
        d = self.__dict__
        d["rows"], d["cols"] = rows, cols
        blocks = -(-cols // 32)
        if tensors is None:
            d["q"] = torch.empty((rows, 32 * blocks), dtype=torch.uint8, device=device)
            d["s"] = torch.empty((rows, blocks), dtype=torch.uint8, device=device)
        else:
            d["q"], d["s"] = tensors
            _need(self.q, "q", torch.uint8, shape=(rows, 32 * blocks))
            _need(self.s, "s", torch.uint8, shape=(rows, blocks))

        self._place()

    def _fits(self, t, name):
        blocks = -(-self.cols // 32)
        _need(t, name, torch.uint8, shape=(self.rows, 32 * blocks if name == "q" else blocks))


def _need_codes(m, name, kind, rows, cols):
    if m.__class__ is kind and m.rows == rows and (m.k if kind is Mxfp4 else m.cols) == cols:
        return
    if not isinstance(m, kind):
        raise TypeError(f"{name}: expected {kind.__name__}, got {type(m).__name__}")
    got = (m.rows, m.k) if kind is Mxfp4 else (m.rows, m.cols)
    if got != (rows, cols):
        raise ValueError(f"{name}: {got[0]} x {got[1]}, expected {rows} x {cols}")


def _apart(a, name_a, lda, b, name_b, ldb):
    """Two outputs of one shape, rows lda and ldb elements apart, share no memory
    (they may be column ranges of one matrix)."""
    pa, pb = a.data_ptr(), b.data_ptr()
    if pb < pa:
        pa, pb, lda, ldb = pb, pa, ldb, lda
    n, cols = a.numel(), a.shape[-1]
    if n == 0:
        return
    rows, at = n // cols, (pb - pa) // a.element_size()
    if at >= (rows - 1) * lda + cols:
        return
    if lda == ldb:
        clear = cols <= at % lda <= lda - cols
    else:  # row i of the first against the first row of the second that ends behind its start
        clear = True
        for i in range(rows):
            j = max(0, -(-(i * lda - cols + 1 - at) // ldb))
            if j < rows and at + j * ldb < i * lda + cols:
                clear = False
                break
    if not clear:
        raise ValueError(f"{name_a} and {name_b} overlap")


def _own_codes(a, name_a, b, name_b):
    """Two operands that one call writes have buffers of their own."""
    if a.q is b.q or a.s is b.s:
        raise ValueError(f"the buffers of {name_a} and {name_b} overlap")


# ------------------------------------------------------------------- MXFP4

def mxfp4_quantize(x: torch.Tensor, q: Mxfp4 = None, qT: Mxfp4 = None, rule: int = MX_FLOOR, stream=None):
    """Codes of x (rows x cols) along its rows into q (rows x cols) and / or along
    its columns into qT (cols x rows)."""
    rows, cols = _matrix(x, "x")
    if q is None and qT is None:
        raise ValueError("mxfp4_quantize: q or qT is needed")
    if q is qT:
        raise ValueError("mxfp4_quantize: q and qT are one object, each needs its own")
    args = []
    for m, name, shape in ((q, "q", (rows, cols)), (qT, "qT", (cols, rows))):
        if m is not None:
            _need_codes(m, name, Mxfp4, *shape)
            _here(m.q, m.s)
        args.append(m.c() if m is not None else None)
    if q is not None and qT is not None:
        _own_codes(q, "q", qT, "qT")
    _here(x)
    _check(lib().mxfp4_quantize(_ptr(x), _TYPE[x.dtype], rows, cols, _rule(rule), args[0], args[1],
                                _stream(stream)), "mxfp4_quantize")


def mxfp4_dequantize(m: Mxfp4, y: torch.Tensor, stream=None):
    """The values of m's codes into y (rows x k)."""
    rows, k = _matrix(y, "y")
    _need_codes(m, "m", Mxfp4, rows, k)
    _here(y, m.q, m.s)
    c = m.c()
    _check(lib().mxfp4_dequantize(c, rows, k, _ptr(y), _TYPE[y.dtype], _stream(stream)), "mxfp4_dequantize")


def mxfp4_gemm(A: Mxfp4, B: Mxfp4, C: torch.Tensor, stream=None):
    """C[M,N] = A[M,K] B[N,K]^T in C's dtype."""
    M, N = _matrix(C, "C")
    for m, name in ((A, "A"), (B, "B")):
        if not isinstance(m, Mxfp4):
            raise TypeError(f"{name}: expected Mxfp4, got {type(m).__name__}")
    _need_codes(A, "A", Mxfp4, M, A.k)
    _need_codes(B, "B", Mxfp4, N, A.k)
    _here(C, A.q, A.s, B.q, B.s)
    a, b = A.c(), B.c()
    _check(lib().mxfp4_gemm(a, b, _ptr(C), _TYPE[C.dtype], M, N, A.k, _stream(stream)), "mxfp4_gemm")


class _Operands:
    """A layer's operands, attributes with the names of a C struct's fields; any
    may be exchanged for another operand, e.g. for one that two layers share."""

    def __init__(self, dims, *operands):
        d = self.__dict__
        struct = self._struct()
        d.update(zip(self._names, operands))
        d["dims"], d["_all"], d["_at"] = dims, struct, ctypes.addressof(struct)
        self._place()

    def __getstate__(self):  # for copies and pickles: all but the struct of addresses
        return {n: getattr(self, n) for n in self._names + ("dims",)}

    def __setstate__(self, state):
        _Operands.__init__(self, state["dims"], *(state[n] for n in self._names))

    def _place(self):
        """The operands with their places in the struct, for c()."""
        held = self.__dict__["_held"] = []
        for name in self._names:
            pair, m = getattr(self._all, name), getattr(self, name)
            if m is not None:
                held.append((pair, m))
            elif pair.q:
                pair.q = pair.s = None

    def __setattr__(self, name, value):
        if name == "dims":
            raise AttributeError("dims: the operands were made for these sizes")
        if name in self._names:
            if value is not None:
                M, N, K = self.dims
                _need_codes(value, name, Mxfp4, *self._shapes(M, N, K)[self._names.index(name)])
            super().__setattr__(name, value)
            self._place()
        else:
            super().__setattr__(name, value)

    def c(self):
        """Address of the C struct, holding the present operands' present addresses."""
        for pair, m in self._held:
            pair.q, pair.s = m.q.data_ptr(), m.s.data_ptr()
        return self._at


class Mxfp4LinearSaved(_Operands):
    """What the forward of an M x N x K MXFP4 linear leaves for its backward."""
    _struct, _names = _LinSaved, tuple(n for n, _ in _LinSaved._fields_)

    @staticmethod
    def _shapes(M, N, K):
        return (K, M), (K, N)

    def __init__(self, M, N, K, device="cuda", tensors=None):
        t = tensors or (None, None, None, None)
        super().__init__((M, N, K), Mxfp4(K, M, device, t[0:2] if tensors else None),
                         Mxfp4(K, N, device, t[2:4] if tensors else None))

    def tensors(self):
        return self.x_qT.tensors() + self.w_qT.tensors()


class Mxfp4LinearWs(_Operands):
    """Operands that live within one forward or backward call.  The two calls
    use different ones; calls that may overlap in time need a workspace each."""
    _struct, _names = _LinWs, tuple(n for n, _ in _LinWs._fields_)

    @staticmethod
    def _shapes(M, N, K):
        return (M, K), (N, K), (M, N), (N, M)

    def __init__(self, M, N, K, device="cuda", forward=True, backward=True):
        super().__init__((M, N, K),
                         Mxfp4(M, K, device) if forward else None, Mxfp4(N, K, device) if forward else None,
                         Mxfp4(M, N, device) if backward else None, Mxfp4(N, M, device) if backward else None)


def _linear(obj, kind, name, dims, fields):
    if not isinstance(obj, kind):
        raise TypeError(f"{name}: expected {kind.__name__}, got {type(obj).__name__}")
    if obj.dims != dims:
        raise ValueError(f"{name}: made for a layer of {obj.dims}, not {dims}")
    tensors = ()
    for f in fields:
        m = getattr(obj, f)
        if m is None:
            raise ValueError(f"{name}: made without {f}")
        tensors += (m.q, m.s)
    if len(fields) == 2 and (tensors[0] is tensors[2] or tensors[1] is tensors[3]):
        raise ValueError(f"{name}: the buffers of {fields[0]} and {fields[1]} overlap")
    _here(*tensors)


def mxfp4_linear_fwd(x: torch.Tensor, w: torch.Tensor, ws: Mxfp4LinearWs, saved: Mxfp4LinearSaved, y: torch.Tensor,
                     rule: int = MX_FLOOR, stream=None):
    """y[M,N] = x[M,K] w[N,K]^T with both operands quantised to MXFP4; saved (or
    None) receives what the backward needs."""
    M, K = _matrix(x, "x")
    N, K2 = _matrix(w, "w")
    if w.dtype != x.dtype:
        raise TypeError(f"w: dtype {w.dtype}, expected x's {x.dtype}")
    if K2 != K:
        raise ValueError(f"w: {K2} columns, expected {K}")
    _type(y, "y")
    _same(y, "y", y.dtype, x.shape[:-1] + (N,))
    _here(x, w, y)
    _linear(ws, Mxfp4LinearWs, "ws", (M, N, K), ("x_q", "w_q"))
    sv = None
    if saved is not None:
        _linear(saved, Mxfp4LinearSaved, "saved", (M, N, K), ("x_qT", "w_qT"))
        sv = saved.c()
    wc = ws.c()
    _check(lib().mxfp4_linear_fwd(_ptr(x), _ptr(w), _TYPE[x.dtype], M, N, K, _rule(rule), wc, sv,
                                  _ptr(y), _TYPE[y.dtype], _stream(stream)), "mxfp4_linear_fwd")


def mxfp4_linear_bwd(gy: torch.Tensor, ws: Mxfp4LinearWs, saved: Mxfp4LinearSaved, gx, gw, rule: int = MX_FLOOR,
                     stream=None):
    """gx[M,K] = gy[M,N] W and gw[N,K] = gy^T x from what the forward saved; either
    may be None."""
    M, N = _matrix(gy, "gy")
    if not isinstance(saved, Mxfp4LinearSaved):
        raise TypeError(f"saved: expected Mxfp4LinearSaved, got {type(saved).__name__}")
    K = saved.dims[2]
    if gx is None and gw is None:
        raise ValueError("mxfp4_linear_bwd: gx or gw is needed")
    out = gw if gx is None else gx
    _type(out, "gw" if gx is None else "gx")
    need = ()
    if gx is not None:
        _same(gx, "gx", out.dtype, gy.shape[:-1] + (K,))
        need += ("gy_q",)
    if gw is not None:
        _same(gw, "gw", out.dtype, (N, K))
        need += ("gy_qT",)
    px, pw = _ptr(gx), _ptr(gw)
    if px and pw and (pw - px < gx.nbytes if px <= pw else px - pw < gw.nbytes):
        raise ValueError("gx and gw overlap")
    _here(gy, gx, gw)
    _linear(ws, Mxfp4LinearWs, "ws", (M, N, K), need)
    _linear(saved, Mxfp4LinearSaved, "saved", (M, N, K), ("x_qT", "w_qT"))
    wc, sv = ws.c(), saved.c()
    _check(lib().mxfp4_linear_bwd(_ptr(gy), _TYPE[gy.dtype], M, N, K, _rule(rule), wc, sv, px, pw,
                                  _TYPE[out.dtype], _stream(stream)), "mxfp4_linear_bwd")


def mxfp4_linear_apply(x: torch.Tensor, w: Mxfp4, y: torch.Tensor, ws: Mxfp4, rule: int = MX_FLOOR, stream=None):
    """y[M,N] = x[M,K] w^T with the weight held as MXFP4 (N x K); ws: scratch (M x K)."""
    M, K = _matrix(x, "x")
    if not isinstance(w, Mxfp4):
        raise TypeError(f"w: expected Mxfp4, got {type(w).__name__}")
    _need_codes(w, "w", Mxfp4, w.rows, K)
    _need_codes(ws, "ws", Mxfp4, M, K)
    _type(y, "y")
    _same(y, "y", y.dtype, x.shape[:-1] + (w.rows,))
    _here(x, y, w.q, w.s, ws.q, ws.s)
    wc, xc = w.c(), ws.c()
    _check(lib().mxfp4_linear_apply(_ptr(x), _TYPE[x.dtype], wc, M, w.rows, K, _rule(rule), xc, _ptr(y),
                                    _TYPE[y.dtype], _stream(stream)), "mxfp4_linear_apply")


# ---------------------------------------------- 8-bit checkpoints, gated activation

def act8_quantize(x: torch.Tensor, c: Act8, stream=None):
    """The 8-bit checkpoint of x (rows x cols)."""
    rows, cols = _matrix(x, "x")
    _need_codes(c, "c", Act8, rows, cols)
    _here(x, c.q, c.s)
    p = c.c()
    _check(lib().act8_quantize(_ptr(x), _TYPE[x.dtype], rows, cols, p, _stream(stream)), "act8_quantize")


def act8_dequantize(c: Act8, y: torch.Tensor, stream=None):
    """The values of a checkpoint into y (rows x cols)."""
    rows, cols = _matrix(y, "y")
    _need_codes(c, "c", Act8, rows, cols)
    _here(y, c.q, c.s)
    p = c.c()
    _check(lib().act8_dequantize(p, rows, cols, _ptr(y), _TYPE[y.dtype], _stream(stream)), "act8_dequantize")


def _strided(t, name, like, rows, cols):
    """Row stride of a matrix whose rows are contiguous (a column range of a
    wider matrix qualifies); more than two dimensions must be contiguous."""
    if t.__class__ is like.__class__ and t.dtype is like.dtype and t.shape == like.shape and t.is_contiguous():
        return cols
    if _type(t, name) != _TYPE[like.dtype]:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {like.dtype}")
    if t.shape[-1] != cols or _rows(t) != rows:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {rows} x {cols}")
    if t.is_contiguous():
        return cols
    if t.dim() != 2 or (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return t.stride(0) if rows > 1 else cols


def _ckpts(cg, cu, rows, cols, written):
    if (cg is None) != (cu is None):
        raise ValueError("both checkpoints are needed, or none")
    if cg is None:
        return None, None
    if cg is cu and written:
        raise ValueError("g and u need a checkpoint each")
    _need_codes(cg, "g's checkpoint", Act8, rows, cols)
    _need_codes(cu, "u's checkpoint", Act8, rows, cols)
    if written:
        _own_codes(cg, "g's checkpoint", cu, "u's checkpoint")
    _here(cg.q, cg.s, cu.q, cu.s)
    return cg.c(), cu.c()


def swiglu_fwd(g: torch.Tensor, u: torch.Tensor, a: torch.Tensor, cg: Act8 = None, cu: Act8 = None, stream=None):
    """a = silu(g) * u; cg and cu receive 8-bit checkpoints of g and u.  g and u
    may be column ranges of a wider matrix."""
    rows, cols = _matrix(a, "a")
    ldg, ldu = _strided(g, "g", a, rows, cols), _strided(u, "u", a, rows, cols)
    _here(g, u, a)
    pg, pu = _ckpts(cg, cu, rows, cols, True)
    _check(lib().swiglu_fwd(_ptr(g), ldg, _ptr(u), ldu, _TYPE[a.dtype], rows, cols, _ptr(a), pg, pu,
                            _stream(stream)), "swiglu_fwd")


def swiglu_bwd(da: torch.Tensor, g, u, dg: torch.Tensor, du: torch.Tensor, stream=None):
    """The gradients of swiglu_fwd from da and g, u: the forward's inputs, or
    their checkpoints (Act8)."""
    rows, cols = _matrix(da, "da")
    lddg, lddu = _strided(dg, "dg", da, rows, cols), _strided(du, "du", da, rows, cols)
    pdg, pdu = dg.data_ptr(), du.data_ptr()
    if abs(pdu - pdg) < 4 * rows * max(lddg, lddu):  # (farther apart they cannot overlap)
        _apart(dg, "dg", lddg, du, "du", lddu)
    _here(da, dg, du)
    if isinstance(g, Act8) or isinstance(u, Act8):
        pg, pu = _ckpts(g, u, rows, cols, False)
        args = (None, 0, None, 0, pg, pu)
    else:
        ldg, ldu = _strided(g, "g", da, rows, cols), _strided(u, "u", da, rows, cols)
        _here(g, u)
        args = (_ptr(g), ldg, _ptr(u), ldu, None, None)
    _check(lib().swiglu_bwd(_ptr(da), *args, _TYPE[da.dtype], rows, cols, pdg, lddg, pdu, lddu,
                            _stream(stream)), "swiglu_bwd")


# --------------------------------------------------------------------- layer norm

def _params(like, cols, *named):
    """Type code of the parameters (name, tensor): the data's dtype or float32,
    the same for all that are given."""
    dtype, shape = None, (cols,)
    for name, t in named:
        if t is None:
            continue
        if dtype is None:
            _type(t, name)
            dtype = t.dtype
        if dtype is not like.dtype and dtype is not torch.float32 or t.dtype is not dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {like.dtype} (or float32 for all parameters)")
        _same(t, name, dtype, shape)
    return _TYPE[dtype or like.dtype]


def layer_norm_fwd(x: torch.Tensor, w, b, eps: float, y: torch.Tensor, mean=None, rstd=None, ckpt: Act8 = None,
                   stream=None):
    """y = (x - mean) * rstd * w + b over the last dimension; w and b may be None.
    mean and rstd (float32, one value per row, in any shape) and ckpt (an 8-bit copy of x) are
    written for the backward."""
    rows, cols = _matrix(x, "x")
    _same(y, "y", x.dtype, x.shape)
    pt = _params(x, cols, ("w", w), ("b", b))
    pm = pr = None
    if mean is not None or rstd is not None:
        _need(mean, "mean", torch.float32, numel=rows)
        _need(rstd, "rstd", torch.float32, numel=rows)
        pm, pr = mean.data_ptr(), rstd.data_ptr()
        if abs(pr - pm) < 4 * rows:
            raise ValueError("mean and rstd overlap")
    p = None
    if ckpt is not None:
        _need_codes(ckpt, "ckpt", Act8, rows, cols)
        _here(ckpt.q, ckpt.s)
        p = ckpt.c()
    _here(x, y, w, b, mean, rstd)
    _check(lib().layer_norm_fwd(x.data_ptr(), _TYPE[x.dtype], _ptr(w), _ptr(b), pt, rows, cols, eps, y.data_ptr(),
                                pm, pr, p, _stream(stream)), "layer_norm_fwd")


def layer_norm_workspace_len(rows: int, cols: int) -> int:
    """Floats of workspace that layer_norm_bwd needs."""
    return _bytes(rows, cols, "layer_norm_workspace_len", lib().layer_norm_workspace_len)


def layer_norm_bwd(dy: torch.Tensor, x, w, mean, rstd, dx=None, dw=None, db=None, ws=None, stream=None):
    """dx, dw and db (each may be None) from dy, the forward's x or its
    checkpoint (Act8), and the forward's mean and rstd."""
    rows, cols = _matrix(dy, "dy")
    xp = cp = None
    if isinstance(x, Act8):
        _need_codes(x, "x", Act8, rows, cols)
        _here(x.q, x.s)
        cp = x.c()
    else:
        _same(x, "x", dy.dtype, dy.shape)
        _here(x)
        xp = x.data_ptr()
    pt = _params(dy, cols, ("w", w), ("dw", dw), ("db", db))
    _need(mean, "mean", torch.float32, numel=rows)
    _need(rstd, "rstd", torch.float32, numel=rows)
    if dx is not None:
        _same(dx, "dx", dy.dtype, dy.shape)
    pdw, pdb = _ptr(dw), _ptr(db)
    if pdw and pdb and abs(pdb - pdw) < cols * (4 if pt == 2 else 2):
        raise ValueError("dw and db overlap")
    n = 0
    if ws is not None:
        n = ws.numel()
        _need(ws, "ws", torch.float32)
    _here(dy, w, mean, rstd, dx, dw, db, ws)
    _check(lib().layer_norm_bwd(dy.data_ptr(), xp, cp, _TYPE[dy.dtype], _ptr(w), pt, mean.data_ptr(), rstd.data_ptr(),
                                rows, cols, _ptr(dx), pdw, pdb, _ptr(ws), n, _stream(stream)),
           "layer_norm_bwd")
