"""Refusals of the products with an epilogue, their backward pass and dropout, all
before any launch (no GPU needed): the C ABI's and the binding's."""
import ctypes
import os
import re

import pytest
import torch

import fp8_scaled_gemm_amd as F
from fp8_scaled_gemm_amd import epilogue as B
from fp8_scaled_gemm_amd import mx

OK, ENULL, ESHAPE, EALIGN, EFORMAT = 0, 1, 2, 3, 4
A = 0x10000  # fake addresses: validation fails before any use
BIG = (1 << 29) + 1
BF16, F16, F32 = 0, 1, 2
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8sg.h")
PAIR = mx._Pair(A, A)


FIELDS = (("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("pre", ctypes.c_void_p), ("rng", ctypes.c_void_p),
          ("ld_residual", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("p", ctypes.c_float), ("act", ctypes.c_int32),
          ("bias_type", ctypes.c_int32))


class Epilogue(ctypes.Structure):
    _fields_ = FIELDS


def E(**kw):
    e = Epilogue(ld_out=kw.pop("ld_out", 64), ld_residual=kw.pop("ld_residual", 64))
    for k, v in kw.items():
        setattr(e, k, v)
    return ctypes.byref(e)


def test_struct_layout_matches_header():
    body = re.search(r"typedef struct fp8sg_epilogue \{(.*?)\} fp8sg_epilogue;", open(HEADER).read(), re.S).group(1)
    c = {"const void*": ctypes.c_void_p, "void*": ctypes.c_void_p, "const int64_t*": ctypes.c_void_p,
         "int64_t": ctypes.c_int64, "float": ctypes.c_float, "int32_t": ctypes.c_int32}
    assert tuple((n, c[t]) for t, n in re.findall(r"^\s*([\w ]+\*?)\s(\w+);", body, re.M)) == FIELDS
    packed = B._pack(1, 2, 3, 4, 5, 6, 0.5, 7, 8)
    e = Epilogue.from_buffer_copy(packed)
    assert ctypes.sizeof(Epilogue) == len(packed) == 64
    assert [getattr(e, n) for n, _ in FIELDS] == [1, 2, 3, 4, 5, 6, 0.5, 7, 8]


BAD = [  # of a 32 x 64 bf16 result
    (dict(act=-1), EFORMAT), (dict(act=5), EFORMAT), (dict(bias=A, bias_type=3), EFORMAT),
    (dict(ld_out=63), ESHAPE), (dict(ld_out=1 << 40), ESHAPE), (dict(residual=A, ld_residual=63), ESHAPE),
    (dict(residual=A + 1), EALIGN), (dict(pre=A + 1), EALIGN), (dict(bias=A + 2, bias_type=F32), EALIGN),
    (dict(residual=A, ld_residual=128), ESHAPE),  # the output itself with other rows
    (dict(p=-0.1), ESHAPE), (dict(p=1.1), ESHAPE), (dict(p=float("nan")), ESHAPE),
    (dict(p=0.5), ENULL), (dict(p=0.5, rng=A + 4), EALIGN)]


@pytest.mark.parametrize("kw,status", BAD)
def test_epilogue_validation(kw, status):
    L, sv = F.lib(), F._Saved(*[A] * 6)
    ws, ls = mx._LinWs(*[PAIR] * 4), ctypes.byref(sv)
    p = ctypes.addressof(PAIR)
    assert L.fp8_gemm_epilogue(A, A, A, A, E(**kw), A, BF16, 32, 64, 64, None) == status
    assert L.fp8_gemm_rowwise_epilogue(A, A, A, A, E(**kw), A, BF16, 32, 64, 64, None) == status
    assert L.fp8_scaled_linear_fwd_epilogue(A, A, BF16, 32, 64, 64, ls, E(**kw), A, BF16, None) == status
    assert L.mxfp4_gemm_epilogue(p, p, E(**kw), A, BF16, 32, 64, 64, None) == status
    assert L.mxfp4_linear_fwd_epilogue(A, A, BF16, 32, 64, 64, 0, ctypes.byref(ws), None, E(**kw), A, BF16, None) == status
    assert L.mxfp4_linear_apply_epilogue(A, BF16, p, 32, 64, 64, 0, p, E(**kw), A, BF16, None) == status


def test_forward_validation():
    L, sv, p = F.lib(), ctypes.byref(F._Saved(*[A] * 6)), ctypes.addressof(PAIR)
    g = L.fp8_gemm_epilogue
    assert g(A, A, A, A, None, A, BF16, 32, 64, 64, None) == ENULL
    assert g(None, A, A, A, E(), A, BF16, 32, 64, 64, None) == ENULL
    assert g(A, A, None, A, E(), A, BF16, 32, 64, 64, None) == ENULL
    assert g(A, A, A, A, E(), None, BF16, 32, 64, 64, None) == ENULL
    assert g(A, A, A, A, E(), A, 3, 32, 64, 64, None) == EFORMAT
    assert g(A, A, A, A, E(), A, BF16, 33, 64, 64, None) == ESHAPE
    assert g(A, A, A, A, E(), A, BF16, -32, 64, 64, None) == ESHAPE
    assert g(A + 8, A, A, A, E(), A, BF16, 32, 64, 64, None) == EALIGN
    assert g(A, A, A + 4, A, E(), A, BF16, 32, 64, 64, None) == EALIGN
    assert g(A, A, A, A, E(), A + 1, BF16, 32, 64, 64, None) == EALIGN
    f = L.fp8_scaled_linear_fwd_epilogue
    assert f(A, A, F32, 32, 64, 64, sv, E(), A, BF16, None) == EFORMAT
    assert f(A, A, BF16, 0, 64, 64, sv, E(), A, BF16, None) == ESHAPE
    assert f(A, A, BF16, 32, 64, 40, sv, E(), A, BF16, None) == ESHAPE
    assert f(A, A, BF16, 32, 64, 64, None, E(), A, BF16, None) == ENULL
    assert f(A, None, BF16, 32, 64, 64, sv, E(), A, BF16, None) == ENULL
    assert f(A + 2, A, BF16, 32, 64, 64, sv, E(), A, BF16, None) == EALIGN
    assert f(A, A, BF16, 32, 64, 64, sv, E(bias=A, bias_type=F16), A, BF16, None) == EFORMAT
    assert L.mxfp4_gemm_epilogue(None, p, E(), A, BF16, 32, 64, 64, None) == ENULL
    assert L.mxfp4_gemm_epilogue(p, p, E(), A, BF16, 32, BIG, 64, None) == ESHAPE
    assert L.mxfp4_linear_apply_epilogue(A, 5, p, 32, 64, 64, 0, p, E(), A, BF16, None) == EFORMAT
    assert L.mxfp4_linear_apply_epilogue(A, BF16, p, 32, 64, 64, 9, p, E(), A, BF16, None) == EFORMAT


def test_backward_validation():
    L = F.lib()
    b = L.epilogue_bwd
    n = L.epilogue_workspace_len(4096, 64)
    assert n > 0 and L.epilogue_workspace_len(1, 64) == 0 and L.epilogue_workspace_len(0, 0) == 0
    assert L.epilogue_workspace_len(-1, 4) == L.epilogue_workspace_len(BIG, 4) == -1
    full = (4096, 64, A, A, A, n, None)
    assert b(A, BF16, None, *full) == ENULL
    assert b(None, BF16, E(), *full) == ENULL
    assert b(A, 3, E(), *full) == EFORMAT
    assert b(A, BF16, E(act=7), *full) == EFORMAT
    assert b(A, BF16, E(act=1), *full) == ENULL  # no pre
    assert b(A, BF16, E(bias_type=F16), *full) == EFORMAT
    assert b(A, BF16, E(p=0.5), *full) == ENULL
    assert b(A, BF16, E(), 4096, 64, None, None, None, 0, None) == ENULL
    assert b(A, BF16, E(), 4096, 64, A, A, None, 0, None) == ENULL
    assert b(A, BF16, E(), 4096, 64, A, A, A, n - 1, None) == ESHAPE
    assert b(A, BF16, E(), 4096, 64, A, A, A + 2, n, None) == EALIGN
    assert b(A, BF16, E(), -1, 64, A, A, A, n, None) == ESHAPE
    assert b(A + 1, BF16, E(), *full) == EALIGN
    sv, ws = ctypes.byref(F._Saved(*[A] * 6)), F._BwdWs(A, A, A)
    f = L.fp8_scaled_linear_bwd_epilogue
    tail = (A, A, A, n, A, A, BF16, None)
    dims = (4096, 64, 64)
    assert f(A, F32, sv, *dims, ctypes.byref(ws), E(), *tail) == EFORMAT
    assert f(A, BF16, None, *dims, ctypes.byref(ws), E(), *tail) == ENULL
    assert f(A, BF16, sv, *dims, None, E(), *tail) == ENULL
    assert f(A, BF16, sv, 4096, 64, 30, ctypes.byref(ws), E(), *tail) == ESHAPE
    assert f(A + 4, BF16, sv, *dims, ctypes.byref(ws), E(), *tail) == EALIGN
    assert f(A, BF16, sv, *dims, ctypes.byref(ws), E(act=1, pre=A), None, A, A, n, A, A, BF16, None) == ENULL
    assert f(A, BF16, sv, *dims, ctypes.byref(ws), E(), A, A, A, n, None, A, BF16, None) == ENULL
    assert f(A, BF16, sv, *dims, ctypes.byref(ws), E(), A, A, A, n, A, A, 4, None) == EFORMAT
    g = L.mxfp4_linear_bwd_epilogue
    mws, msv = mx._LinWs(*[PAIR] * 4), mx._LinSaved(PAIR, PAIR)
    w, s = ctypes.byref(mws), ctypes.byref(msv)
    assert g(A, BF16, *dims, 0, w, s, E(), A, None, None, 0, None, None, BF16, None) == ENULL
    assert g(A, BF16, *dims, 0, None, s, E(), *tail) == ENULL
    assert g(A, BF16, *dims, 2, w, s, E(), *tail) == EFORMAT
    assert g(A, BF16, *dims, 0, w, s, E(act=1, pre=A), None, A, A, n, A, A, BF16, None) == ENULL
    assert g(A, BF16, 4096, 64, BIG, 0, w, s, E(), *tail) == ESHAPE


def test_dropout_validation():
    L = F.lib()
    f, b = L.dropout_fwd, L.dropout_bwd
    assert f(A, 64, None, 0, 3, 32, 64, 0.5, A, A, 64, None) == EFORMAT
    assert f(None, 64, None, 0, 0, 32, 64, 0.5, A, A, 64, None) == ENULL
    assert f(A, 64, None, 0, 0, 32, 64, 0.5, A, None, 64, None) == ENULL
    assert f(A, 64, None, 0, 0, 32, 64, 0.5, None, A, 64, None) == ENULL
    assert f(A, 63, None, 0, 0, 32, 64, 0.5, A, A, 64, None) == ESHAPE
    assert f(A, 64, A, 63, 0, 32, 64, 0.5, A, A, 64, None) == ESHAPE
    assert f(A, 64, None, 0, 0, 32, 64, 0.5, A, A, 65, None) == ESHAPE  # x itself with other rows
    assert f(A, 64, None, 0, 0, 32, BIG, 0.5, A, A, BIG, None) == ESHAPE
    assert f(A, 64, None, 0, 0, 32, 64, 1.5, A, A, 64, None) == ESHAPE
    assert f(A, 64, None, 0, 2, 32, 64, 0.5, A, A + 2, 64, None) == EALIGN
    assert f(A, 64, None, 0, 0, 32, 64, 0.5, A + 4, A, 64, None) == EALIGN
    assert f(None, 0, None, 0, 0, 0, 64, 0.5, A, None, 0, None) == OK  # empty
    assert b(None, 64, 0, 32, 64, 0.5, A, A, 64, None) == ENULL


def raises(kind, fn, *args, match=None, **kw):
    with pytest.raises(kind, match=match):
        fn(*args, **kw)


def reaches_device(fn, *args, **kw):
    """Nothing is wrong but that the tensors are the host's."""
    with pytest.raises((ValueError, RuntimeError), match="device tensors|GPU|HIP"):
        fn(*args, **kw)


def test_binding_refusals():
    """dtypes, shapes, strides and overlaps, before a device is asked for."""
    bf = torch.bfloat16
    y, b = torch.zeros(32, 64, dtype=bf), torch.zeros(64, dtype=bf)

    def ep(y=y, in_dtype=bf, bias=None, act=0, residual=None, pre=None, p=0.0, rng=None):
        return B._epilogue(y, (32, 64), 32, 64, in_dtype, bias, act, residual, pre, p, rng)
    raises(TypeError, ep, bias=b.half(), match="bias")
    raises(TypeError, ep, bias=[0.0], match="bias")
    raises(ValueError, ep, bias=torch.zeros(63, dtype=bf), match="bias")
    raises(ValueError, ep, bias=torch.zeros(128, dtype=bf)[::2], match="bias")
    raises(ValueError, ep, act=9)
    raises(ValueError, ep, act="gelu")
    raises(TypeError, ep, residual=y.float(), match="residual")
    raises(ValueError, ep, residual=torch.zeros(32, 128, dtype=bf)[:, ::2], match="residual")
    raises(ValueError, ep, residual=y[:, :32], match="residual")
    raises(ValueError, ep, residual=b.expand(32, 64), match="residual")
    raises(ValueError, ep, y=torch.zeros(64, 32, dtype=bf).t())
    raises(ValueError, ep, pre=torch.zeros(32, 128, dtype=bf)[:, :64], match="pre")
    raises(TypeError, ep, pre=y.float(), match="pre")
    raises(ValueError, ep, pre=y, match="overlap")
    raises(ValueError, ep, pre=y.clone(), p=0.5, match="rng")
    raises(ValueError, ep, p=1.5)
    raises(ValueError, ep, p=float("nan"))
    raises(TypeError, ep, p=0.5, rng=torch.zeros(2))
    raises(ValueError, ep, p=0.5, rng=torch.zeros(3, dtype=torch.int64))
    wide = torch.zeros(33 * 64, dtype=bf)
    raises(ValueError, ep, y=wide[:2048].view(32, 64), residual=wide[64:].view(32, 64), match="overlap")
    half = torch.zeros(32, 100, dtype=bf)
    raises(ValueError, ep, y=half[:, :64], residual=half[:, 36:], match="overlap")
    r = torch.zeros(32, 64, dtype=bf)
    raises(ValueError, ep, residual=r, pre=r, match="overlap")
    reaches_device(ep)  # all is well but the device
    reaches_device(ep, residual=y)  # in place
    two = torch.zeros(32, 128, dtype=bf)
    reaches_device(ep, y=two[:, :64], residual=two[:, 64:])  # halves of one matrix


def test_binding_backward_refusals():
    bf = torch.bfloat16
    gy = torch.zeros(32, 64, dtype=bf)

    def bw(gh=None, gb=None, pre=None, act=0, p=0.0, rng=None, part=None, alone=False):
        return B._backward(gy, gh, gb, pre, act, p, rng, part, 32, 64, alone)
    raises(ValueError, bw, act=F.ACT_RELU, pre=gy.clone(), match="gh")
    raises(ValueError, bw, gh=gy.clone(), act=F.ACT_RELU, match="pre")
    raises(TypeError, bw, gh=gy.float(), match="gh")
    raises(ValueError, bw, gh=gy[:16], match="gh")
    raises(TypeError, bw, gb=torch.zeros(64, dtype=torch.float16), match="gb")
    raises(TypeError, bw, gb=3, match="gb")
    raises(ValueError, bw, gb=torch.zeros(32, dtype=bf), match="gb")
    raises(ValueError, bw, gb=gy[0], match="overlap")
    raises(TypeError, bw, gb=torch.zeros(64, dtype=bf), part=torch.zeros(64, dtype=bf), match="part")
    pre = gy.clone()
    raises(ValueError, bw, gh=pre, pre=pre, act=F.ACT_RELU, match="overlap")
    big = torch.zeros(33 * 64, dtype=bf)
    gy2 = big[:2048].view(32, 64)
    with pytest.raises(ValueError, match="overlap"):
        B._backward(gy2, big[64:].view(32, 64), None, None, 0, 0.0, None, None, 32, 64, True)
    reaches_device(bw, gh=gy)  # in place


def test_calls_refuse_mismatched_operands():
    bf = torch.bfloat16
    x, w, y = torch.zeros(32, 64, dtype=bf), torch.zeros(48, 64, dtype=bf), torch.zeros(32, 48, dtype=bf)
    saved = F.LinearSaved(32, 48, 64, device="cpu")
    f = F.fp8_scaled_linear_fwd_epilogue
    raises(TypeError, f, x.float(), w.float(), saved, y)
    raises(TypeError, f, x, w.half(), saved, y)
    raises(ValueError, f, x, w[:, :32].contiguous(), saved, y)
    raises(ValueError, f, x, w, saved, y[:, :32])
    raises(TypeError, f, x, w, None, y)
    raises(ValueError, F.epilogue_bwd, y)
    raises(ValueError, F.dropout_fwd, x, 0.5, None, x.clone())
    raises(ValueError, F.dropout_fwd, x, -0.5, None, x.clone())
    raises(TypeError, F.dropout_fwd, x, 0.5, None, x.float())
    raises(ValueError, F.dropout_fwd, x, 0.0, None, x[:16])
    raises(ValueError, F.dropout_fwd, torch.zeros((), dtype=bf), 0.0, None, torch.zeros((), dtype=bf))
    raises(TypeError, F.dropout_fwd, x.int(), 0.0, None, x.int())
    reaches_device(F.dropout_fwd, x, 0.0, None, x)
    wide = torch.zeros(33 * 64, dtype=bf)
    raises(ValueError, F.dropout_fwd, wide[:2048].view(32, 64), 0.0, None, wide[64:].view(32, 64), match="overlap")
    raises(ValueError, F.dropout_bwd, wide[:2048].view(32, 64), 0.0, None, wide[64:].view(32, 64), match="overlap")
    q = F.Mxfp4(48, 64, device="cpu")
    raises(ValueError, F.mxfp4_linear_apply_epilogue, x, F.Mxfp4(48, 32, device="cpu"), y, F.Mxfp4(32, 64, device="cpu"))
    raises(TypeError, F.mxfp4_gemm_epilogue, q, None, y)
    raises(ValueError, F.mxfp4_gemm_epilogue, q, q, y)
    msv = F.Mxfp4LinearSaved(32, 48, 64, "cpu")
    mws = F.Mxfp4LinearWs(32, 48, 64, "cpu")
    raises(ValueError, F.mxfp4_linear_bwd_epilogue, y, mws, msv, None, None)
    raises(ValueError, F.mxfp4_linear_bwd_epilogue, y, mws, msv, y[:, :8], None)
