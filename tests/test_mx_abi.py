"""Refusals of the MXFP4, checkpoint, gated-activation and layer-norm entry
points, all before any launch (no GPU needed), and the reference's own rounding."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from fp8_scaled_gemm_amd import mx
from tests import mx_reference as R

OK, ENULL, ESHAPE, EALIGN, EFORMAT = 0, 1, 2, 3, 4
A = 0x10000  # fake addresses: validation fails before any use
BIG = (1 << 29) + 1
PAIR = mx._Pair(A, A)
NOPAIR = mx._Pair(None, None)
OFFPAIR = mx._Pair(A + 8, A)


def P(s):
    return ctypes.addressof(s)


def test_sizes():
    L = F.lib()
    for rows, k in ((0, 0), (1, 1), (1, 256), (3, 257), (128, 512), (129, 100), (14336, 4096)):
        nk = -(-k // 256)
        assert L.mxfp4_code_bytes(rows, k) == rows * 128 * nk
        assert L.mxfp4_scale_bytes(rows, k) == -(-rows // 32) * nk * 256
    for bad in ((-1, 4), (4, -1), (BIG, 1), (1, BIG), (1 << 20, 1 << 20)):
        assert L.mxfp4_code_bytes(*bad) == -1 and L.mxfp4_scale_bytes(*bad) == -1
        assert L.layer_norm_workspace_len(*bad) == -1


def test_mxfp4_validation():
    L, p = F.lib(), P(PAIR)
    assert L.mxfp4_quantize(A, 0, 4, 64, 0, None, None, None) == ENULL
    assert L.mxfp4_quantize(None, 0, 4, 64, 0, p, None, None) == ENULL
    assert L.mxfp4_quantize(A, 3, 4, 64, 0, p, None, None) == EFORMAT
    assert L.mxfp4_quantize(A, 0, 4, 64, 2, p, None, None) == EFORMAT
    assert L.mxfp4_quantize(A, 0, -4, 64, 0, p, None, None) == ESHAPE
    assert L.mxfp4_quantize(A, 0, 4, BIG, 0, p, None, None) == ESHAPE
    assert L.mxfp4_quantize(A + 1, 0, 4, 64, 0, p, None, None) == EALIGN
    assert L.mxfp4_quantize(A + 2, 2, 4, 64, 0, p, None, None) == EALIGN
    assert L.mxfp4_quantize(A, 0, 4, 64, 0, P(NOPAIR), None, None) == ENULL
    assert L.mxfp4_quantize(A, 0, 4, 64, 0, p, P(OFFPAIR), None) == EALIGN
    assert L.mxfp4_dequantize(None, 4, 64, A, 0, None) == ENULL
    assert L.mxfp4_dequantize(p, 4, 64, None, 0, None) == ENULL
    assert L.mxfp4_dequantize(p, 4, 64, A, 7, None) == EFORMAT
    assert L.mxfp4_dequantize(p, 4, -1, A, 0, None) == ESHAPE
    assert L.mxfp4_dequantize(P(OFFPAIR), 4, 64, A, 0, None) == EALIGN
    assert L.mxfp4_gemm(None, p, A, 0, 4, 4, 64, None) == ENULL
    assert L.mxfp4_gemm(p, p, None, 0, 4, 4, 64, None) == ENULL
    assert L.mxfp4_gemm(p, p, A, -1, 4, 4, 64, None) == EFORMAT
    assert L.mxfp4_gemm(p, p, A, 0, 1 << 20, 1 << 20, 64, None) == ESHAPE
    assert L.mxfp4_gemm(p, p, A, 0, 4, 4, -64, None) == ESHAPE
    assert L.mxfp4_gemm(p, p, A + 2, 2, 4, 4, 64, None) == EALIGN
    assert L.mxfp4_linear_apply(A, 0, None, 1, 4, 64, 0, p, A, 0, None) == ENULL
    assert L.mxfp4_linear_apply(A, 0, p, 1, 4, 64, 0, None, A, 0, None) == ENULL
    assert L.mxfp4_linear_apply(A, 0, p, 1, 4, 64, 9, p, A, 0, None) == EFORMAT
    assert L.mxfp4_linear_apply(A, 0, p, 1, -4, 64, 0, p, A, 0, None) == ESHAPE
    assert L.mxfp4_linear_apply(A, 0, P(OFFPAIR), 1, 4, 64, 0, p, A, 0, None) == EALIGN


def test_linear_validation():
    L = F.lib()
    ws, sv = mx._LinWs(PAIR, PAIR, PAIR, PAIR), mx._LinSaved(PAIR, PAIR)
    assert L.mxfp4_linear_fwd(A, A, 0, 4, 4, 64, 0, None, None, A, 0, None) == ENULL
    assert L.mxfp4_linear_fwd(A, None, 0, 4, 4, 64, 0, P(ws), None, A, 0, None) == ENULL
    assert L.mxfp4_linear_fwd(A, A, 5, 4, 4, 64, 0, P(ws), None, A, 0, None) == EFORMAT
    assert L.mxfp4_linear_fwd(A, A, 0, 4, 4, 64, 3, P(ws), None, A, 0, None) == EFORMAT
    assert L.mxfp4_linear_fwd(A, A, 0, 4, 4, 64, 0, P(ws), None, A, 3, None) == EFORMAT
    assert L.mxfp4_linear_fwd(A, A, 0, 4, BIG, 64, 0, P(ws), None, A, 0, None) == ESHAPE
    assert L.mxfp4_linear_fwd(A, A, 0, 4, 4, 64, 0, P(ws), P(mx._LinSaved(PAIR, NOPAIR)), A, 0, None) == ENULL
    assert L.mxfp4_linear_fwd(A, A, 0, 4, 4, 64, 0, P(mx._LinWs(OFFPAIR, PAIR, PAIR, PAIR)), None, A, 0, None) == EALIGN
    assert L.mxfp4_linear_fwd(A, A, 0, 4, 4, 64, 0, P(ws), P(sv), None, 0, None) == ENULL
    assert L.mxfp4_linear_bwd(A, 0, 4, 4, 64, 0, P(ws), None, A, A, 0, None) == ENULL
    assert L.mxfp4_linear_bwd(A, 0, 4, 4, 64, 0, P(ws), P(sv), None, None, 0, None) == ENULL
    assert L.mxfp4_linear_bwd(A, 0, 4, 4, 64, 0, P(ws), P(sv), A, A + 1, 0, None) == EALIGN
    assert L.mxfp4_linear_bwd(A, 0, 4, 4, 64, 0, P(mx._LinWs(PAIR, PAIR, PAIR, NOPAIR)), P(sv), A, A, 0, None) == ENULL
    assert L.mxfp4_linear_bwd(A, 0, -4, 4, 64, 0, P(ws), P(sv), A, A, 0, None) == ESHAPE
    # both gradients are empty (and so NULL): nothing is enqueued, gy is not cast either
    assert L.mxfp4_linear_bwd(A, 0, 4, 4, 0, 0, P(ws), P(sv), None, None, 0, None) == OK


def test_swiglu_and_checkpoint_validation():
    L, p = F.lib(), P(PAIR)
    assert L.act8_quantize(A, 0, 4, 64, None, None) == ENULL
    assert L.act8_quantize(None, 0, 4, 64, p, None) == ENULL
    assert L.act8_quantize(A, 3, 4, 64, p, None) == EFORMAT
    assert L.act8_quantize(A, 0, 4, -64, p, None) == ESHAPE
    assert L.act8_quantize(A, 0, 4, 64, P(OFFPAIR), None) == EALIGN
    assert L.act8_dequantize(p, 4, 64, None, 0, None) == ENULL
    assert L.act8_dequantize(p, 4, 64, A + 1, 0, None) == EALIGN
    assert L.swiglu_fwd(A, 64, A, 64, 3, 4, 64, A, None, None, None) == EFORMAT
    assert L.swiglu_fwd(A, 63, A, 64, 0, 4, 64, A, None, None, None) == ESHAPE
    assert L.swiglu_fwd(A, 64, A, BIG, 0, 4, 64, A, None, None, None) == ESHAPE
    assert L.swiglu_fwd(None, 64, A, 64, 0, 4, 64, A, None, None, None) == ENULL
    assert L.swiglu_fwd(A, 64, A, 64, 0, 4, 64, A, p, None, None) == ENULL
    assert L.swiglu_fwd(A, 64, A, 64, 0, 4, 64, A, P(NOPAIR), p, None) == ENULL
    assert L.swiglu_fwd(A, 64, A + 1, 64, 0, 4, 64, A, None, None, None) == EALIGN
    assert L.swiglu_bwd(A, A, 64, None, 64, None, None, 0, 4, 64, A, 64, A, 64, None) == ENULL
    assert L.swiglu_bwd(A, None, 0, None, 0, None, p, 0, 4, 64, A, 64, A, 64, None) == ENULL
    assert L.swiglu_bwd(A, None, 0, None, 0, p, p, 0, 4, 64, A, 32, A, 64, None) == ESHAPE
    assert L.swiglu_bwd(A, None, 0, None, 0, p, p, 0, 4, 64, A, 64, None, 64, None) == ENULL
    assert L.swiglu_bwd(A, None, 0, None, 0, p, P(OFFPAIR), 0, 4, 64, A, 64, A, 64, None) == EALIGN


def test_layer_norm_validation():
    L, p = F.lib(), P(PAIR)

    def fwd(x=A, t=0, w=A, b=A, pt=0, rows=4, cols=64, eps=1e-5, y=A, mean=A, rstd=A, c=None):
        return L.layer_norm_fwd(x, t, w, b, pt, rows, cols, eps, y, mean, rstd, c, None)
    assert fwd(x=None) == ENULL and fwd(y=None) == ENULL and fwd(rstd=None) == ENULL
    assert fwd(t=3) == EFORMAT and fwd(pt=1) == EFORMAT and fwd(t=2, pt=0) == EFORMAT
    assert fwd(cols=0) == ESHAPE and fwd(rows=-1) == ESHAPE and fwd(eps=-1.0) == ESHAPE and fwd(eps=float("nan")) == ESHAPE
    assert fwd(w=A + 1) == EALIGN and fwd(mean=A + 2) == EALIGN and fwd(c=P(OFFPAIR)) == EALIGN
    assert fwd(pt=2, b=A + 2) == EALIGN and fwd(c=P(NOPAIR)) == ENULL

    need = L.layer_norm_workspace_len(4, 64)

    def bwd(dy=A, x=A, c=None, t=0, w=A, pt=0, mean=A, rstd=A, rows=4, cols=64, dx=A, dw=A, db=A, ws=A, n=need):
        return L.layer_norm_bwd(dy, x, c, t, w, pt, mean, rstd, rows, cols, dx, dw, db, ws, n, None)
    assert bwd(dy=None) == ENULL and bwd(x=None) == ENULL and bwd(c=p) == ENULL and bwd(mean=None) == ENULL
    assert bwd(ws=None) == ENULL and bwd(n=need - 1) == ESHAPE and bwd(cols=0) == ESHAPE
    assert bwd(t=4) == EFORMAT and bwd(pt=1) == EFORMAT
    assert bwd(dw=A + 1) == EALIGN and bwd(x=None, c=P(OFFPAIR)) == EALIGN and bwd(ws=A + 4) == EALIGN


def test_binding_refuses_mismatches_before_any_call():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="needed"):
        F.mxfp4_quantize(x)
    with pytest.raises(TypeError, match="Mxfp4"):
        F.mxfp4_quantize(x, x)
    with pytest.raises(ValueError, match="expected 64 x 4"):
        F.mxfp4_quantize(x, qT=F.Mxfp4(4, 64, device="cpu"))
    with pytest.raises(TypeError, match="dtype"):
        F.mxfp4_quantize(x.int(), F.Mxfp4(4, 64, device="cpu"))
    with pytest.raises(ValueError, match="contiguous"):
        F.mxfp4_quantize(x.t(), F.Mxfp4(64, 4, device="cpu"))
    with pytest.raises(ValueError, match="expected 5 x 64"):
        F.mxfp4_gemm(F.Mxfp4(4, 64, device="cpu"), F.Mxfp4(6, 64, device="cpu"), torch.zeros(4, 5))
    with pytest.raises(ValueError, match="size limits"):
        F.Mxfp4(-1, 5, device="cpu")
    with pytest.raises(ValueError, match="shape"):
        F.Act8(4, 40, tensors=(torch.zeros(4, 40, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)))
    with pytest.raises(ValueError, match="elements"):
        F.Mxfp4(4, 40, tensors=(torch.zeros(4, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8)))


def test_outputs_that_would_be_one_buffer_are_refused():
    x, m, c = torch.zeros(64, 64), F.Mxfp4(64, 64, device="cpu"), F.Act8(64, 64, device="cpu")
    with pytest.raises(ValueError, match="each needs its own"):
        F.mxfp4_quantize(x, m, m)
    with pytest.raises(ValueError, match="a checkpoint each"):
        mx._ckpts(c, c, 64, 64, True)


@pytest.mark.parametrize("call", [
    lambda x: F.mxfp4_quantize(x, F.Mxfp4(4, 64, device="cpu")),
    lambda x: F.mxfp4_dequantize(F.Mxfp4(4, 64, device="cpu"), x),
    lambda x: F.mxfp4_gemm(F.Mxfp4(4, 32, device="cpu"), F.Mxfp4(64, 32, device="cpu"), x),
    lambda x: F.act8_quantize(x, F.Act8(4, 64, device="cpu")),
    lambda x: F.swiglu_fwd(x, x, x.clone()),
    lambda x: F.layer_norm_fwd(x, None, None, 1e-5, x.clone()),
])
def test_host_tensors_are_refused(call):
    with pytest.raises((ValueError, RuntimeError, AssertionError)):  # without a GPU torch itself may refuse first
        call(torch.zeros(4, 64))


def test_operands_of_a_layer_lie_in_its_struct():
    """A layer's buffers reach the library at their present addresses, also after
    one was exchanged, and from an operand taken out of its layer."""
    for obj in (F.Mxfp4LinearSaved(40, 24, 70, "cpu"), F.Mxfp4LinearWs(40, 24, 70, "cpu", backward=False)):
        names = [n for n, _ in obj._all._fields_ if getattr(obj, n) is not None]
        getattr(obj, names[0]).q = torch.zeros_like(getattr(obj, names[0]).q)
        got = type(obj._all).from_address(obj.c())
        for n in names:
            m = getattr(obj, n)
            assert (getattr(got, n).q, getattr(got, n).s) == (m.q.data_ptr(), m.s.data_ptr())
        m = getattr(obj, names[1])
        del obj, got
        pair = mx._Pair.from_address(m.c())
        assert (pair.q, pair.s) == (m.q.data_ptr(), m.s.data_ptr())


def test_strided_rows():
    m = torch.zeros(6, 40)
    like = torch.zeros(6, 16)
    assert mx._strided(m[:, 8:24], "g", like, 6, 16) == 40
    assert mx._strided(like, "g", like, 6, 16) == 16
    assert mx._strided(torch.zeros(2, 3, 16), "g", like, 6, 16) == 16
    for bad in (m[:, 0:32:2], m.t()[:6, :].t()[:6], like.expand(6, 16)[:1].expand(6, 16)):
        with pytest.raises(ValueError):
            mx._strided(bad, "g", like, 6, 16)
    with pytest.raises(TypeError):
        mx._strided(like.half(), "g", like, 6, 16)


def test_build_reads_where_products_add():
    """The build's guard on the matrix instructions sees a result that moves."""
    from fp8_scaled_gemm_amd.build import moved_products
    asm = """_Zkern:
\tv_mfma_scale_f32_16x16x128_f8f6f4 v[4:7], v[14:17], v[50:53], v[4:7], v1, v136 op_sel_hi:[0,0,0] cbsz:4 blgp:4
.LBB0_1:
\tv_mfma_scale_f32_16x16x128_f8f6f4 v[4:7], v[14:17], v[50:53], v[6:9], v1, v136 op_sel_hi:[0,0,0] cbsz:4 blgp:4
_Zother:
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], 0
"""
    assert moved_products(asm) == {"_Zkern": 1, "_Zother": 1}


def test_reference_rounding():
    """Known roundings of the reference the GPU tests compare with."""
    v = np.zeros((1, 32))
    v[0, :8] = [6, 0.25, 0.75, 1.25, 2.5, 5, -3.5, -0.2]
    assert R.fp4_values(v, False)[0, :8].tolist() == [6, 0, 1, 1, 2, 4, -4, 0]
    v[0, 0] = 7.5  # floor: saturates; fit: the scale doubles
    assert R.fp4_values(v, False)[0, 0] == 6 and R.fp4_values(v, True)[0, 0] == 8
    assert R.fp4(np.zeros((1, 32)), False)[1][0, 0] == 0
    v[0, 0] = np.nan
    assert np.isnan(R.fp4_values(v, True)).all()
    a = np.zeros((1, 32))
    a[0, :4] = [448, 17, 2.0 ** -10, -3 * 2.0 ** -10]
    assert R.act8_values(a)[0, :4].tolist() == [448, 16, 0, -2.0 ** -8]
    assert len(R.E4M3) == 127 and R.E4M3[-1] == 448


def test_a_wanted_gradient_that_is_empty():
    """No rows, only gx wanted, or no outputs, only gw wanted: the gradient is empty
    and so NULL, which is no missing argument."""
    L = F.lib()
    ws, sv = mx._LinWs(PAIR, PAIR, PAIR, PAIR), mx._LinSaved(PAIR, PAIR)
    assert L.mxfp4_linear_bwd(None, 0, 0, 4, 64, 0, P(ws), P(sv), None, None, 0, None) == OK
    assert L.mxfp4_linear_bwd(None, 0, 4, 0, 64, 0, P(ws), P(sv), None, None, 0, None) == OK
    assert L.mxfp4_linear_bwd(A, 0, 4, 4, 64, 0, P(ws), P(sv), None, None, 0, None) == ENULL
    # the other sizes of such a call are still looked at
    assert L.mxfp4_linear_bwd(None, 3, 0, 4, 64, 0, P(ws), P(sv), None, None, 0, None) == EFORMAT
    assert L.mxfp4_linear_bwd(None, 0, 0, -4, 64, 0, P(ws), P(sv), None, None, 0, None) == ESHAPE
