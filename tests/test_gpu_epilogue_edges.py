"""Calls of the products with an epilogue at the edges of what they allow: offsets past
32 bits, rows apart and results in place in every FP8 tiling, empty batches, first
calls inside a capture, two graphs, unaligned vectors."""
import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as F
from fp8_scaled_gemm_amd import nn as N
from tests import epilogue_reference as E
from tests import mx_reference as R
from tests.test_gpu_epilogue import GUARD, fp8_product, mx_operands, rand, rng_words, tensors, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"


def keep_rows(rng, first, rows, cols, p):
    """E.keep of rows [first, first + rows) of a larger matrix."""
    g = -(-cols // 8)
    n = np.arange(first * g, (first + rows) * g, dtype=np.uint64)
    seed, off = (v % 2 ** 64 for v in rng)
    m = 0xFFFFFFFF
    ctr = np.stack([n & np.uint64(m), n >> np.uint64(32), np.full_like(n, off & m), np.full_like(n, off >> 32)], -1)
    w = E.philox(ctr, (seed & m, seed >> 32))
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(rows, 8 * g)[:, :cols]
    t = int(65536 * p + 0.5)
    return np.where(u >= t, 65536 / (65536 - t), 0.0)


def test_results_past_2_to_31_elements():
    M, N_, K = 33000, 65544, 32
    x, w = rand((M, K), "bf16", 1), rand((N_, K), "bf16", 2, 0.1)
    a, b = F.Mxfp4(M, K), F.Mxfp4(N_, K)
    F.mxfp4_quantize(x, a)
    F.mxfp4_quantize(w, b)
    bias, rng = rand((N_,), "bf16", 3), rng_words(4)
    y = torch.full((M, N_), 2.0, dtype=torch.bfloat16, device=DEV)
    pre = torch.empty_like(y)
    F.mxfp4_gemm_epilogue(a, b, y, bias=bias, act=F.ACT_RELU, residual=y, pre=pre, p=0.25, rng=rng)
    for first in (0, M - 3):  # the last rows lie past 2^31 elements
        rows = slice(first, first + 3)
        prod, err = R.dot(R.fp4_values(R.f64(x[rows]), False), R.fp4_values(R.f64(w), False))
        ref = {"bias": R.f64(bias), "residual": np.full((3, N_), 2.0),
               "factor": keep_rows(rng.tolist(), first, 3, N_, 0.25)}
        verify(y[rows], pre[rows], prod, err, F.ACT_RELU, ref, True, first)
    del y
    gy = torch.full((M, N_), 0.5, dtype=torch.bfloat16, device=DEV)
    F.epilogue_bwd(gy, gy, pre=pre, act=F.ACT_RELU, p=0.25, rng=rng)
    for first in (0, M - 3):
        want, err, _, _ = E.backward(np.full((3, N_), 0.5), R.f64(pre[first:first + 3]), E.RELU,
                                     keep_rows(rng.tolist(), first, 3, N_, 0.25), True)
        R.check(gy[first:first + 3], want, err, first)


# small layer in one launch, tiles of 64, 128, 256 and 224
@pytest.mark.parametrize("M,N_,K", [(64, 256, 128), (336, 528, 144), (2048, 2304, 144), (2880, 3104, 144),
                                    (3584, 4096, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_fp8_rows_apart_and_in_place(M, N_, K, dtype):
    x, w = rand((M, K), dtype, 1), rand((N_, K), dtype, 2, 0.1)
    saved = F.LinearSaved(M, N_, K, transposed=False)
    kw, ref = tensors(M, N_, dtype, "f32", True, 0.25, 3)
    t = R.DTYPES[dtype]
    first = None
    for off, ld in ((0, N_), (1, N_ + 3), (8, 2 * N_)):
        wide = torch.full((M + 2, ld + 16), GUARD, dtype=t, device=DEV)
        y = wide[1:M + 1, off:off + N_]
        res = torch.zeros(M, ld + 8, dtype=t, device=DEV)[:, off:off + N_]
        res.copy_(kw["residual"])
        F.fp8_scaled_linear_fwd_epilogue(x, w, saved, y, act=F.ACT_GELU, **{**kw, "residual": res})
        if first is None:
            first = y.clone()
            verify(first, None, *fp8_product(saved), F.ACT_GELU, ref, True, (M, N_, K))
        assert torch.equal(y, first)
        y.copy_(kw["residual"])
        F.fp8_scaled_linear_fwd_epilogue(x, w, saved, y, act=F.ACT_GELU, **{**kw, "residual": y})
        assert torch.equal(y, first)
        y.fill_(GUARD)
        assert (wide == GUARD).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_vectors_of_any_alignment(dtype):
    M, N_, K = 70, 333, 100
    _, _, a, b, (prod, err) = mx_operands(M, N_, K, 1)
    kw, ref = tensors(M, N_, dtype, dtype, True, 0.25, 2)
    y, want = (torch.empty(M, N_, dtype=R.DTYPES[dtype], device=DEV) for _ in range(2))
    F.mxfp4_gemm_epilogue(a, b, want, act=F.ACT_SILU, **kw)
    verify(want, None, prod, err, F.ACT_SILU, ref, dtype != "f32", "aligned")
    for off in (1, 3):
        bias = torch.zeros(N_ + 8, dtype=y.dtype, device=DEV)[off:off + N_]
        bias.copy_(kw["bias"])
        F.mxfp4_gemm_epilogue(a, b, y, act=F.ACT_SILU, **{**kw, "bias": bias})
        assert torch.equal(y, want)
        flat = torch.zeros(3, M * N_ + 8, dtype=y.dtype, device=DEV)
        gy, pre, gh = (flat[i, off:off + M * N_].view(M, N_) for i in range(3))
        gy.copy_(kw["residual"])
        pre.copy_(want)
        plain = torch.empty_like(y)
        gb, gb2 = torch.zeros(N_ + 8, dtype=y.dtype, device=DEV)[off:off + N_], torch.empty(N_, dtype=y.dtype, device=DEV)
        F.epilogue_bwd(gy, gh, gb, pre=pre, act=F.ACT_SILU)
        F.epilogue_bwd(kw["residual"], plain, gb2, pre=want, act=F.ACT_SILU)
        assert torch.equal(gh, plain) and torch.equal(gb, gb2)


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_empty_batches(act):
    m = N.MXFP4EpilogueLinear(40, 24, activation=act, dropout=0.5, device=DEV)
    torch.nn.init.normal_(m.weight)
    torch.nn.init.normal_(m.bias)
    x = torch.zeros(0, 40, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    res = torch.zeros(0, 24, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    y = m(x, res)
    assert y.shape == (0, 24)
    y.sum().backward()
    assert x.grad.shape == (0, 40) and (m.weight.grad == 0).all() and (m.bias.grad == 0).all()
    p = N.PackedMXFP4EpilogueLinear.from_float(m)
    assert p(x.detach()).shape == (0, 24)
    d = N.Dropout(0.5)
    e = torch.zeros(3, 0, device=DEV, requires_grad=True)
    d(e, e).sum().backward()
    assert e.grad.shape == (3, 0)


def test_calls_first_used_in_a_capture_and_two_graphs():
    """A kernel's first launch inside a capture; two graphs of one layer with buffers of
    their own, replayed in turns."""
    M, N_, K = 200, 264, 640
    x, w, _, b, (prod, err) = mx_operands(M, N_, K, 7, dtype="f16")
    kw, ref = tensors(M, N_, "f16", "f16", True, 0.5, 4)
    outs, graphs = [], []
    for act in (F.ACT_GELU_TANH, F.ACT_RELU):
        y = torch.zeros(M, N_, dtype=torch.float16, device=DEV)
        ws = F.Mxfp4(M, K)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            F.mxfp4_linear_apply_epilogue(x, b, y, ws, act=act, **kw)
        outs.append((act, y))
        graphs.append(g)
    for k in range(4):
        for g in graphs if k % 2 else graphs[::-1]:
            g.replay()
        for act, y in outs:
            verify(y, None, prod, err, act, ref, True, act)
            y.zero_()


def test_two_streams_at_once():
    """Calls of one operator on two streams, with buffers of their own."""
    M, N_ = 3000, 1031
    gy, pre = rand((M, N_), "bf16", 1), rand((M, N_), "bf16", 2)

    def buffers():
        return (torch.empty_like(gy), torch.empty(N_, device=DEV), torch.empty(F.epilogue_workspace_len(M, N_), device=DEV))
    want = buffers()
    F.epilogue_bwd(gy, want[0], want[1], pre=pre, act=F.ACT_GELU, part=want[2])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (gh, gb, part) in zip(streams, got):
            F.epilogue_bwd(gy, gh, gb, pre=pre, act=F.ACT_GELU, part=part, stream=s)
    torch.cuda.synchronize()
    for gh, gb, _ in got:
        assert torch.equal(gh, want[0]) and torch.equal(gb, want[1])


def test_the_same_tensor_twice():
    """Inputs may share memory: gy is also h, the residual is also x."""
    gy = rand((48, 64), "bf16", 1)
    gh, want = torch.empty_like(gy), torch.empty_like(gy)
    F.epilogue_bwd(gy, gh, pre=gy, act=F.ACT_GELU)
    F.epilogue_bwd(gy, want, pre=gy.clone(), act=F.ACT_GELU)
    assert torch.equal(gh, want)
    with pytest.raises(ValueError, match="overlap"):
        F.epilogue_bwd(gy, gy, pre=gy, act=F.ACT_GELU)
    w = rand((64, 64), "bf16", 2, 0.1)
    saved = F.LinearSaved(48, 64, 64)
    y, y2 = torch.empty_like(gy), torch.empty_like(gy)
    F.fp8_scaled_linear_fwd_epilogue(gy, w, saved, y, residual=gy)
    F.fp8_scaled_linear_fwd_epilogue(gy, w, saved, y2, residual=gy.clone())
    assert torch.equal(y, y2)
    x = rand((48, 64), "bf16", 3)
    a, b = torch.empty_like(x), torch.empty_like(x)
    rng = rng_words(1)
    F.dropout_fwd(x, 0.5, rng, a, residual=x)
    F.dropout_fwd(x, 0.5, rng, b, residual=x.clone())
    assert torch.equal(a, b)


@pytest.mark.parametrize("M,N_,dtype", [(64, 256, "f32"), (63, 255, "f16"), (257, 1000, "bf16"), (4100, 520, "f16"),
                                        (1, 8200, "bf16"), (65536, 40, "bf16"), (65537, 40, "bf16"), (300, 72, "f32"),
                                        (9100, 4232, "bf16")])
def test_mx_backward_in_one_pass_or_two(M, N_, dtype):
    """gh, its codes and gb of one pass, or past 65536 rows of two, are those of the
    step and the plain backward pass one after the other; all kinds, and in place."""
    K = 40
    x, w = rand((M, K), dtype, 1), rand((N_, K), dtype, 2, 0.05)
    gy, pre, rng = rand((M, N_), dtype, 3, 0.1), rand((M, N_), dtype, 4, 2.0), rng_words(5)
    gy.view(-1)[0] = float("inf")
    ws, saved = F.Mxfp4LinearWs(M, N_, K), F.Mxfp4LinearSaved(M, N_, K)
    F.mxfp4_linear_fwd(x, w, ws, saved, torch.empty(M, N_, dtype=gy.dtype, device=DEV))
    part = torch.full((F.epilogue_workspace_len(M, N_) + 5,), GUARD, device=DEV)
    new = lambda *s: torch.full(s, GUARD, dtype=gy.dtype, device=DEV)  # noqa: E731
    for act, p in ((F.ACT_GELU, 0.25), (F.ACT_RELU, 0.0), (F.ACT_NONE, 0.5), (F.ACT_GELU_TANH, 1.0)):
        kw = {"pre": pre if act else None, "act": act, "p": p, "rng": rng if p else None, "part": part}
        gh, gb = torch.empty_like(gy), torch.empty(N_, device=DEV)
        F.epilogue_bwd(gy, gh, gb, **kw)
        for kinds in ("xwb", "xw", "xb", "w"):
            gx, gw = (new(M, K) if "x" in kinds else None), (new(N_, K) if "w" in kinds else None)
            want = [None if g is None else torch.empty_like(g) for g in (gx, gw)]
            F.mxfp4_linear_bwd(gh, ws, saved, *want)
            b = new(N_).float() if "b" in kinds else None
            gh2 = gy.clone() if kinds == "xb" else new(M, N_)  # (in place)
            ws.gy_q.q.fill_(255), ws.gy_qT.q.fill_(255)
            F.mxfp4_linear_bwd_epilogue(gh2 if kinds == "xb" else gy, ws, saved, gx, gw, gh=gh2, gb=b, **kw)
            assert torch.equal(gh2.view(torch.uint8), gh.view(torch.uint8)), (act, kinds)
            for got, ref in ((gx, want[0]), (gw, want[1])):
                assert got is None or torch.equal(got.view(torch.uint8), ref.view(torch.uint8)), (act, kinds)
            if b is not None:
                # each of the two orders rounds M times, by 2^-24 of the magnitudes' sum at
                # most; a magnitude is at most |gy| 1.13 (the largest slope) / (1 - p)
                live = torch.isfinite(gb)
                assert torch.equal(torch.isfinite(b), live)
                tol = 2 * M * 2.0 ** -24 * 1.2 * gy.double().abs().sum(0) / (1 - p if p < 1 else 1)
                assert ((b - gb).double().abs() <= tol)[live].all(), (act, kinds)
        assert (part[F.epilogue_workspace_len(M, N_):] == GUARD).all()


@pytest.mark.parametrize("M", [64, 65, 256])
def test_few_rows_need_no_workspace(M):
    N_, K = 144, 48
    gy, pre = rand((M, N_), "bf16", 3, 0.1), rand((M, N_), "bf16", 4, 2.0)
    ws, saved = F.Mxfp4LinearWs(M, N_, K), F.Mxfp4LinearSaved(M, N_, K)
    F.mxfp4_linear_fwd(rand((M, K), "bf16", 1), rand((N_, K), "bf16", 2), ws, saved, torch.empty_like(gy))
    got = []
    for part in (None, torch.empty(F.epilogue_workspace_len(M, N_), device=DEV)):
        out = [torch.empty(s, dtype=gy.dtype, device=DEV) for s in ((M, N_), (M, K), (N_, K))] + [torch.empty(N_, device=DEV)]
        F.mxfp4_linear_bwd_epilogue(gy, ws, saved, out[1], out[2], gh=out[0], gb=out[3], pre=pre, act=F.ACT_SILU, part=part)
        got.append(out)
    for a, b in zip(*(g[:3] for g in got)):
        assert torch.equal(a, b)
    # two orders of M roundings, of magnitudes up to |gy| 1.1 (the largest slope)
    tol = 2 * M * 2.0 ** -24 * 1.1 * gy.double().abs().sum(0)
    assert ((got[0][3] - got[1][3]).double().abs() <= tol).all()
    gb = torch.empty(N_, device=DEV)  # and the step on its own
    F.epilogue_bwd(gy, None, gb, pre=pre, act=F.ACT_SILU)
    assert ((gb - got[0][3]).double().abs() <= tol).all()
