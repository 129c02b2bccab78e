"""The registered operators of the MXFP4 layer, the gated activation and the norm:
schema, fake tensors, autograd and ahead-of-time tracing of each, and a block
compiled once for batches of several sizes."""
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests.test_gpu_mx_nn import make

pytestmark = pytest.mark.gpu
DEV = "cuda"
OPS = torch.ops.fp8sg


def rand(*shape, dtype=torch.bfloat16, grad=False, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype).requires_grad_(grad)


def forward_calls():
    for dtype in (torch.bfloat16, torch.float32):
        x, w = rand(5, 96, dtype=dtype, grad=True), rand(40, 96, dtype=dtype, grad=True, seed=1)
        yield "mxfp4_linear", OPS.mxfp4_linear_fwd, (x, w, F.MX_FIT, True)
        for save in (False, True):
            yield "swiglu", OPS.swiglu_fwd, (x, rand(5, 96, dtype=dtype, grad=True, seed=2), save)
            for pdtype in sorted({dtype, torch.float32}, key=str):
                p, b = (rand(96, dtype=pdtype, grad=True, seed=s) for s in (3, 4))
                yield "layer_norm", OPS.layer_norm_fwd, (x, p, b, 1e-5, save)
            yield "layer_norm without parameters", OPS.layer_norm_fwd, (x, None, None, 1e-5, save)


def test_forward_operators():
    """opcheck's own four: schema, autograd registration, fake tensors, tracing
    with dynamic shapes (which compares outputs and gradients with eager ones)."""
    for name, op, args in forward_calls():
        print(name, [a.dtype if isinstance(a, torch.Tensor) else a for a in args], flush=True)
        torch.library.opcheck(op, args)


def test_backward_operators():
    x, w, gy = rand(5, 96), rand(40, 96, seed=1), rand(5, 40, seed=2)
    _, xq, xs, wq, ws = OPS.mxfp4_linear_fwd(x, w, F.MX_FLOOR, True)
    _, gq, gs, uq, us = OPS.swiglu_fwd(x, x + 1, True)
    p = rand(96, dtype=torch.float32)
    _, mean, rstd, cq, cs = OPS.layer_norm_fwd(x, p, None, 1e-5, True)
    which = ("test_schema", "test_faketensor", "test_autograd_registration")
    for need in ((True, True), (True, False), (False, True)):
        torch.library.opcheck(OPS.mxfp4_linear_bwd, (gy, xq, xs, wq, ws, 96, F.MX_FLOOR, *need), test_utils=which)
    torch.library.opcheck(OPS.swiglu_bwd, (x, gq, gs, uq, us), test_utils=which)
    torch.library.opcheck(OPS.swiglu_bwd_plain, (x, x + 1, x + 2), test_utils=which)
    for need in range(1, 8):
        torch.library.opcheck(OPS.layer_norm_bwd, (x, x, None, None, p, mean, rstd, need, torch.float32), test_utils=which)
        torch.library.opcheck(OPS.layer_norm_bwd, (x, None, cq, cs, p, mean, rstd, need, torch.float32), test_utils=which)


@pytest.mark.parametrize("checkpoint", [False, True])
def test_compiled_for_batches_of_several_sizes(checkpoint):
    """One compiled block, dynamic in its batch: bit for bit the eager one's outputs
    and gradients at every size."""
    m = make(checkpoint=checkpoint)
    torch._dynamo.reset()
    c = torch.compile(m, fullgraph=True, dynamic=True, backend="aot_eager")
    for i, lead in enumerate([(16,), (33,), (7,), (100,)]):
        x = rand(*lead, 96, grad=True, seed=i)
        got = []
        for f in (m, c):
            x.grad = None
            m.zero_grad(set_to_none=True)
            y = f(x)
            y.backward(torch.ones_like(y) / 7)
            got.append([y.detach(), x.grad.clone()] + [p.grad.clone() for p in m.parameters()])
        for a, b in zip(*got):
            assert torch.equal(a, b), lead


def test_a_second_derivative_is_refused():
    """The backward operators have no derivative: asking for one raises, it does not
    give zeros."""
    for f in (lambda x: OPS.swiglu_fwd(x, x + 1, False)[0], lambda x: OPS.layer_norm_fwd(x, None, None, 1e-5, False)[0],
              lambda x: OPS.mxfp4_linear_fwd(x, rand(40, 96), F.MX_FLOOR, True)[0]):
        x = rand(5, 96, grad=True)
        (gx,) = torch.autograd.grad(f(x).float().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            gx.float().square().sum().backward()
