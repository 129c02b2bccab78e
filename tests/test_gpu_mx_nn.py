"""The MXFP4, SwiGLU and LayerNorm modules through autograd: a low-precision MLP
block forward and backward, each stage against the definition at the values it
really received."""
import pytest
import torch
from torch import nn

import fp8_scaled_gemm_amd as F
from fp8_scaled_gemm_amd.nn import (GradScaler, LayerNorm, MXFP4Linear, PackedMXFP4Linear, SwiGLU,
                                    convert_to_mxfp4_serving, convert_to_mxfp4_training)
from tests import mx_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Block(nn.Module):
    def __init__(self, d, f, dtype, checkpoint, pdtype=None):
        super().__init__()
        kw = dict(bias=False, device=DEV, dtype=dtype)
        self.norm = LayerNorm(d, checkpoint=checkpoint, device=DEV, dtype=pdtype or dtype)
        self.gate, self.up, self.down = nn.Linear(d, f, **kw), nn.Linear(d, f, **kw), nn.Linear(f, d, **kw)
        self.act = SwiGLU(checkpoint)

    def forward(self, x, keep=None):
        h = self.norm(x)
        g, u = self.gate(h), self.up(h)
        a = self.act(g, u)
        y = self.down(a)
        if keep is not None:
            for n, t in (("h", h), ("g", g), ("u", u), ("a", a)):
                if t.requires_grad:
                    t.retain_grad()
                keep[n] = t
            y.register_hook(lambda grad: keep.__setitem__("gy", grad.reshape(-1, grad.shape[-1])))
        return x + y


def make(d=96, f=200, dtype=torch.bfloat16, checkpoint=True, rule="floor", seed=0, pdtype=None):
    torch.manual_seed(seed)
    return convert_to_mxfp4_training(Block(d, f, dtype, checkpoint, pdtype), rule=rule)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("dtype,rule", [("bf16", "floor"), ("bf16", "fit"), ("f16", "floor"), ("f32", "fit")])
@pytest.mark.parametrize("lead,d,f", [((3, 17), 96, 200), ((64,), 128, 256), ((1, 1), 33, 70)])
def test_block(lead, d, f, dtype, rule, checkpoint):
    t = R.DTYPES[dtype]
    m = make(d, f, t, checkpoint, rule, pdtype=torch.float32)
    x = torch.randn(*lead, d, device=DEV).to(t).requires_grad_()
    keep = {}
    y = m(x, keep)
    y.backward(torch.randn_like(y))
    gy, fit = keep["gy"], rule == "fit"

    def val(v):
        return R.fp4_values(R.f64(v), fit)

    def rows(v):
        return v.detach().reshape(-1, v.shape[-1])
    # forward
    ln = R.LayerNorm(R.f64(rows(x)), R.f64(m.norm.weight), R.f64(m.norm.bias), m.norm.eps)
    R.check(rows(keep["h"]), ln.y, ln.y_err, "h")
    h_val = val(rows(keep["h"]))
    for n, lin in (("g", m.gate), ("u", m.up)):
        R.check(rows(keep[n]), *R.dot(h_val, val(lin.weight)), n)
    R.check(rows(keep["a"]), *R.swiglu(R.f64(rows(keep["g"])), R.f64(rows(keep["u"]))), "a")
    # backward, at the gradients each stage received
    da = rows(keep["a"].grad)
    R.check(da, *R.dot(val(gy), val(m.down.weight.t())), "da")
    R.check(m.down.weight.grad, *R.dot(val(gy.t()), val(rows(keep["a"]).t())), "dW down")
    vg, vu = (R.f64(rows(keep[n])) for n in ("g", "u"))
    if checkpoint:
        vg, vu = R.act8_values(vg), R.act8_values(vu)
    (wg, bg), (wu, bu) = R.swiglu_grad(R.f64(da), vg, vu)
    R.check(rows(keep["g"].grad), wg, bg, "dg")
    R.check(rows(keep["u"].grad), wu, bu, "du")
    ht = val(rows(keep["h"]).t())
    for n, lin in (("g", m.gate), ("u", m.up)):
        R.check(lin.weight.grad, *R.dot(val(rows(keep[n].grad).t()), ht), f"dW {n}")
    xv = R.f64(rows(x))
    (_, _), (dw, dw_err), (db, db_err) = ln.grads(R.f64(rows(keep["h"].grad)), R.act8_values(xv) if checkpoint else xv)
    R.check(m.norm.weight.grad, dw, dw_err, "norm dw")
    R.check(m.norm.bias.grad, db, db_err, "norm db")
    assert x.grad.shape == x.shape and torch.isfinite(x.grad).all()


def test_checkpoints_change_no_output_and_halve_what_is_kept():
    x = torch.randn(512, 96, device=DEV).to(torch.bfloat16)
    plain, small = make(checkpoint=False), make(checkpoint=True)
    kept = []
    for m in (plain, small):
        total = [0]

        def pack(t, total=total):
            total[0] += t.numel() * t.element_size()
            return t
        with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
            g = torch.randn(512, 200, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(x.dtype)
            m.act(g.requires_grad_(), g.detach().flip(0).requires_grad_())
        kept.append(total[0])
    assert torch.equal(plain(x), small(x))
    assert kept[1] < 0.6 * kept[0]


def test_gradients_only_where_wanted():
    m = make()
    x = torch.randn(8, 96, device=DEV, dtype=torch.bfloat16)
    for p in m.parameters():
        p.requires_grad_(False)
    m.down.weight.requires_grad_(True)
    m(x).sum().backward()
    assert m.down.weight.grad is not None and m.gate.weight.grad is None
    lin = m.gate
    xg = x.clone().requires_grad_()
    lin(xg).sum().backward()
    assert xg.grad is not None and lin.weight.grad is None
    with torch.no_grad():
        assert not lin(x).requires_grad


def test_shared_weight_accumulates():
    lin = MXFP4Linear(64, 32, device=DEV)
    nn.init.normal_(lin.weight)
    x = torch.randn(16, 64, device=DEV, dtype=torch.bfloat16)
    lin(x).sum().backward()
    once = lin.weight.grad.clone()
    lin.weight.grad = None
    (lin(x).sum() + lin(x).sum()).backward()
    assert torch.equal(lin.weight.grad, once + once)


def test_strided_inputs_and_expanded_gradients():
    """The halves of one projection as gate and up; a sum's gradient arrives as an
    expanded scalar."""
    act = SwiGLU()
    both = torch.randn(20, 128, device=DEV, dtype=torch.bfloat16).requires_grad_()
    g, u = both[:, :64], both[:, 64:]
    act(g, u).sum().backward()
    gc, uc = g.detach().contiguous().requires_grad_(), u.detach().contiguous().requires_grad_()
    act(gc, uc).sum().backward()
    assert torch.equal(both.grad, torch.cat([gc.grad, uc.grad], 1))
    t = torch.randn(6, 64, 5, device=DEV, dtype=torch.bfloat16).transpose(1, 2)  # rows not contiguous
    ln = LayerNorm(64, device=DEV)
    assert torch.equal(ln(t), ln(t.contiguous()))
    assert act(both[:0, :64], both[:0, 64:]).shape == (0, 64)


def test_no_input_features():
    """A sum over nothing: zeros, and a gradient of nothing."""
    lin = MXFP4Linear(0, 24, device=DEV)
    x = torch.zeros(5, 3, 0, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    y = lin(x)
    assert y.shape == (5, 3, 24) and not bool(y.any())
    y.sum().backward()
    assert x.grad.shape == x.shape and lin.weight.grad.shape == (24, 0)


def test_empty_batch():
    m = make()
    x = torch.empty(0, 96, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    m(x).sum().backward()
    assert x.grad.shape == (0, 96)
    for p in (m.gate.weight, m.down.weight, m.norm.weight, m.norm.bias):
        assert (p.grad == 0).all()


@pytest.mark.parametrize("tokens", [1, 3, 5, 40])
def test_serving(tokens):
    m = make(seed=3)
    x = torch.randn(tokens, 96, device=DEV, dtype=torch.bfloat16)
    with torch.no_grad():
        want = m(x)
    convert_to_mxfp4_serving(m)
    assert all(type(getattr(m, n)) is PackedMXFP4Linear for n in ("gate", "up", "down"))
    got = m(x)
    # the same codes, sums in another order: equal up to a rounding of each stage
    torch.testing.assert_close(got.float(), want.float(), rtol=2e-2, atol=2e-2)
    other = convert_to_mxfp4_serving(make(seed=4))
    other.load_state_dict(m.state_dict())
    assert torch.equal(other(x), m(x))


def test_packed_layer_is_the_training_layer_in_64_bits():
    lin = nn.Linear(300, 70, bias=False, device=DEV, dtype=torch.float16)
    p = PackedMXFP4Linear.from_float(lin, rule="fit")
    for tokens in (1, 4, 30):
        x = torch.randn(2, tokens, 300, device=DEV, dtype=torch.float16)
        y = p(x)
        assert y.shape == (2, tokens, 70)
        want, bound = R.dot(R.fp4_values(R.f64(x.view(-1, 300)), True), R.fp4_values(R.f64(lin.weight), True))
        R.check(y.view(-1, 70), want, bound, "y")


def test_captured_training_step_replays():
    m = make(128, 256)
    x = torch.randn(64, 128, device=DEV, dtype=torch.bfloat16)
    params = list(m.parameters())

    def step():
        for p in params:
            p.grad = None
        m(x).float().square().mean().backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for p in params:
        p.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [p.grad for p in params]
    for i in range(4):
        x.copy_(torch.randn(64, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = [g.clone() for g in held]
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        for a, p in zip(got, params):
            assert torch.equal(a, p.grad)


def test_grad_scaler_takes_its_gradients():
    m = make(dtype=torch.float16)
    opt = torch.optim.SGD(m.parameters(), lr=0.1)
    scaler = GradScaler(init_scale=1024.0)
    x = torch.randn(32, 96, device=DEV, dtype=torch.float16)
    before = m.gate.weight.detach().clone()
    scaler.scale(m(x).float().square().mean()).backward()
    raw = m.gate.weight.grad.clone()
    scaler.unscale_(opt)
    assert torch.equal(m.gate.weight.grad, (raw.float() / 1024).half())
    scaler.step(opt)
    scaler.update()
    assert not torch.equal(before, m.gate.weight)
    m.gate.weight.grad[0, 0] = float("inf")
    opt.zero_grad()
    x[0, 0] = float("inf")  # a block of NaN reaches the gradients: the step is skipped
    scaler.scale(m(x).float().square().mean()).backward()
    before = m.gate.weight.detach().clone()
    scaler.step(opt)
    assert torch.equal(before, m.gate.weight)


def test_compiled_whole():
    m = make()
    x = torch.randn(16, 96, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    want = m(x)
    want.sum().backward()
    grads = [x.grad.clone()] + [p.grad.clone() for p in m.parameters()]
    x.grad = None
    for p in m.parameters():
        p.grad = None
    c = torch.compile(m, fullgraph=True, backend="aot_eager")
    got = c(x)
    got.sum().backward()
    assert torch.equal(got, want)
    for a, b in zip(grads, [x.grad] + [p.grad for p in m.parameters()]):
        assert torch.equal(a, b)


def test_registered_operators_are_well_formed():
    x = torch.randn(5, 96, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(40, 96, device=DEV, dtype=torch.bfloat16)
    torch.library.opcheck(torch.ops.fp8sg.mxfp4_linear_fwd, (x, w, F.MX_FLOOR, True), test_utils=("test_schema", "test_faketensor"))
    torch.library.opcheck(torch.ops.fp8sg.swiglu_fwd, (x, x + 1, True), test_utils=("test_schema",))
    torch.library.opcheck(torch.ops.fp8sg.layer_norm_fwd, (x, None, None, 1e-5, False), test_utils=("test_schema",))


@pytest.mark.parametrize("rule", ["floor", "fit"])
def test_serving_quantises_as_training_did(rule):
    """The packed weight has the codes of the training layer's forward, and its
    inputs are cast by the same rule."""
    m = make(96, 200, rule=rule, seed=5)
    w = {n: getattr(m, n).weight.detach() for n in ("gate", "up", "down")}
    convert_to_mxfp4_serving(m)
    x = torch.randn(9, 96, device=DEV, dtype=torch.bfloat16)
    for n, weight in w.items():
        p = getattr(m, n)
        want = F.Mxfp4(*weight.shape)
        F.mxfp4_quantize(weight, want, rule=F.MX_FIT if rule == "fit" else F.MX_FLOOR)
        torch.cuda.synchronize()
        rows = p.weight_q.numel()
        assert torch.equal(p.weight_q, want.q) and rows == want.q.numel()
        got, need = R.fp4_unpack(p._packed()), R.fp4_unpack(want)  # (scales of rows past the last are anyone's)
        assert (got[1] == need[1]).all()
    fit = rule == "fit"
    y = m.gate(x)
    R.check(y, *R.dot(R.fp4_values(R.f64(x), fit), R.fp4_values(R.f64(w["gate"]), fit)), "y")


def test_empty_batch_with_frozen_weights():
    m = make()
    for p in m.parameters():
        p.requires_grad_(False)
    x = torch.empty(2, 0, 96, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    m(x).sum().backward()
    assert x.grad.shape == (2, 0, 96)
    lin = MXFP4Linear(64, 0, device=DEV)  # no outputs: the weight's gradient is empty, and the only one wanted
    y = lin(torch.zeros(5, 64, dtype=torch.bfloat16, device=DEV))
    y.sum().backward()
    assert y.shape == (5, 0) and lin.weight.grad.shape == (0, 64)
