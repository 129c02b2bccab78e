"""The layers with an epilogue and dropout through autograd, against the library's
calls (which are held to the definition elsewhere), and a transformer's feed-forward
block of them against its definition."""
import numpy as np
import pytest
import torch
from torch import nn
from torch.utils.checkpoint import checkpoint

import fp8_scaled_gemm_amd as F
from fp8_scaled_gemm_amd import nn as N
from tests import epilogue_reference as E
from tests import mx_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
OPS = torch.ops.fp8sg
BF = torch.bfloat16


def rand(*shape, dtype=BF, grad=False, seed=0, sigma=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(dtype).requires_grad_(grad)


def layer(kind, i, o, act="none", p=0.0, dtype=BF, bias=True, seed=0):
    m = kind(i, o, bias=bias, activation=act, dropout=p, dtype=dtype, device=DEV)
    with torch.no_grad():
        m.weight.copy_(rand(o, i, dtype=dtype, seed=seed, sigma=0.1))
        if bias:
            m.bias.copy_(rand(o, dtype=dtype, seed=seed + 1))
    return m


def words(seed):
    """The words that a module draws next, with the generator left as it was."""
    torch.cuda.manual_seed(seed)
    w = N.dropout_words(torch.device(DEV, 0))
    torch.cuda.manual_seed(seed)
    return w


@pytest.mark.parametrize("act,p,bias,residual", [("gelu", 0.0, True, False), ("none", 0.25, True, True),
                                                 ("silu", 0.5, False, True), ("none", 0.0, True, True)])
@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_float8_layer(act, p, bias, residual, dtype):
    m = layer(N.Float8EpilogueLinear, 48, 80, act, p, dtype, bias)
    x = rand(4, 8, 48, dtype=dtype, grad=True, seed=3)
    res = rand(4, 8, 80, dtype=dtype, grad=True, seed=4) if residual else None
    gy = rand(4, 8, 80, dtype=dtype, seed=5, sigma=0.1)
    rng = words(7) if p else None
    y = m(x, res)
    y.backward(gy)
    M, K, O = 32, 48, 80
    xt, wt, gt = F.fp8_linear_copies(M, O, K)
    saved = F.LinearSaved(M, O, K, x_transposed=xt, w_transposed=wt)
    want, pre = torch.empty(M, O, dtype=dtype, device=DEV), torch.empty(M, O, dtype=dtype, device=DEV)
    a = N.ACTIVATIONS[act]
    F.fp8_scaled_linear_fwd_epilogue(x.detach().view(M, K), m.weight.detach(), saved, want, bias=m.bias, act=a,
                                     residual=res.detach().view(M, O) if residual else None, pre=pre, p=p, rng=rng)
    assert torch.equal(y.view(M, O), want)
    gx, gw, gb = torch.empty(M, K, dtype=dtype, device=DEV), torch.empty_like(m.weight), torch.empty(O, dtype=dtype, device=DEV)
    F.fp8_scaled_linear_bwd_epilogue(gy.view(M, O), saved, F.LinearBwdWs(M, O, transposed=gt), gx, gw,
                                     gh=torch.empty_like(pre), gb=gb, pre=pre, act=a, p=p, rng=rng,
                                     part=torch.empty(F.epilogue_workspace_len(M, O), device=DEV))
    assert torch.equal(x.grad.view(M, K), gx) and torch.equal(m.weight.grad, gw)
    assert not bias or torch.equal(m.bias.grad, gb)
    assert res is None or torch.equal(res.grad, gy)


@pytest.mark.parametrize("act,p,bias,residual", [("gelu_tanh", 0.0, True, False), ("none", 0.25, True, True),
                                                 ("relu", 0.5, False, True), ("none", 0.0, True, False)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_mxfp4_layer(act, p, bias, residual, dtype):
    m = layer(N.MXFP4EpilogueLinear, 50, 77, act, p, dtype, bias)
    x = rand(33, 50, dtype=dtype, grad=True, seed=3)
    wide = rand(33, 90, dtype=dtype, grad=True, seed=4)
    gy = rand(33, 77, dtype=dtype, seed=5, sigma=0.1)
    rng = words(9) if p else None
    y = m(x, wide[:, 5:82] if residual else None)  # rows apart
    y.backward(gy)
    ws, saved = F.Mxfp4LinearWs(33, 77, 50), F.Mxfp4LinearSaved(33, 77, 50)
    want, pre = torch.empty(33, 77, dtype=dtype, device=DEV), torch.empty(33, 77, dtype=dtype, device=DEV)
    a = N.ACTIVATIONS[act]
    F.mxfp4_linear_fwd_epilogue(x.detach(), m.weight.detach(), ws, saved, want, bias=m.bias, act=a,
                                residual=wide.detach()[:, 5:82] if residual else None, pre=pre, p=p, rng=rng)
    assert torch.equal(y, want)
    gx, gw, gb = torch.empty(33, 50, dtype=dtype, device=DEV), torch.empty_like(m.weight), torch.empty(77, dtype=dtype, device=DEV)
    F.mxfp4_linear_bwd_epilogue(gy, ws, saved, gx, gw, gh=torch.empty_like(pre), gb=gb, pre=pre, act=a, p=p, rng=rng,
                                part=torch.empty(F.epilogue_workspace_len(33, 77), device=DEV))
    assert torch.equal(x.grad, gx) and torch.equal(m.weight.grad, gw)
    assert not bias or torch.equal(m.bias.grad, gb)
    assert not residual or (torch.equal(wide.grad[:, 5:82], gy) and wide.grad[:, :5].eq(0).all())


@pytest.mark.parametrize("kind", [N.Float8EpilogueLinear, N.MXFP4EpilogueLinear])
def test_only_what_is_wanted(kind):
    """Frozen parameters, frozen inputs, and a residual's gradient alone."""
    full = layer(kind, 48, 80, "gelu", 0.25)
    x, gy = rand(16, 48, grad=True, seed=3), rand(16, 80, seed=5)
    torch.cuda.manual_seed(1)
    full(x).backward(gy)
    for frozen in (("weight",), ("bias",), ("weight", "bias"), ("x",), ("x", "weight")):
        m = layer(kind, 48, 80, "gelu", 0.25)
        for n in frozen:
            if n != "x":
                getattr(m, n).requires_grad_(False)
        x2 = x.detach().clone().requires_grad_("x" not in frozen)
        torch.cuda.manual_seed(1)
        m(x2).backward(gy)
        for n, got, want in (("x", x2.grad, x.grad), ("weight", m.weight.grad, full.weight.grad),
                             ("bias", m.bias.grad, full.bias.grad)):
            assert got is None if n in frozen else torch.equal(got, want), (frozen, n)
    m = layer(kind, 48, 80, "gelu", 0.25).requires_grad_(False)
    res = rand(16, 80, grad=True, seed=6)
    m(x.detach(), res).backward(gy)
    assert torch.equal(res.grad, gy)
    with torch.no_grad():
        assert not m(x, res).requires_grad


@pytest.mark.parametrize("kind", [N.Float8EpilogueLinear, N.MXFP4EpilogueLinear])
def test_evaluation_drops_nothing_and_seeds_repeat(kind):
    m = layer(kind, 48, 80, "silu", 0.5)
    x = rand(16, 48, seed=3)
    torch.cuda.manual_seed(5)
    a, b = m(x), m(x)
    torch.cuda.manual_seed(5)
    assert torch.equal(m(x), a) and not torch.equal(a, b)
    assert 0.3 < (a == 0).float().mean() < 0.7
    m.eval()
    full = m(x)
    assert torch.equal(full, m(x)) and (full == 0).float().mean() < 0.01


class FeedForward(nn.Module):
    """x + dropout(fc2(gelu(fc1(norm(x)))))"""

    def __init__(self, kind, d=64, f=160, p=0.25, dtype=BF):
        super().__init__()
        self.norm = N.LayerNorm(d, device=DEV, dtype=dtype)
        self.fc1 = layer(kind, d, f, "gelu", 0.0, dtype, seed=1)
        self.fc2 = layer(kind, f, d, "none", p, dtype, seed=2)

    def forward(self, x):
        return self.fc2(self.fc1(self.norm(x)), x)


def test_feed_forward_block_against_its_definition():
    """MXFP4 in fp32: every stage from the values that the stage before really gave."""
    m = FeedForward(N.MXFP4EpilogueLinear, dtype=torch.float32)
    x = rand(3, 11, 64, dtype=torch.float32, grad=True, seed=3)
    keep = {}
    for n in ("norm", "fc1"):
        getattr(m, n).register_forward_hook(lambda mod, i, o, n=n: (o.retain_grad(), keep.__setitem__(n, o)) and None)
    rng = words(11)
    y = m(x)
    gy = rand(3, 11, 64, dtype=torch.float32, seed=4, sigma=0.1)
    y.backward(gy)

    def mat(t):
        return R.f64(t).reshape(33, -1)

    def val(a):
        return R.fp4_values(a, False)
    h, a, w1, w2 = mat(keep["norm"]), mat(keep["fc1"]), R.f64(m.fc1.weight), R.f64(m.fc2.weight)
    b1, b2 = R.f64(m.fc1.bias), R.f64(m.fc2.bias)
    factor = E.keep(rng.tolist(), 33, 64, 0.25)
    pre, pre_err, want, err = E.forward(*R.dot(val(h), val(w1)), b1, E.GELU, None, np.ones((33, 160)), False)
    R.check(keep["fc1"].reshape(33, -1), want, err, "fc1")
    _, _, want, err = E.forward(*R.dot(val(a), val(w2)), b2, E.NONE, mat(x), factor, False)
    R.check(y.reshape(33, -1), want, err, "fc2")
    # backward: dropout, fc2's products, gelu, fc1's products; x's gradient through both paths
    g2, g2_err, gb2, gb2_err = E.backward(mat(gy), mat(gy), E.NONE, factor, False)
    R.check(m.fc2.bias.grad, gb2, gb2_err, "fc2 bias")
    g2r = g2.astype(np.float32).astype(np.float64)  # (exact up to the rounding that the codes' blocks take anyway)
    R.check(m.fc2.weight.grad, *R.dot(val(g2r.T), val(a.T)), "fc2 weight")
    R.check(keep["fc1"].grad.reshape(33, -1), *R.dot(val(g2r), val(w2.T)), "fc1 output's gradient")
    _, _, gb1, gb1_err = E.backward(mat(keep["fc1"].grad), pre, E.GELU, np.ones((33, 160)), False)
    slack = 2.0 * np.abs(mat(keep["fc1"].grad)) * (pre_err + 2.0 ** -23 * np.abs(pre))  # |gelu''| < 0.8; h as kept
    R.check(m.fc1.bias.grad, gb1, gb1_err + slack.sum(axis=0), "fc1 bias")
    ln = R.LayerNorm(mat(x), R.f64(m.norm.weight), R.f64(m.norm.bias), m.norm.eps)
    (dx, dx_err), _, _ = ln.grads(mat(keep["norm"].grad), mat(x))
    R.check(x.grad.reshape(33, -1), dx + mat(gy), dx_err + 2.0 ** -22 * (np.abs(dx) + np.abs(mat(gy))), "x")


@pytest.mark.parametrize("kind", [N.Float8EpilogueLinear, N.MXFP4EpilogueLinear])
def test_recomputation_draws_the_same_masks(kind):
    """torch.utils.checkpoint restores the generator, so the second forward is the first."""
    got = []
    for use in (False, True):
        m = FeedForward(kind)
        x = rand(32, 64, grad=True, seed=3)
        torch.cuda.manual_seed(3)
        y = checkpoint(m, x, use_reentrant=False) if use else m(x)
        torch.cuda.manual_seed(99)
        y.backward(rand(32, 64, seed=5))
        got.append([y.detach(), x.grad] + [p.grad for p in m.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_a_captured_step_draws_new_masks_at_each_replay():
    m = FeedForward(N.Float8EpilogueLinear)
    x, gy = rand(32, 64, seed=3), torch.ones(32, 64, device=DEV, dtype=BF)
    m.fc2.bias.data.fill_(1.0)

    def step():
        return m.fc2(m.fc1(m.norm(x)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.no_grad():
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph), torch.no_grad():
        y = step()
    seen = []
    with torch.no_grad():
        m.fc2.dropout = 0.0
        full = step()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        seen.append(y.clone())
        kept = y != 0
        assert 0.6 < kept.float().mean() < 0.9
        assert torch.allclose(y[kept].float(), full[kept].float() / 0.75, rtol=2.0 ** -7)
        (full.float() + 1).sum().item()  # eager work and a wait between replays
    assert not torch.equal(seen[0], seen[1])


def test_dropout_module():
    d = N.Dropout(0.25)
    for lead in ((40,), (2, 3, 5)):
        x, r = rand(*lead, 77, grad=True, seed=1), rand(*lead, 77, grad=True, seed=2)
        rng = words(4)
        y = d(x, r)
        gy = rand(*lead, 77, seed=3)
        y.backward(gy)
        n = x.numel() // 77
        want, gx = torch.empty(n, 77, dtype=BF, device=DEV), torch.empty(n, 77, dtype=BF, device=DEV)
        F.dropout_fwd(x.detach().view(n, 77), 0.25, rng, want, residual=r.detach().view(n, 77))
        F.dropout_bwd(gy.view(n, 77), 0.25, rng, gx)
        assert torch.equal(y.view(n, 77), want) and torch.equal(x.grad.view(n, 77), gx) and torch.equal(r.grad, gy)
    x = rand(40, 77, grad=True)
    d(x).sum().backward()  # (a gradient of stride 0)
    assert set(x.grad.float().unique().tolist()) == {0.0, float(torch.tensor(1 / 0.75).to(BF))}
    half = rand(40, 200)[:, 10:87]
    torch.cuda.manual_seed(1)
    a = d(half)
    torch.cuda.manual_seed(1)
    assert torch.equal(a, d(half.contiguous()))


@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
def test_serving_form(dtype):
    m = nn.Sequential(layer(N.MXFP4EpilogueLinear, 96, 200, "gelu", 0.5, dtype),
                      nn.Linear(200, 64, dtype=dtype, device=DEV), nn.Linear(64, 32, bias=False, dtype=dtype, device=DEV))
    m[0].rule = "fit"
    kept = N.convert_to_mxfp4_serving(nn.Sequential(*m), lambda mod, fqn: True if getattr(mod, "bias", None) is None else False)
    assert type(kept[0]) is N.MXFP4EpilogueLinear and type(kept[2]) is N.PackedMXFP4Linear
    x = rand(3, 96, dtype=dtype)
    m.eval()
    with torch.no_grad():
        want = m[0](x)
    weight, bias = m[1].weight.detach(), m[1].bias.detach()
    N.convert_to_mxfp4_serving(m, biased=True)
    assert [type(c) for c in m] == [N.PackedMXFP4EpilogueLinear] * 2 + [N.PackedMXFP4Linear]
    assert m[0].rule == "fit" and m[0].activation == "gelu" and m[1].rule == "floor"
    got = m[0](x)
    # the same product, its fp32 sums in another order at most
    tol = {BF: 2.0 ** -7, torch.float16: 2.0 ** -10, torch.float32: 2.0 ** -18}[dtype]
    assert (got.float() - want.float()).abs().max() <= tol * want.float().abs().max()
    for lead in ((1,), (2, 7), (100,)):
        a, r = rand(*lead, 200, dtype=dtype, seed=8), rand(*lead, 64, dtype=dtype, seed=9)
        y = m[1](a, r)
        n = a.numel() // 200
        prod, err = R.dot(R.fp4_values(R.f64(a).reshape(n, 200), False), R.fp4_values(R.f64(weight), False))
        _, _, v, v_err = E.forward(prod, err, R.f64(bias), E.NONE, R.f64(r).reshape(n, 64), np.ones((n, 64)),
                                   dtype != torch.float32)
        R.check(y.reshape(n, 64), v, v_err, "served")


def test_fp16_training_with_a_grad_scaler():
    torch.manual_seed(0)
    m = nn.Sequential(nn.Linear(64, 128, dtype=torch.float16, device=DEV), nn.Linear(128, 64, dtype=torch.float16, device=DEV))
    N.convert_to_float8_training(m, biased=True)
    assert all(type(c) is N.Float8EpilogueLinear for c in m)
    x = rand(32, 64, dtype=torch.float16)
    opt, scaler = torch.optim.SGD(m.parameters(), lr=0.0), N.GradScaler(init_scale=1024.0)
    m(x).float().square().mean().backward()
    plain = [p.grad.clone() for p in m.parameters()]
    opt.zero_grad()
    scaler.scale(m(x).float().square().mean()).backward()
    scaler.unscale_(opt)
    # scaled by a power of two, every gradient is the same up to its own rounding and subnormals
    for a, b in zip(plain, (p.grad for p in m.parameters())):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -3 * a.float().abs().max()
    scaler.step(opt)
    scaler.update()
    assert scaler.state()[2] == 0


# ------------------------------------------------------------------------- operators

def test_forward_operators():
    x, w = rand(16, 48, grad=True), rand(32, 48, grad=True, seed=1)
    b, r, rng = rand(32, grad=True, seed=2), rand(16, 32, grad=True, seed=3), torch.tensor([5, 6], device=DEV)
    for args in ((x, w, b, r, rng, F.ACT_GELU, 0.25), (x, w, None, None, None, F.ACT_NONE, 0.0), (x, w, b, None, rng, F.ACT_NONE, 0.5)):
        print([a if not isinstance(a, torch.Tensor) else a.dtype for a in args], flush=True)
        # (its scale records hold bytes that nothing writes or reads, so two runs' outputs
        # are not compared byte for byte; the compiled block below compares what counts)
        torch.library.opcheck(OPS.scaled_linear_epilogue_fwd, (*args, True),
                              test_utils=("test_schema", "test_faketensor", "test_autograd_registration"))
        torch.library.opcheck(OPS.mxfp4_linear_epilogue_fwd, (*args, F.MX_FIT, True))
    torch.library.opcheck(OPS.dropout_fwd, (x, rand(16, 48, grad=True, seed=9), rng, 0.25))
    torch.library.opcheck(OPS.dropout_fwd, (x, None, rng, 0.25))


def test_backward_operators():
    x, w, gy, rng = rand(16, 48), rand(32, 48, seed=1), rand(16, 32, seed=2), torch.tensor([5, 6], device=DEV)
    which = ("test_schema", "test_faketensor", "test_autograd_registration")
    for act, p, words_ in ((F.ACT_GELU, 0.25, rng), (F.ACT_NONE, 0.0, None)):
        kept = OPS.scaled_linear_epilogue_fwd(x, w, None, None, words_, act, p, True)[1:]
        for need in (True, False):
            torch.library.opcheck(OPS.scaled_linear_epilogue_bwd, (gy, kept[0], words_, *kept[1:], act, p, need, BF),
                                  test_utils=which)
        kept = OPS.mxfp4_linear_epilogue_fwd(x, w, None, None, words_, act, p, F.MX_FIT, True)[1:]
        for need in range(1, 8):
            torch.library.opcheck(OPS.mxfp4_linear_epilogue_bwd,
                                  (gy, kept[0], words_, *kept[1:], 48, act, p, F.MX_FIT, need, torch.float32), test_utils=which)
    torch.library.opcheck(OPS.dropout_bwd, (gy, rng, 0.25), test_utils=which)


@pytest.mark.parametrize("kind,leads", [(N.MXFP4EpilogueLinear, [16, 33, 7, 100]), (N.Float8EpilogueLinear, [16, 48])])
def test_compiled_for_batches_of_several_sizes(kind, leads):
    """One compiled block, dynamic in its batch: the eager one's outputs and gradients."""
    m = FeedForward(kind, p=0.0)
    torch._dynamo.reset()
    c = torch.compile(m, fullgraph=True, dynamic=True, backend="aot_eager")
    for i, lead in enumerate(leads):
        x = rand(lead, 64, grad=True, seed=i)
        got = []
        for f in (m, c):
            x.grad = None
            m.zero_grad(set_to_none=True)
            y = f(x)
            y.backward(torch.ones_like(y) / 7)
            got.append([y.detach(), x.grad.clone()] + [p.grad.clone() for p in m.parameters()])
        assert all(torch.equal(a, b) for a, b in zip(*got)), lead


def test_a_second_derivative_is_refused():
    for f in (lambda x: OPS.scaled_linear_epilogue_fwd(x, rand(32, 48), None, None, None, F.ACT_GELU, 0.0, True)[0],
              lambda x: OPS.mxfp4_linear_epilogue_fwd(x, rand(32, 48), None, None, None, F.ACT_GELU, 0.0, F.MX_FLOOR, True)[0],
              lambda x: OPS.dropout_fwd(x, None, torch.tensor([1, 2], device=DEV), 0.5)):
        x = rand(16, 48, grad=True)
        (gx,) = torch.autograd.grad(f(x).float().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            gx.float().square().sum().backward()
