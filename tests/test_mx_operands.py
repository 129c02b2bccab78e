"""Operands of the MXFP4 layers and checkpoints as Python objects: what a call
passes on is what its checks saw (no kernel runs here)."""
import copy
import io
import pickle

import pytest
import torch

import fp8_scaled_gemm_amd as F


def addresses(obj):
    """{operand: (q, s)} as the C struct of a layer's buffers holds them in a call."""
    got = type(obj._all).from_address(obj.c())
    return {n: (getattr(got, n).q, getattr(got, n).s) for n, _ in got._fields_}


def own_addresses(obj):
    held = {n: getattr(obj, n) for n, _ in obj._all._fields_}
    return {n: (m.q.data_ptr(), m.s.data_ptr()) if m is not None else (None, None) for n, m in held.items()}


@pytest.mark.parametrize("make", [lambda: F.Mxfp4LinearSaved(40, 24, 70, "cpu"), lambda: F.Mxfp4LinearWs(40, 24, 70, "cpu")])
def test_an_exchanged_operand_is_the_one_that_is_passed(make):
    """Two layers that share an operand, and an operand made anew: both layers
    pass the present buffers, in either order of their calls."""
    a, b = make(), make()
    for name, _ in a._all._fields_:
        old = getattr(b, name)
        setattr(b, name, getattr(a, name))
        del old  # its tensors are free from here on
        for obj in (b, a, b):
            assert addresses(obj) == own_addresses(obj)
    first = a._all._fields_[0][0]
    size = getattr(a, first)
    setattr(a, first, F.Mxfp4(size.rows, size.k, "cpu"))
    getattr(b, first).q = torch.zeros_like(getattr(b, first).q)
    for obj in (a, b):
        assert addresses(obj) == own_addresses(obj)
    assert addresses(a)[first] != addresses(b)[first]


def operands():
    yield F.Mxfp4(4, 300, "cpu")
    yield F.Act8(4, 40, "cpu")


@pytest.mark.parametrize("m", operands(), ids=lambda m: type(m).__name__)
@pytest.mark.parametrize("which", ["q", "s"])
def test_an_exchanged_buffer_is_checked(m, which):
    """A buffer put into an operand has its size and type, or is refused and the
    old one stays: the calls after it check the operand's size only."""
    old = getattr(m, which)
    for bad in (old[:1], torch.zeros(0, dtype=torch.uint8), torch.cat([old, old]), torch.stack([old, old], -1)[..., 0]):
        with pytest.raises(ValueError, match=f"^{which}: "):
            setattr(m, which, bad)
    for bad in (old.to(torch.int16), None, old.tolist()):
        with pytest.raises(TypeError, match=f"^{which}: "):
            setattr(m, which, bad)
    assert getattr(m, which) is old
    new = torch.zeros_like(old)
    setattr(m, which, new)
    assert getattr(m, which) is new and m.tensors()["qs".index(which)] is new
    assert type(m._pair).from_address(m.c()).s == m.s.data_ptr()


@pytest.mark.parametrize("m", operands(), ids=lambda m: type(m).__name__)
def test_an_operands_size_is_fixed(m):
    """Its buffers were made for it."""
    for name in ("rows", "k" if isinstance(m, F.Mxfp4) else "cols"):
        with pytest.raises(AttributeError, match=name):
            setattr(m, name, 400)


def test_an_exchanged_operand_is_checked():
    ws = F.Mxfp4LinearWs(40, 24, 70, "cpu", backward=False)
    before = own_addresses(ws)
    for name, bad in (("x_q", F.Mxfp4(24, 70, "cpu")), ("w_q", F.Mxfp4(24, 69, "cpu")), ("gy_q", F.Mxfp4(40, 25, "cpu"))):
        with pytest.raises(ValueError, match=f"^{name}: "):
            setattr(ws, name, bad)
    with pytest.raises(TypeError, match="^x_q: "):
        ws.x_q = torch.zeros(40, 70)
    with pytest.raises(AttributeError, match="dims"):
        ws.dims = (80, 24, 70)
    assert own_addresses(ws) == before == addresses(ws)
    ws.gy_q = F.Mxfp4(40, 24, "cpu")
    ws.w_q = None
    assert own_addresses(ws) == addresses(ws)
    saved = F.Mxfp4LinearSaved(40, 24, 70, "cpu")
    for name, bad in (("x_qT", F.Mxfp4(40, 70, "cpu")), ("w_qT", F.Mxfp4(24, 70, "cpu"))):
        with pytest.raises(ValueError, match=f"^{name}: "):
            setattr(saved, name, bad)


def on_device(monkeypatch):
    """Let host tensors through to the last check before the library, which is not reached."""
    from fp8_scaled_gemm_amd import mx
    monkeypatch.setattr(mx, "_here", lambda *t: None)
    monkeypatch.setattr(mx, "_stream", lambda s: pytest.fail("went on to the library"))


def test_two_outputs_in_one_buffer_are_refused(monkeypatch):
    on_device(monkeypatch)
    x, t = torch.zeros(64, 64), torch.zeros(64, 200)
    row = torch.zeros(64)
    one = dict(match="overlap")
    with pytest.raises(ValueError, **one):
        F.swiglu_bwd(x, x + 1, x + 2, t[:, :64], t[:, :64])
    with pytest.raises(ValueError, **one):  # partly
        F.swiglu_bwd(x, x + 1, x + 2, t[:, :64], t[:, 63:127])
    with pytest.raises(ValueError, **one):  # the later rows of one among the other's
        F.swiglu_bwd(x[:32], x[:32] + 1, x[:32] + 2, t[:32, :64], t[5:37, :64])
    with pytest.raises(ValueError, **one):  # different row lengths
        F.swiglu_bwd(x, x + 1, x + 2, t[:, :64], t.view(-1)[64 * 5:64 * 69].view(64, 64))
    with pytest.raises(ValueError, **one):
        F.layer_norm_bwd(x, x + 1, row, row, row, dw=row, db=row, ws=torch.zeros(1 << 16))
    with pytest.raises(ValueError, **one):
        F.layer_norm_fwd(x, row, row, 1e-5, x + 1, mean=row, rstd=row)
    ws, saved = F.Mxfp4LinearWs(64, 64, 64, "cpu"), F.Mxfp4LinearSaved(64, 64, 64, "cpu")
    g = torch.zeros(64, 64)
    with pytest.raises(ValueError, **one):
        F.mxfp4_linear_bwd(x, ws, saved, g, g)
    a, b = F.Mxfp4(64, 64, "cpu"), F.Mxfp4(64, 64, "cpu")
    for which in ("q", "s"):
        old = getattr(b, which)
        setattr(b, which, getattr(a, which))
        with pytest.raises(ValueError, **one):
            F.mxfp4_quantize(x, a, b)
        setattr(b, which, old)
    c, d = F.Act8(64, 64, "cpu"), F.Act8(64, 64, "cpu")
    d.s = c.s
    with pytest.raises(ValueError, **one):
        F.swiglu_fwd(x, x + 1, x + 2, c, d)


@pytest.mark.parametrize("fields", [("x_q", "w_q"), ("gy_q", "gy_qT"), ("x_qT", "w_qT")])
def test_operands_of_one_call_in_one_buffer_are_refused(monkeypatch, fields):
    """Of equal sizes; operands of the forward may be those of the backward."""
    on_device(monkeypatch)
    x = torch.zeros(64, 64)
    ws, saved = F.Mxfp4LinearWs(64, 64, 64, "cpu"), F.Mxfp4LinearSaved(64, 64, 64, "cpu")
    obj = saved if "x_qT" in fields else ws
    setattr(obj, fields[1], getattr(obj, fields[0]))
    if "gy_q" not in fields:
        with pytest.raises(ValueError, match="overlap"):
            F.mxfp4_linear_fwd(x, x + 1, ws, saved, x + 2)
    if "x_q" not in fields:
        with pytest.raises(ValueError, match="overlap"):
            F.mxfp4_linear_bwd(x, ws, saved, x + 1, x + 2)


def test_outputs_side_by_side_are_taken(monkeypatch):
    from fp8_scaled_gemm_amd import mx
    t = torch.zeros(64, 200)
    for a, b in ((t[:, :64], t[:, 64:128]), (t[:, 64:128], t[:, :64]), (t[:, 136:], t[:, :64]), (t[:32, :64], t[32:, :64]),
                 (t[:1, :64], t[:1, 64:128]), (t[:0, :64], t[:0, :64]), (t[:32, :100], t[32:, :100])):
        mx._apart(a, "dg", a.stride(0), b, "du", b.stride(0))
    mx._apart(t.view(-1)[:64 * 64].view(64, 64), "dg", 64, t.view(-1)[64 * 64:64 * 128].view(64, 64), "du", 64)
    mx._apart(t[:0], "dg", 200, t[:0], "du", 200)


@pytest.mark.parametrize("how", ["deepcopy", "copy", "pickle", "save"])
@pytest.mark.parametrize("make", [
    lambda: F.Mxfp4(4, 300, "cpu"), lambda: F.Act8(4, 40, "cpu"), lambda: F.Mxfp4LinearSaved(40, 24, 70, "cpu"),
    lambda: F.Mxfp4LinearWs(40, 24, 70, "cpu", forward=False), lambda: F.Mxfp4LinearWs(40, 24, 70, "cpu")])
def test_copies_and_pickles(make, how):
    """A copy has the sizes and the values, buffers of its own (a shallow one: the
    same buffers) and its own place for their addresses."""
    obj = make()
    parts = [obj] if hasattr(obj, "q") else [m for n in obj._names if (m := getattr(obj, n)) is not None]
    for i, m in enumerate(parts):
        m.q.fill_(17 + i)
        m.s.fill_(120 + i)
    if how == "deepcopy":
        new = copy.deepcopy(obj)
    elif how == "copy":
        new = copy.copy(obj)
    elif how == "pickle":
        new = pickle.loads(pickle.dumps(obj))
    else:
        f = io.BytesIO()
        torch.save(obj, f)
        f.seek(0)
        new = torch.load(f, weights_only=False)
    assert type(new) is type(obj)
    news = [new] if hasattr(new, "q") else [m for n in new._names if (m := getattr(new, n)) is not None]
    assert len(news) == len(parts) and getattr(new, "dims", None) == getattr(obj, "dims", None)
    for a, b in zip(parts, news):
        assert all(getattr(a, n) == getattr(b, n) for n in a._fixed)
        assert torch.equal(a.q, b.q) and torch.equal(a.s, b.s)
        assert (a.q.data_ptr() == b.q.data_ptr()) is (how == "copy")
    assert new.c() != obj.c()
    if not hasattr(obj, "q"):
        assert addresses(new) == own_addresses(new) and addresses(obj) == own_addresses(obj)
    with pytest.raises(AttributeError, match="fixed|made for"):
        setattr(new, "dims" if hasattr(obj, "dims") else "rows", 3)


def test_a_copy_keeps_what_its_operands_share():
    a = F.Mxfp4LinearWs(64, 64, 64, "cpu")
    a.gy_q = a.x_q
    b = copy.deepcopy(a)
    assert b.gy_q is b.x_q and b.x_q is not a.x_q and addresses(b) == own_addresses(b)


class Reached(Exception):
    pass


@pytest.mark.parametrize("shape", [(6,), (2, 3), (2, 3, 1), (1, 6)])
def test_statistics_of_any_shape_with_one_value_a_row(shape, monkeypatch):
    """As the leading dimensions of x, kept as a last one or not."""
    from fp8_scaled_gemm_amd import mx
    monkeypatch.setattr(mx, "_here", lambda *t: None)

    def stream(s):
        raise Reached
    monkeypatch.setattr(mx, "_stream", stream)
    x, w = torch.zeros(2, 3, 40), torch.ones(40)
    mean, rstd = torch.zeros(shape), torch.zeros(shape)
    with pytest.raises(Reached):
        F.layer_norm_fwd(x, w, w, 1e-5, x + 1, mean, rstd)
    with pytest.raises(Reached):
        F.layer_norm_bwd(x, x + 1, w, mean, rstd, dx=x + 2)
    for bad in (torch.zeros(5), torch.zeros(2, 3, 40), torch.zeros(2, 12)[:, ::4]):
        for m, r in ((bad, rstd), (mean, bad)):
            with pytest.raises(ValueError, match="^mean: |^rstd: "):
                F.layer_norm_fwd(x, w, w, 1e-5, x + 1, m, r)
            with pytest.raises(ValueError, match="^mean: |^rstd: "):
                F.layer_norm_bwd(x, x + 1, w, m, r, dx=x + 2)
    for bad in (mean.double(), None, [0.0] * 6):
        with pytest.raises(TypeError, match="^mean: "):
            F.layer_norm_bwd(x, x + 1, w, bad, rstd, dx=x + 2)
