"""Operands of the MXFP4 layers and checkpoints as Python objects: what a call
passes on is what its checks saw (no kernel runs here)."""
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
