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
