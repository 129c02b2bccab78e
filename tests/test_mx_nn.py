"""Module conversion for the MXFP4 layers, on the CPU (no kernel runs here)."""
import pytest
import torch
from torch import nn

from fp8_scaled_gemm_amd.nn import (LayerNorm, MXFP4Linear, PackedMXFP4Linear, SwiGLU,
                                    convert_to_mxfp4_training)


class Block(nn.Module):
    def __init__(self):
        super().__init__()
        self.norm = LayerNorm(40, dtype=torch.bfloat16)
        self.gate = nn.Linear(40, 72, bias=False, dtype=torch.bfloat16)
        self.up = nn.Linear(40, 72, bias=False, dtype=torch.bfloat16)
        self.down = nn.Linear(72, 40, bias=False, dtype=torch.bfloat16)
        self.lm_head = nn.Linear(40, 11, bias=False, dtype=torch.bfloat16)
        self.biased = nn.Linear(40, 8, dtype=torch.bfloat16)


def test_training_conversion_shares_weights_and_keeps_heads():
    m = nn.ModuleDict({"a": Block(), "b": Block()})
    before = {n: p for n, p in m.named_parameters()}
    convert_to_mxfp4_training(m, rule="fit")
    for blk in m.values():
        assert all(type(getattr(blk, n)) is MXFP4Linear for n in ("gate", "up", "down"))
        assert type(blk.lm_head) is nn.Linear and type(blk.biased) is nn.Linear
        assert blk.gate.rule == "fit"
    after = {n: p for n, p in m.named_parameters()}
    assert before.keys() == after.keys() and all(before[n] is after[n] for n in before)


def test_filter_is_asked_with_the_full_name():
    m = nn.ModuleDict({"a": Block(), "b": Block()})
    seen = []
    convert_to_mxfp4_training(m, lambda mod, fqn: seen.append(fqn) or fqn == "a.gate")
    assert type(m["a"].gate) is MXFP4Linear and type(m["b"].gate) is nn.Linear
    assert "b.lm_head" in seen and len(seen) == 10


def test_packed_buffers_are_in_the_state():
    p = PackedMXFP4Linear(300, 40)
    sd = p.state_dict()
    assert sd["weight_q"].shape == (40 * 256,) and sd["weight_s"].shape == (2 * 2 * 256,)
    PackedMXFP4Linear(300, 40).load_state_dict(sd)


def test_refusals():
    with pytest.raises(ValueError, match="bias"):
        MXFP4Linear.from_float(nn.Linear(4, 4, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="weight"):
        MXFP4Linear.from_float(nn.Linear(4, 4, bias=False, dtype=torch.float64))
    with pytest.raises(ValueError, match="rule"):
        MXFP4Linear(4, 4, rule="ceil")
    with pytest.raises(TypeError, match="dtype"):
        MXFP4Linear(4, 4)(torch.zeros(2, 4))
    with pytest.raises(ValueError, match="differ"):
        SwiGLU()(torch.zeros(2, 4), torch.zeros(2, 5))
    with pytest.raises(ValueError, match="at least 1"):
        LayerNorm(0)
    with pytest.raises(ValueError, match="over 8"):
        LayerNorm(8)(torch.zeros(2, 4))
    with pytest.raises(ValueError, match="bias"):
        PackedMXFP4Linear.from_float(nn.Linear(4, 4))


@pytest.mark.parametrize("layer", [MXFP4Linear(16, 4), PackedMXFP4Linear(16, 4)])
@pytest.mark.parametrize("shape", [(4, 8), (0, 8), (32,), ()])
def test_inputs_of_another_width_are_refused(layer, shape):
    """Also where the elements would fill whole rows of the layer's width."""
    with pytest.raises(ValueError, match="over 16"):
        layer(torch.zeros(shape, dtype=torch.bfloat16))


@pytest.mark.parametrize("rule", ["floor", "fit"])
def test_serving_keeps_the_rule_a_layer_was_trained_with(rule, monkeypatch):
    """Unless the caller names another; an nn.Linear has none and takes "floor"."""
    from fp8_scaled_gemm_amd import nn as N
    used = []
    monkeypatch.setattr(N, "mxfp4_quantize", lambda w, q, rule: used.append(rule))
    blk = Block()
    blk.down = MXFP4Linear.from_float(blk.down, rule)
    want = {"gate": "floor", "down": rule}
    N.convert_to_mxfp4_serving(blk)
    for n in want:
        layer = getattr(blk, n)
        assert type(layer) is PackedMXFP4Linear and layer.rule == want[n] and f"rule={want[n]}" in repr(layer)
    assert used.count(N.MX_FIT) == (rule == "fit")
    lin = MXFP4Linear(16, 4, rule=rule)
    assert PackedMXFP4Linear.from_float(lin).rule == rule
    assert PackedMXFP4Linear.from_float(nn.Linear(16, 4, bias=False)).rule == "floor"
    for named in ("floor", "fit"):
        assert PackedMXFP4Linear.from_float(lin, rule=named).rule == named
        m = nn.Sequential(MXFP4Linear(16, 4, rule=rule), nn.Linear(4, 4, bias=False))
        assert [layer.rule for layer in N.convert_to_mxfp4_serving(m, rule=named)] == [named, named]
    with pytest.raises(ValueError, match="rule"):
        PackedMXFP4Linear.from_float(lin, rule="ceil")


def test_default_filters_leave_other_types_alone(monkeypatch):
    """A linear that MXFP4 does not take (float64) stays as it is in both conversions."""
    from fp8_scaled_gemm_amd import nn as N

    def quantize(w, q, rule):
        if w.dtype not in (torch.bfloat16, torch.float16, torch.float32):
            raise TypeError(w.dtype)
    monkeypatch.setattr(N, "mxfp4_quantize", quantize)
    for convert, kind in ((convert_to_mxfp4_training, MXFP4Linear), (N.convert_to_mxfp4_serving, PackedMXFP4Linear)):
        m = nn.Sequential(nn.Linear(8, 8, bias=False), nn.Linear(8, 8, bias=False, dtype=torch.float64), nn.Linear(8, 8))
        convert(m)
        assert [type(c) for c in m] == [kind, nn.Linear, nn.Linear]
