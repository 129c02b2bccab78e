"""The layers with an epilogue: construction, conversion and refusals, on the CPU (no
kernel runs here)."""
import pytest
import torch
from torch import nn

from fp8_scaled_gemm_amd.nn import (Dropout, Float8EpilogueLinear, Float8Linear, MXFP4EpilogueLinear, MXFP4Linear,
                                    PackedMXFP4EpilogueLinear, convert_to_float8_training, convert_to_mxfp4_training)

BF = torch.bfloat16


class Block(nn.Module):
    def __init__(self, dtype=BF):
        super().__init__()
        self.fc1 = nn.Linear(32, 64, dtype=dtype)
        self.fc2 = nn.Linear(64, 32, dtype=dtype)
        self.plain = nn.Linear(32, 32, bias=False, dtype=dtype)
        self.odd = nn.Linear(30, 8, dtype=dtype)
        self.router = nn.Linear(32, 16, dtype=dtype)


def kinds(m):
    return [type(getattr(m, n)) for n in ("fc1", "fc2", "plain", "odd", "router")]


def test_float8_conversion():
    m = convert_to_float8_training(Block())
    assert kinds(m) == [nn.Linear, nn.Linear, Float8Linear, nn.Linear, nn.Linear]  # biased layers are left alone
    m = Block()
    before = dict(m.named_parameters())
    convert_to_float8_training(m, biased=True)
    assert kinds(m) == [Float8EpilogueLinear, Float8EpilogueLinear, Float8Linear, nn.Linear, nn.Linear]
    after = dict(m.named_parameters())
    assert before.keys() == after.keys() and all(before[n] is after[n] for n in before)
    with pytest.raises(ValueError, match="dynamic"):
        convert_to_float8_training(Block(), biased=True, scaling="rowwise")
    m = Block()
    m.fc1.bias = nn.Parameter(m.fc1.bias.detach().double())  # of another type: left alone
    assert kinds(convert_to_float8_training(m, biased=True))[0] is nn.Linear


def test_mxfp4_conversion():
    m = convert_to_mxfp4_training(Block())
    assert kinds(m) == [nn.Linear, nn.Linear, MXFP4Linear, nn.Linear, nn.Linear]
    m = Block(torch.float32)
    before = dict(m.named_parameters())
    convert_to_mxfp4_training(m, rule="fit", biased=True)
    assert kinds(m) == [MXFP4EpilogueLinear, MXFP4EpilogueLinear, MXFP4Linear, MXFP4EpilogueLinear, nn.Linear]
    assert m.fc1.rule == "fit" and m.fc1.activation == "none" and m.fc1.dropout == 0
    after = dict(m.named_parameters())
    assert before.keys() == after.keys() and all(before[n] is after[n] for n in before)


def test_state_of_the_layers():
    a = Float8EpilogueLinear(16, 32, activation="gelu", dropout=0.1)
    assert set(a.state_dict()) == {"weight", "bias"} and a.weight.dtype == a.bias.dtype == BF
    assert set(Float8EpilogueLinear(16, 32, bias=False).state_dict()) == {"weight"}
    f = Float8EpilogueLinear.from_float(nn.Linear(16, 32, dtype=torch.float16), "relu", 0.5)
    assert f.weight.dtype == torch.float16 and f.activation == "relu" and f.dropout == 0.5 and f.out_features == 32
    p = PackedMXFP4EpilogueLinear(300, 40, activation="silu")
    assert set(p.state_dict()) == {"weight_q", "weight_s", "bias"}
    PackedMXFP4EpilogueLinear(300, 40).load_state_dict(p.state_dict())
    assert set(PackedMXFP4EpilogueLinear(300, 40, bias=False).state_dict()) == {"weight_q", "weight_s"}


def test_refusals():
    for make in (Float8EpilogueLinear, MXFP4EpilogueLinear):
        with pytest.raises(ValueError, match="activation"):
            make(16, 16, activation="tanh")
        with pytest.raises(ValueError, match="dropout"):
            make(16, 16, dropout=1.5)
        with pytest.raises(TypeError):
            make(16, 16, dtype=torch.float64)
        with pytest.raises(TypeError, match="weight"):
            make.from_float(nn.Linear(16, 16, dtype=torch.float64))
        lin = nn.Linear(16, 16, dtype=BF)
        lin.bias = nn.Parameter(lin.bias.detach().half())
        with pytest.raises(TypeError, match="bias"):
            make.from_float(lin)
        with pytest.raises(TypeError, match="dtype"):
            make(16, 16)(torch.zeros(16, 16))
        with pytest.raises(ValueError, match="16 values"):
            make(16, 16)(torch.zeros(16, 8, dtype=BF))
        for bad in (torch.zeros(16, 16), torch.zeros(8, 16, dtype=BF), torch.zeros(1, 16, 16, dtype=BF)):
            with pytest.raises(ValueError, match="residual"):
                make(16, 16)(torch.zeros(16, 16, dtype=BF), bad)
    with pytest.raises(TypeError):
        Float8EpilogueLinear(16, 16, dtype=torch.float32)
    with pytest.raises(ValueError, match="rule"):
        MXFP4EpilogueLinear(16, 16, rule="ceil")
    with pytest.raises(TypeError):
        PackedMXFP4EpilogueLinear(16, 16, dtype=torch.int8)
    with pytest.raises(ValueError):
        Dropout(-0.1)
    with pytest.raises(TypeError):
        Dropout(0.5)(torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="residual"):
        Dropout(0.5)(torch.zeros(4, 4), torch.zeros(4))


def test_dropout_in_evaluation():
    x, r = torch.randn(3, 4), torch.randn(3, 4)
    for d in (Dropout(0.5).eval(), Dropout(0.0)):
        assert d(x) is x and torch.equal(d(x, r), x + r)
