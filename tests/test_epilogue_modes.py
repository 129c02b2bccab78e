"""A layer made from another, or put in its place, is in that one's mode (no GPU needed)."""
import pytest
import torch
from torch import nn

from fp8_scaled_gemm_amd import nn as N

MAKE = {"float8": lambda m: N.Float8EpilogueLinear.from_float(m, "gelu", 0.5),
        "mxfp4": lambda m: N.MXFP4EpilogueLinear.from_float(m, "gelu", 0.5)}


@pytest.mark.parametrize("training", [True, False])
@pytest.mark.parametrize("kind", MAKE)
def test_from_float_keeps_the_mode(kind, training):
    new = MAKE[kind](nn.Linear(32, 48, dtype=torch.bfloat16).train(training))
    assert new.training is training
    assert new.dropout == 0.5 and new.activation == "gelu"


@pytest.mark.parametrize("training", [True, False])
@pytest.mark.parametrize("convert", [N.convert_to_float8_training, N.convert_to_mxfp4_training])
def test_conversions_keep_the_mode(convert, training):
    model = nn.Sequential(nn.Linear(32, 48), nn.Linear(48, 32)).to(torch.bfloat16).train(training)
    model[0].train(not training)  # (a part of a model may be in the other mode)
    convert(model, biased=True)
    assert type(model[0]) is not nn.Linear and type(model[1]) is not nn.Linear
    assert model[0].training is (not training) and model[1].training is training
