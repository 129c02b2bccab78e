"""An fp16 model converted with biased=True and a GradScaler: layers that unscale in their
product and layers that leave it to unscale_ end with the same, unscaled gradients."""
import pytest
import torch
from torch import nn

import fp8_scaled_gemm_amd.nn as N

pytestmark = pytest.mark.gpu


def model():
    torch.manual_seed(1)
    m = nn.Sequential(nn.Linear(64, 96, bias=True), nn.Linear(96, 64, bias=False), nn.Linear(64, 32, bias=True))
    return m.to("cuda", torch.float16)


def grads(scale, attach):
    m, s = model(), N.GradScaler(init_scale=scale)
    N.convert_to_float8_training(m, biased=True, grad_scaler=s if attach else None)
    opt = torch.optim.SGD(m.parameters(), lr=0.0)
    x = torch.randn(48, 64, generator=torch.Generator().manual_seed(2)).to("cuda", torch.float16)
    s.scale(m(x).float().square().mean()).backward()
    s.unscale_(opt)
    assert s.state()[2] == 0
    return [p.grad.clone() for p in m.parameters()]


def test_gradients_are_unscaled_once():
    """(The unscale inside a product gives the bits of the pass of its own.)"""
    a, b = grads(1024.0, True), grads(1024.0, False)
    assert len(a) == 5 and all(torch.equal(u, v) for u, v in zip(a, b))
    assert all(torch.isfinite(u).all() and (u != 0).any() for u in a)


def test_an_fp32_bias_is_refused_by_the_scaler():
    m = N.Float8EpilogueLinear(32, 48, device="cuda", dtype=torch.float16)
    nn.init.normal_(m.weight)
    m.bias = nn.Parameter(torch.zeros(48, device="cuda"))
    s = N.GradScaler(init_scale=8.0)
    s.scale(m(torch.ones(16, 32, device="cuda", dtype=torch.float16)).float().sum()).backward()
    with pytest.raises(TypeError, match="fp16 gradients only"):
        s.unscale_(torch.optim.SGD(m.parameters(), lr=0.0))
