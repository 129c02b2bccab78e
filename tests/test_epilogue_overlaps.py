"""A product's results over its own codes are refused before any launch (no GPU needed)."""
import pytest
import torch

import fp8_scaled_gemm_amd as F
from tests.test_epilogue_abi import reaches_device


def test_results_over_operands_are_refused():
    raw = torch.zeros(4096, dtype=torch.uint8)
    A, B = raw[:1024].view(16, 64), torch.zeros(32, 64, dtype=torch.uint8)
    C, over = torch.zeros(16, 32, dtype=torch.bfloat16), raw[512:1536].view(torch.bfloat16).view(16, 32)
    for y, pre, name in ((over, None, "C"), (C, over, "pre")):
        for a, b, dims in ((A, B, (16, 32)), (B, A, (32, 16))):
            with pytest.raises(ValueError, match=f"{name} and an operand overlap"):
                F.fp8_gemm_epilogue(a, b, 0, 0, y.view(dims), pre=pre if pre is None else pre.view(dims))
    a, b = F.Mxfp4(16, 64, device="cpu"), F.Mxfp4(32, 64, device="cpu")
    for m in (a, b):
        for buf in (m.q, m.s):
            whole = torch.zeros(buf.numel() + 1024, dtype=torch.uint8)
            m.q, m.s = (whole[1024:], m.s) if buf is m.q else (m.q, whole[1024:])
            y = whole[:1026][2:].view(torch.bfloat16).view(16, 32)
            with pytest.raises(ValueError, match="C and an operand overlap"):
                F.mxfp4_gemm_epilogue(a, b, y)
            m.q, m.s = (buf, m.s) if m.q.data_ptr() == whole[1024:].data_ptr() else (m.q, buf)
    reaches_device(F.fp8_gemm_epilogue, A, B, 0, 0, C)  # all is well but the device
