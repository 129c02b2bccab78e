"""The series that gelu's tail is made of, with the constants of the source, in 64 bits
against the normal distribution's (no GPU needed)."""
import os
import re

import numpy as np
import pytest
from scipy.special import erfcx

HPP = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_scaled_gemm_amd", "csrc", "epilogue.hpp")


def series():
    """(c of t = 1 / (1 + c z), coefficients), first the short form, then the long one."""
    body = open(HPP).read().split("__device__ __forceinline__ Tail tail(float z) {")[1].split("return Tail{t, p, e};")
    num, out = r"(-?[\d.]+)f", []
    for part in body[:2]:
        c, = re.findall(rf"fmaf\({num}, z, 1\.0f\)", part)
        first, second = re.findall(rf"float p = fmaf\({num}, t, {num}\)", part)[0]
        out.append((np.float32(c), [np.float32(v) for v in (first, second, *re.findall(rf"p = fmaf\(p, t, {num}\)", part))]))
    return out


@pytest.mark.parametrize("form,terms,bound", [(0, 6, 8.6e-6), (1, 9, 1.06e-7)])
def test_relative_error_on_the_whole_range(form, terms, bound):
    c, p = series()[form]
    assert len(p) == terms
    z = np.linspace(0, 16, 1600001)
    t, v = 1 / (1 + float(c) * z), 0.0
    for k in p:
        v = v * t + float(k)
    off = np.abs(t * v / (erfcx(z / np.sqrt(2)) / 2) - 1).max()  # Q(z) exp(z^2 / 2) is erfcx's half
    assert 0.9 * bound < off <= bound
