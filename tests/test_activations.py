"""The epilogues' activations at FP32 precision, and the polynomial in gelu.

The polynomial: the constants are read out of the source, evaluated exactly and with every step rounded to FP32, against erfcx(a / sqrt 2) / 2.

On the GPU: a 16-bit layer of zero weights puts out act(bias) in FP32. The bounds are the source's own, with steps of 2^-23 of the value and v the argument:
|v| + 8 for silu (its exponent's two roundings cost |v| / 2 each in steps, the exponential 2, sum, quotient and product 4), v^2 + 8 for gelu (the exponent v^2 / 2
rounds twice and its constant once: 3/4 v^2; the polynomial 4, the exponential 2, products 2), 3 |v| + |v|^3 / 4 + 8 for gelu_tanh (the exponent
1.6 |v| + 0.0714 |v|^3 takes at most six roundings of half a step). 1.1e-36 covers quotients by more than 2^126, which are 0: |v| / 2^126 for |v| < 88.
"""
import os
import re

import numpy as np
import pytest

from tests.test_fp8_epilogue import act64
from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_gemm_fmpq_gb300", "csrc", "epilogue.cuh")


def polynomial():
    """The factor of a in t, and the coefficients from the highest power down, as the source has them."""
    body = re.search(r"float gelu\(float v\) \{(.*?)\n\}", open(SOURCE).read(), re.S).group(1)
    factor = re.search(r"fmaf\(a, ([\d.]+)f, 1\.0f\)", body).group(1)
    first = re.search(r"float g = (-?[\d.]+)f;", body).group(1)
    rest = re.findall(r"g = fmaf\(g, t, (-?[\d.]+)f\);", body)
    return np.float32(factor), [np.float32(c) for c in [first, *rest]]


@pytest.mark.parametrize("fp32,bound", [(False, 3.9e-8), (True, 4e-7)])
def test_the_polynomial_of_gelu(fp32, bound):
    from scipy.special import erfcx
    factor, coefficients = polynomial()
    assert len(coefficients) == 9
    a = np.linspace(0, 20, 400001).astype(np.float32).astype(np.float64)
    kept = (lambda v: v.astype(np.float32).astype(np.float64)) if fp32 else (lambda v: v)   # (a product and a sum of FP32 values fit 64 bits: one rounding)
    t = kept(1 / kept(a * np.float64(factor) + 1))
    g = np.full_like(t, coefficients[0])
    for c in coefficients[1:]:
        g = kept(g * t + np.float64(c))
    g = kept(g * t)
    want = erfcx(a / np.sqrt(2)) / 2
    assert np.abs(g / want - 1).max() <= bound


def steps(act, v):
    v = v.abs()
    return {"relu": 0 * v, "silu": v + 8, "gelu": v ** 2 + 8, "gelu_tanh": 3 * v + v ** 3 / 4 + 8}[act]


def arguments():
    import torch
    g = torch.Generator().manual_seed(7)
    spread = torch.exp(torch.rand(20000, generator=g) * 120 - 70) * torch.where(torch.rand(20000, generator=g) < 0.5, -1.0, 1.0)   # 4e-31 to 5e21
    return torch.cat([torch.linspace(-30, 30, 24001), torch.linspace(-200, 200, 8001), torch.linspace(-92, -84, 4001), spread]).float()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("added", [False, True])
def test_in_fp32(fmpq_mod, act, added):  # noqa: F811
    """Without a residual and with one of zeros, which take different forms of the epilogue."""
    import torch
    v = arguments()
    N, K, M = len(v), 8, 3
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16)
    Wp = fmpq_mod.w16_pack_weights(layer, torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"))
    X = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    residual = torch.zeros(M, N, device="cuda") if added else None
    Y = fmpq_mod.w16_gemm(layer, X, Wp, bias=v.cuda(), activation=act, residual=residual, dtype=torch.float32).cpu().double()
    ref = act64(act, v.double())
    bound = steps(act, v.double()) * 2.0 ** -23 * ref.abs() + (0 if act == "relu" else 1.1e-36)
    err = (Y - ref).abs()
    assert bool((err <= bound).all()), (float((err / bound).max()), float(v[int((err / bound).max(0).values.argmax())]))
