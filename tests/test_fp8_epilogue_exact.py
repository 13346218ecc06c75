"""E4M3 products with an epilogue on whole numbers: outputs equal the exact value's one rounding, bit for bit.

Every block of 128 channels of a token holds one 448, so its scale is 1 and the codes are the values; the others and the weights are -3 .. 3 without 0,
weight scales are 1, 2 or 4. All sums are whole and below 2^24 (asserted).
"""
import pytest

from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)
from tests.test_w16_exact import equal, whole

BLOCK = 128


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,pad", [(1, 8192, 1024, 0), (1, 1024, 512, 0), (7, 2048, 130, 8), (32, 4096, 1000, 4), (33, 300, 257, 1), (64, 512, 8192, 0),
                                       (300, 260, 515, 5), (520, 384, 1028, 4), (777, 2900, 640, 0), (2000, 1000, 2500, 3)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_one_rounding(fmpq_mod, M, K, N, pad, dtype):  # noqa: F811
    import torch
    dtype = getattr(torch, dtype)
    nb = -(-K // BLOCK)
    X, codes = whole((M, K), dtype, M + K), whole((N, K), torch.float32, N)
    for b in range(nb):
        X[:, min(K - 1, b * BLOCK + 17 * b % BLOCK)] = 448 if b % 2 else -448
    scales = 2.0 ** (torch.arange(-(-N // BLOCK) * nb, device="cuda").view(-1, nb) % 3)
    layer = fmpq_mod.Fp8Layer(K, N)
    W = fmpq_mod.fp8_pack_codes(layer, codes.to(torch.float8_e4m3fn), scales)
    w = codes.double() * scales.double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    sums = X.double() @ w.t()
    bias, residual = whole((N,), torch.float32, 5, 2047), whole((M, N + pad), dtype, 6, 255)[:, :N]
    full = sums + bias.double() + residual.double()
    assert float(full.abs().max()) < 2 ** 24 and float(sums.abs().max()) < 2 ** 24
    A, s = fmpq_mod.fp8_quantize(layer, X)
    assert bool((s[:, :M] == 1).all())
    equal(fmpq_mod.fp8_quantize_gemm(layer, X, *W), sums.float())
    equal(fmpq_mod.fp8_gemm(layer, A, s, *W, M, dtype=dtype, bias=bias, residual=residual), full.float())
    equal(fmpq_mod.fp8_quantize_gemm(layer, X, *W, bias=bias, activation="relu"), (sums + bias.double()).clamp_min(0).float())
    equal(fmpq_mod.fp8_quantize_gemm(layer, X, *W, residual=residual), (sums + residual.double()).float())
