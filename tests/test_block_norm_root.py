"""block_norm's 1 / sqrt(mean square + eps) is the real one rounded once: no tolerance.

Every row holds a, -a, b, -b (whole numbers up to 1000) and zeros, and K is a power of two: its mean is 0, its sum of squares at most
4e6 and its mean square are exact in FP32 in any order. So y's largest value is fl(max|x| * inv) and its block's scale
fl(that / 448), where inv = fl(1 / sqrt(fl(mean square + eps))): FP32 values that the scales must equal.
"""
import numpy as np
import pytest

from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)


def rows_of(M, K, seed):
    rng = np.random.default_rng(seed)
    a, b = rng.integers(1, 1001, M), rng.integers(0, 1001, M)
    X = np.zeros((M, K), np.float32)
    X[:, 3], X[:, 7] = a, -a
    X[:, 40], X[:, 41] = -b, b
    return X, np.maximum(a, b).astype(np.float32), 2 * (a * a + b * b).astype(np.float64)


def inverse_root(squares, K, eps):
    """fl(1 / sqrt(d)) of d = fl(squares / K + eps), which 64 bits decide: no d here lies too near to a tie."""
    d = ((squares / K).astype(np.float32) + np.float32(eps)).astype(np.float64)
    inv = 1.0 / np.sqrt(d)
    got = inv.astype(np.float32)
    assert (got == (inv * (1 - 4e-16)).astype(np.float32)).all() and (got == (inv * (1 + 4e-16)).astype(np.float32)).all()
    return got


def scales_of(most, inv):
    return (most * inv).astype(np.float32) / np.float32(448)


def test_the_definition_by_hand():
    """3, -3 and 0s at K = 2 and eps = 7: 1 / sqrt(16)."""
    assert inverse_root(np.array([18.0]), 2, 7.0) == np.float32(0.25)
    assert scales_of(np.float32([448]), np.float32([0.25])) == np.float32(0.25)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("M,K,shift", [(9, 512, 0), (300, 4096, 0), (2, 32768, 0), (2000, 2048, 0), (2000, 4096, 1), (400, 16384, 0), (1300, 256, 0)])
def test_the_root_is_rounded_once(fmpq_mod, M, K, shift, kind):  # noqa: F811
    import torch
    X, most, squares = rows_of(M, K, M + K)
    buf = torch.zeros(M * K + shift, dtype=torch.float16, device="cuda")
    rows = buf[shift:].view(M, K)
    rows.copy_(torch.from_numpy(X))
    for eps in (1e-6, 1e-5, 0.25):
        out = fmpq_mod.block_norm(rows, kind=kind, eps=eps, layer=fmpq_mod.Fp8Layer(K, 16))
        want = torch.from_numpy(scales_of(most, inverse_root(squares, K, eps)))
        assert torch.equal(out.a_scales[0, :M].cpu(), want), int((out.a_scales[0, :M].cpu() != want).sum())
        assert bool((out.a_scales[1:, :M] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(9, 512), (2000, 2048), (2, 32768)])
def test_so_is_the_one_of_a_norm_before_it(fmpq_mod, M, K):  # noqa: F811
    """u = norm(X) alone: r in 16 bits is fl16(fl(x * inv))."""
    import torch
    X, _, squares = rows_of(M, K, K)
    inv = torch.from_numpy(inverse_root(squares, K, 1e-6))[:, None]
    out = fmpq_mod.block_norm(torch.from_numpy(X).half().cuda(), post_norm=True, pre_norm=False)
    assert torch.equal(out.R.cpu(), (torch.from_numpy(X) * inv).half())
