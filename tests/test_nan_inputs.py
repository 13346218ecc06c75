"""NaN and infinity in an input reach the outputs that depend on it, for any number of tokens, and no others."""
import pytest

from tests.test_fp8_linear import draw
from tests.test_moe import fmpq_mod  # noqa: F401  (the fixture)

NAN, INF = float("nan"), float("inf")


def spoil(X):
    """Tokens 0, 2, 4, 6: a block of NaN, one NaN, one infinity, nothing but NaN. Returns them."""
    X[0, 128:256] = NAN
    X[2, 7] = NAN
    X[4, 200] = -INF
    X[6] = NAN
    return [0, 2, 4, 6]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(8, 300, 130), (60, 512, 256), (600, 300, 513), (3000, 256, 1024)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_linear(fmpq_mod, M, K, N, dtype):  # noqa: F811
    import torch
    X = draw(M, K, getattr(torch, dtype), M + N)
    layer = fmpq_mod.Fp8Layer(K, N)
    W = fmpq_mod.fp8_pack_weights(layer, torch.randn(N, K, generator=torch.Generator().manual_seed(N)).to(X.dtype).cuda())
    clean = fmpq_mod.fp8_quantize_gemm(layer, X, *W)
    X = X.clone()
    bad = torch.zeros(M, dtype=torch.bool)
    bad[spoil(X)] = True
    Y = fmpq_mod.fp8_quantize_gemm(layer, X, *W)
    assert bool(torch.isnan(Y.cpu()[bad]).all())
    assert torch.equal(Y.cpu()[~bad], clean.cpu()[~bad])


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
def test_weights(fmpq_mod, gated):  # noqa: F811
    """A weight block that is all NaN, and one NaN in a block: the rows that hold them are not 0."""
    import torch
    N, K = 512, 384
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(3)).half()
    w[:128, 128:256] = NAN
    w[300, 5] = NAN
    layer = fmpq_mod.Fp8Layer(K, N, gated=gated)
    got = fmpq_mod.fp8_unpack_weights(layer, *fmpq_mod.fp8_pack_weights(layer, w.cuda())).cpu()
    assert bool(torch.isnan(got[w.isnan()]).all())
