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


@pytest.mark.gpu
@pytest.mark.parametrize("T,F", [(8, 200), (200, 128), (3000, 256)])
def test_experts(fmpq_mod, T, F):  # noqa: F811
    import torch
    H, N, E, k = 256, 264, 4, 2
    g = torch.Generator().manual_seed(T)
    X = torch.randn(T, H, generator=g).bfloat16().cuda()
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.int().cuda()
    w = (torch.rand(T, k, generator=g) + 0.1).cuda()
    Lu, Ld = fmpq_mod.Fp8Layer(H, 2 * F, experts=E, gated=True), fmpq_mod.Fp8Layer(F, N, experts=E)
    Wu = fmpq_mod.fp8_pack_weights(Lu, (torch.randn(E, 2 * F, H, generator=g) / 16).bfloat16().cuda())
    Wd = fmpq_mod.fp8_pack_weights(Ld, (torch.randn(E, N, F, generator=g) / 16).bfloat16().cuda())
    clean = fmpq_mod.moe_experts(Lu, Ld, X, ids, w, *Wu, *Wd)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[spoil(X)] = True
    Y = fmpq_mod.moe_experts(Lu, Ld, X, ids, w, *Wu, *Wd)
    assert bool(torch.isnan(Y.cpu()[bad]).all())
    assert torch.equal(Y.cpu()[~bad], clean.cpu()[~bad])
    # NaN scales of a block of gate rows
    up = torch.zeros(E, 2 * F, H)
    up[:, :, 0] = 1.0
    Wu = fmpq_mod.fp8_pack_codes(Lu, up.to(torch.float8_e4m3fn).cuda(), nan_scales(Lu, F))
    Y = fmpq_mod.moe_experts(Lu, Ld, torch.ones_like(X), ids, w, *Wu, *Wd)
    assert bool(torch.isnan(Y).all())


def nan_scales(layer, F):
    """Scales of 1, the last block of gate rows NaN."""
    import torch
    s = torch.ones(layer.experts, layer.scale_rows, layer.nb, device="cuda")
    s[:, layer.scale_rows // 2 - 1, 0] = NAN
    return s


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 6000])
def test_one_hidden_channel(fmpq_mod, T):  # noqa: F811
    """inf * 0 in one channel of a hidden block: its scale is NaN whatever the kernel, whatever the other channels."""
    import torch
    layer = fmpq_mod.Fp8Layer(128, 256, gated=True)
    w = torch.zeros(1, 256, 128)
    w[0, :128] = 0.5
    w[0, 128:] = 2.0 ** -9
    w[0, 9], w[0, 128 + 9] = 448.0, 0.0
    scales = torch.ones(1, 2, 1, device="cuda")
    scales[0, 0, 0] = 3e38 / 128
    W = fmpq_mod.fp8_pack_codes(layer, w.to(torch.float8_e4m3fn).cuda(), scales)
    plan = fmpq_mod.moe_plan(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1)
    X = torch.ones(T, 128, dtype=torch.bfloat16, device="cuda")
    _, s = fmpq_mod.moe_up(layer, plan, *fmpq_mod.moe_quantize(layer, plan, X), *W)
    assert bool(torch.isnan(s[0, :T]).all())
