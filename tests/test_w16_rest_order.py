"""A 16-bit product whose last units have a launch of their own, followed without a wait by each of the library's calls that start as programmatic
dependents and read its outputs: the same as with a wait between them, eager and captured."""
import pytest

from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)
from tests.test_w16 import matrix


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(300, 4096, 20480), (1, 8192, 28672), (2048, 2048, 12288)])
def test_readers_behind_the_rest(fmpq_mod, M, K, N):  # noqa: F811
    import torch
    bf16 = torch.bfloat16
    wide, back = fmpq_mod.W16Layer(K, N, bf16), fmpq_mod.W16Layer(N, 512, bf16)
    odd = fmpq_mod.W16Layer(N - 3, 512, bf16)            # its rows are copied first
    W = fmpq_mod.w16_pack_weights(wide, matrix(N, K, bf16, 2, 0, K ** -0.5))
    Wb = fmpq_mod.w16_pack_weights(back, matrix(512, N, bf16, 3, 0, N ** -0.5))
    Wo = fmpq_mod.w16_pack_weights(odd, matrix(512, N - 3, bf16, 3, 0, N ** -0.5))
    codes = fmpq_mod.Fp8Layer(N, 512)
    Wc = fmpq_mod.fp8_pack_weights(codes, matrix(512, N, bf16, 4, 0, N ** -0.5))
    inputs = [matrix(M, K, bf16, 10 + i) for i in range(3)]
    stream = matrix(M, N, bf16, 5)
    Y = torch.zeros(M, N, dtype=bf16, device="cuda")

    def readers():
        return [lambda: fmpq_mod.block_norm(Y, stream, layer=codes), lambda: (fmpq_mod.w16_gemm(back, Y, Wb),), lambda: (fmpq_mod.w16_gemm(odd, Y[:, :N - 3], Wo),),
                lambda: fmpq_mod.fp8_quantize(codes, Y), lambda: (fmpq_mod.fp8_quantize_gemm(codes, Y, *Wc),),
                lambda: (fmpq_mod.fp8_quantize_gemm(codes, stream, *Wc, residual=Y[:, :512]),), lambda: (fmpq_mod.w16_gemm(wide, inputs[0], W, residual=Y),)]

    def chain(wait=False):
        out = []
        for i, read in enumerate(readers()):
            fmpq_mod.w16_gemm(wide, inputs[i % 3], W, Y=Y)
            if wait:
                torch.cuda.synchronize()
            out += [t for t in read() if t is not None]
            if wait:
                torch.cuda.synchronize()
        return out

    def same(got):
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            if a.dim() == 2 and a.dtype == torch.float32:
                a, b = a[:, :M], b[:, :M]        # (scales; what rounds rows up to 4 is not written)
            assert torch.equal(a, b), i

    want = chain(True)
    for _ in range(5):
        same(chain())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for _ in range(5):
        graph.replay()
        same(got)
    assert fmpq_mod.w16_device_status(wide) == 0
