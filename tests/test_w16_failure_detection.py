"""Waits of the 16-bit product that give up, without a GPU fault: the library's test hook leaves out one copy of weights, so that the waits for it run out
after a few thousand polls. The call returns, the status reads FMPQ_ERR_TIMEOUT, and the next call is right."""
import time

import pytest

from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)
from tests.test_w16 import matrix

FMPQ_ERR_TIMEOUT = 5


# one unit a pair; units in turn, an aborted one's later ones too; units of two parts; K split, the first pair or another one fails; a rest in a launch of its own
@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,cta,copy", [(100, 192, 1000, 0, 0), (100, 192, 1000, 1, 2), (100, 512, 512, 0, 3), (2000, 1024, 10240, 0, 40), (2000, 1024, 10240, 5, 3), (777, 2048, 5632, 2, 31),
                                            (1, 8192, 1024, 0, 0), (1, 8192, 1024, 2, 5), (1, 8192, 1024, 7, 31), (16, 2048, 512, 3, 2), (300, 4096, 20480, 1, 10)])
def test_withheld_copy_times_out_and_recovers(fmpq_mod, M, K, N, cta, copy):  # noqa: F811
    import torch
    X, W = matrix(M, K, torch.bfloat16, 1), matrix(N, K, torch.bfloat16, 2, 0, K ** -0.5)
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    want = fmpq_mod.w16_gemm(layer, X, Wp)
    torch.cuda.synchronize()
    assert fmpq_mod.w16_device_status(layer) == 0
    buf = torch.full((M + 8, N), 7.0, dtype=X.dtype, device="cuda")
    t0 = time.perf_counter()
    assert fmpq_mod._lib.w16_gemm_fault_test(layer.handle, X.data_ptr(), K, M, Wp.data_ptr(), buf[4:].data_ptr(), N, cta, copy, 1 << 14, None) == 0
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert fmpq_mod.w16_device_status(layer, clear=True) == FMPQ_ERR_TIMEOUT
    assert elapsed < 5.0, f"the aborted call took {elapsed:.1f} s"
    assert bool((buf[:4] == 7).all()) and bool((buf[-4:] == 7).all())
    for _ in range(2):
        assert torch.equal(fmpq_mod.w16_gemm(layer, X, Wp), want)
    assert fmpq_mod.w16_device_status(layer) == 0


@pytest.mark.gpu
def test_the_hook_refuses(fmpq_mod):  # noqa: F811
    import torch
    X = matrix(40, 128, torch.float16, 1)
    plain, gated = fmpq_mod.W16Layer(128, 256, torch.float16), fmpq_mod.W16Layer(128, 256, torch.float16, gated=True)
    Wp = fmpq_mod.w16_pack_weights(plain, matrix(256, 128, torch.float16, 2))
    Y = torch.full((40, 256), 7.0, dtype=torch.float16, device="cuda")

    def call(layer=plain, x=X.data_ptr(), ldx=128, M=40, cta=0, copy=0, polls=1 << 14):
        return fmpq_mod._lib.w16_gemm_fault_test(layer.handle, x, ldx, M, Wp.data_ptr(), Y.data_ptr(), 256, cta, copy, polls, None)

    assert fmpq_mod._lib.w16_gemm_fault_test(None, None, 8, 1, None, None, 8, 0, 0, 1 << 14, None) == 1
    for code, kw in [(1, dict(layer=gated)), (1, dict(cta=-1)), (1, dict(copy=-1)), (1, dict(polls=1023)), (2, dict(M=0)), (2, dict(ldx=127)),
                     (3, dict(ldx=129)), (3, dict(x=X.data_ptr() + 2))]:
        assert call(**kw) == code, kw
    torch.cuda.synchronize()
    assert bool((Y == 7).all()) and fmpq_mod.w16_device_status(plain) == 0


def test_the_hook_refuses_without_a_layer():
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    assert fmpq.load_library().w16_gemm_fault_test(None, 4096, 8, 1, 4096, 4096, 8, 0, 0, 1 << 14, None) == 1
