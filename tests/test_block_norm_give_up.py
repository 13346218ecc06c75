"""A wait of block_norm that gives up, without a GPU fault: the library's test hook leaves out the copy of one row, so that the wait for it
runs out after a few thousand polls. That row and those that its CTA takes after it are NaN, whole; every other row is the normal
call's, bit for bit; the kernel ends by itself, and the next call is right."""
import ctypes
import time

import pytest

from tests.test_block_norm import draw, vectors
from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)


def args_of(fmpq, X, residual, kind, post, pre, w, R, Y, A, s):
    M, K = X.shape
    a = fmpq.BlockNormArgs(X=X.data_ptr(), ldx=K, M=M, K=K, dtype=1, param_dtype=1, kind=kind == "layer", post_norm=post, pre_norm=pre,
                           eps=1e-6, residual_scale=1.0, R=R.data_ptr(), ldo=K)
    if residual is not None:
        a.residual, a.ldr = residual.data_ptr(), K
    if post:
        a.post_weight = w[0].data_ptr()
    if pre:
        a.weight, a.bias, a.Y, a.ldy = w[1].data_ptr(), w[2].data_ptr(), Y.data_ptr(), K
        a.A_packed, a.a_scales = A.data_ptr(), s.data_ptr()
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,row", [(2000, 4096, 700), (2000, 4096, 0), (1500, 512, 1499), (1300, 16384, 400), (3001, 1024, 50)])
@pytest.mark.parametrize("kind,post,pre,added", [("rms", False, True, True), ("layer", True, True, True), ("rms", False, False, True), ("rms", True, False, False)])
def test_withheld_row_and_those_behind_it(fmpq_mod, M, K, row, kind, post, pre, added):  # noqa: F811
    import torch
    X, residual = draw(M, K, torch.bfloat16, 1), draw(M, K, torch.bfloat16, 2) if added else None
    w, layer = vectors(K, torch.bfloat16, 3, 3), fmpq_mod.Fp8Layer(K, 16)

    def outputs():
        A, s = layer.activations(M, X.device)
        return (torch.full_like(X, 7.0), torch.full_like(X, 7.0), A.fill_(7), s.fill_(7.0))

    want, got, again = outputs(), outputs(), outputs()
    lib = fmpq_mod._lib
    assert lib.fmpq_block_norm(ctypes.addressof(args_of(fmpq_mod, X, residual, kind, post, pre, w, *want)), None) == 0
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    a = args_of(fmpq_mod, X, residual, kind, post, pre, w, *got)
    assert lib.fmpq_block_norm_fault_test(ctypes.addressof(a), row, 1 << 14, None) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 30.0
    lost = (got[0] != want[0]).any(1).nonzero().flatten().tolist()      # (NaN differs)
    steps = {b - a for a, b in zip(lost, lost[1:])}
    assert lost[0] == row and len(steps) <= 1 and (lost[-1] + (steps or {M}).pop()) >= M
    kept = torch.ones(M, dtype=torch.bool, device="cuda")
    kept[lost] = False
    assert bool(got[0][lost].isnan().all()) and torch.equal(got[0][kept], want[0][kept])
    if pre:
        assert bool(got[1][lost].isnan().all()) and torch.equal(got[1][kept], want[1][kept])
        scales, right = got[3][:, :M], want[3][:, :M]
        assert bool(scales[:, lost].isnan().all()) and torch.equal(scales[:, kept], right[:, kept])
        assert torch.equal(got[2][:, kept], want[2][:, kept])
    assert lib.fmpq_block_norm(ctypes.addressof(args_of(fmpq_mod, X, residual, kind, post, pre, w, *again)), None) == 0
    assert all(torch.equal(x, y) for x, y in zip(want, again))


@pytest.mark.gpu
def test_the_hook_refuses(fmpq_mod):  # noqa: F811
    import torch
    X, w, layer = draw(1000, 1024, torch.bfloat16, 1), vectors(1024, torch.bfloat16, 3, 3), fmpq_mod.Fp8Layer(1024, 16)
    R, Y = torch.full_like(X, 7.0), torch.full_like(X, 7.0)
    A, s = layer.activations(1000, X.device)

    def call(row=5, polls=1 << 14, **kw):
        a = args_of(fmpq_mod, X, None, "rms", False, True, w, R, Y, A, s)
        for name, v in kw.items():
            setattr(a, name, v)
        return fmpq_mod._lib.fmpq_block_norm_fault_test(ctypes.addressof(a), row, polls, None)

    assert fmpq_mod._lib.fmpq_block_norm_fault_test(None, 0, 1 << 14, None) == 1
    for code, kw in [(1, dict(row=-1)), (1, dict(row=1000)), (1, dict(polls=1023)), (2, dict(M=100)), (2, dict(dtype=0, param_dtype=0)),
                     (2, dict(param_dtype=2)), (2, dict(ldy=1025)), (2, dict(K=504)), (1, dict(eps=0.0))]:
        assert call(**kw) == code, kw
    torch.cuda.synchronize()
    assert bool((R == 7).all()) and bool((Y == 7).all())


def test_the_hook_refuses_before_a_device():
    """(No GPU.) Arguments, the row and the bound of polls."""
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    lib = fmpq.load_library()
    a = fmpq.BlockNormArgs(X=4096, ldx=512, M=400, K=512, Y=8192, ldy=512, eps=1e-6, residual_scale=1.0, pre_norm=1, dtype=1, param_dtype=1)
    at = ctypes.addressof(a)
    assert lib.fmpq_block_norm_fault_test(None, 0, 1 << 14, None) == 1
    for row, polls in [(-1, 1 << 14), (400, 1 << 14), (1 << 40, 1 << 14), (0, 0), (0, 1023)]:
        assert lib.fmpq_block_norm_fault_test(at, row, polls, None) == 1
    a.ldx = 511
    assert lib.fmpq_block_norm_fault_test(at, 0, 1 << 14, None) == 2
    a.ldx, a.X = 512, 4097
    assert lib.fmpq_block_norm_fault_test(at, 0, 1 << 14, None) == 3
