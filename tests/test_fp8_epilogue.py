"""E4M3 products with bias, activation and residual in their epilogue, against 64 bits; refusals.

Tolerances, with e = 2^-24. The sum before the activation: test_fp8_linear's bound for the product, and e of the value for
the bias. An activation passes that on at most 1.13 times (the steepest slope of the four) and errs itself: exponential
and quotient 2 steps each, products and sums half a step: 16 e of the value; gelu's erfc at an argument that is off by 1.5 e
grows that by 2 x^2 = v^2 times (erfc falls as e^-x^2), and gelu_tanh's exponential at an argument u off by 3 e by 3 |u|,
|u| <= 1.6 (|v| + 0.045 |v|^3). Quotients by more than 2^126 are 0: 1e-35 covers them. The residual's sum rounds once in FP32,
the output by half a step of its type.
"""
import pytest

from tests.test_binding_checks import NoLibrary, elsewhere, f32, half, layer_of, on_gpu, overlapping, u8, weights_of
from tests.test_fp8_linear import draw, fmpq_mod, values, weight_blocks, expand  # noqa: F401  (the fixture)

E = 2.0 ** -24
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


def act64(name, v):
    import torch
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.special.erfc(-v / 2 ** 0.5)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    return v


def check(Y, sum64, off, act, residual, bias=None):
    """Y against act(sum64 + bias) + residual; off: the sum's own error bound."""
    import torch
    info = torch.finfo(Y.dtype)
    v = sum64 if bias is None else sum64 + bias.cpu().double()
    off = off + 2 * E * v.abs()
    a = act64(act, v)
    if act is not None:
        off = 1.13 * off + (16 + 2 * v ** 2 + 5 * 1.6 * (v.abs() + 0.045 * v.abs() ** 3)) * E * a.abs() + 1e-35
    ref = a if residual is None else a + residual.cpu().double()
    off = off + 2 * E * ref.abs()
    bound = off * (1 + info.eps) + ref.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2
    err = (Y.cpu().double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def padded(M, N, dtype, seed, pad, shift=0):
    """Rows with a stride of N + pad, beginning `shift` elements into their buffer."""
    import torch
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((M * (N + pad) + shift,), 7.0, dtype=dtype)
    rows = buf[shift:].view(M, N + pad)
    rows[:, :N] = (torch.randn(M, N, generator=g) * 2).to(dtype)
    return buf.cuda()[shift:].view(M, N + pad)[:, :N]


# M: one token, split K, two warps in turn, 64-token tiles, several of them, 256-token tiles and a rest
SIZES = [(1, 1024, 512, 0, 0), (7, 2048, 130, 8, 0), (32, 4096, 1000, 4, 4), (33, 300, 257, 1, 1), (64, 512, 8192, 0, 0),
         (100, 256, 20000, 0, 0), (300, 260, 515, 5, 0), (520, 384, 1028, 4, 4), (777, 512, 640, 0, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,pad,shift", SIZES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_epilogue(fmpq_mod, M, K, N, pad, shift, act, dtype):  # noqa: F811
    import torch
    dtype = getattr(torch, dtype)
    g = torch.Generator().manual_seed(M + N)
    X = draw(M, K, dtype, M + N)
    w = (torch.randn(N, K, generator=g) * 2 / K ** 0.5).to(dtype)
    layer = fmpq_mod.Fp8Layer(K, N)
    W = fmpq_mod.fp8_pack_weights(layer, w.cuda())
    bias = torch.randn(N, generator=g).to(torch.float32 if N % 2 else dtype).cuda()
    residual = padded(M, N, dtype, M, pad, shift)
    x, wv = values(X), expand(*weight_blocks(w))
    nb = -(-K // 128)
    sum64, off = x @ wv.t(), (K + 2 * nb + 2) * 2 * E * (x.abs() @ wv.abs().t())
    Y = fmpq_mod.fp8_quantize_gemm(layer, X, *W, bias=bias, activation=act, residual=residual)
    check(Y, sum64, off, act, residual, bias)
    A = fmpq_mod.fp8_quantize(layer, X)
    out = torch.full((M, N + 3), 7.0, dtype=dtype, device="cuda")
    Z = fmpq_mod.fp8_gemm(layer, *A, *W, M, Y=out[:, :N], bias=bias, activation=act, residual=residual)
    assert torch.equal(Y, Z) and bool((out[:, N:] == 7).all())
    check(fmpq_mod.fp8_quantize_gemm(layer, X, *W, bias=bias, activation=act), sum64, off, act, None, bias)
    check(fmpq_mod.fp8_gemm(layer, *A, *W, M, dtype=dtype, activation=act, residual=residual), sum64, off, act, residual)
    # in place of the residual
    fmpq_mod.fp8_quantize_gemm(layer, X, *W, bias=bias, activation=act, residual=residual, Y=residual)
    assert torch.equal(residual, Y)
    if pad:
        assert bool((residual.as_strided((M - 1, pad), (N + pad, 1), residual.storage_offset() + N) == 7).all())
    assert fmpq_mod.fp8_device_status(layer) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 32, 50, 300])
def test_an_epilogue_that_adds_nothing_changes_nothing(fmpq_mod, M):  # noqa: F811
    import torch
    K, N = 1000, 776
    X = draw(M, K, torch.bfloat16, M)
    layer = fmpq_mod.Fp8Layer(K, N)
    W = fmpq_mod.fp8_pack_weights(layer, draw(N, K, torch.bfloat16, 1))
    Y = fmpq_mod.fp8_quantize_gemm(layer, X, *W)
    zeros = torch.zeros(M, N, dtype=X.dtype, device="cuda")
    assert torch.equal(Y, fmpq_mod.fp8_quantize_gemm(layer, X, *W, bias=zeros[0], residual=zeros))
    Z = fmpq_mod.fp8_quantize_gemm(layer, X, *W, activation="relu")
    assert torch.equal(Z, Y.clamp_min(0))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 40, 300])
@pytest.mark.parametrize("act", ACTS)
def test_nan_infinity_and_extremes(fmpq_mod, M, act):  # noqa: F811
    """NaN and infinity of a residual, a bias or a token reach their own outputs alone; arguments from -200 to 200."""
    import torch
    K, N = 256, 400
    X = draw(M, K, torch.bfloat16, M)
    layer = fmpq_mod.Fp8Layer(K, N)
    W = fmpq_mod.fp8_pack_weights(layer, torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"))
    bias = torch.linspace(-200, 200, N).cuda()
    residual = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    check(fmpq_mod.fp8_quantize_gemm(layer, X, *W, bias=bias, activation=act), torch.zeros(M, N).double(), 0, act, None, bias)
    residual[1, 2], residual[M - 1, N - 1] = float("nan"), float("-inf")
    bias[5], bias[6] = float("nan"), float("inf")
    X[3, 0] = float("nan")
    Y = fmpq_mod.fp8_quantize_gemm(layer, X, *W, bias=bias, activation=act, residual=residual)
    assert bool(Y[3].isnan().all()) and bool(Y[:, 5].isnan().all()) and bool(Y[1, 2].isnan())
    assert float(Y[M - 1, N - 1]) == float("-inf") and float(Y[0, 6]) == float("inf")
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3], bad[:, 5:7], bad[1, 2], bad[M - 1, N - 1] = True, True, True, True
    assert bool(torch.isfinite(Y[~bad]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 32, 300])
def test_graph_and_stream(fmpq_mod, M):  # noqa: F811
    """A block's second half on a stream and captured: the residual is updated in place at every replay."""
    import torch
    K, N = 4096, 1024
    X, start = draw(M, K, torch.bfloat16, M), padded(M, N, torch.bfloat16, 3, 0)
    layer = fmpq_mod.Fp8Layer(K, N)
    W = fmpq_mod.fp8_pack_weights(layer, draw(N, K, torch.bfloat16, 1))
    kw = dict(bias=draw(1, N, torch.bfloat16, 2)[0], activation="gelu")
    ref = start.clone()
    for _ in range(3):
        fmpq_mod.fp8_quantize_gemm(layer, X, *W, residual=ref, Y=ref, **kw)
    r = start.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fmpq_mod.fp8_quantize_gemm(layer, X, *W, residual=r, Y=r, **kw)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = start.clone()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        fmpq_mod.fp8_quantize_gemm(layer, X, *W, residual=r, Y=r, stream=side, **kw)
    side.synchronize()
    assert torch.equal(r, ref)


# ---- refusals (no GPU) ------------------------------------------------------------------------

@pytest.fixture
def no_gpu(monkeypatch):
    from bit_quantized_gemm_fmpq_gb300 import fmpq
    monkeypatch.setattr(fmpq, "load_library", NoLibrary)
    monkeypatch.setattr(fmpq, "_lib", NoLibrary())
    monkeypatch.setattr(fmpq, "_on", lambda X: 0)
    monkeypatch.setattr(fmpq, "_device", lambda: 0)
    monkeypatch.setattr(fmpq, "_stream", lambda s: 0)


def test_the_binding_refuses(no_gpu):
    import torch

    from bit_quantized_gemm_fmpq_gb300 import fmpq
    layer = layer_of(256, 128)
    W, s = weights_of(layer)
    X, Y = half(5, 256), half(5, 128)
    flat = half(5 * 128 + 64)
    bad = [dict(bias=half(127)), dict(bias=half(1, 128)), dict(bias=half(256)[::2]), dict(bias=torch.zeros(128)),
           dict(bias=on_gpu(torch.zeros(128, dtype=torch.bfloat16))), dict(bias=elsewhere(f32(128))), dict(activation="tanh"),
           dict(residual=half(5, 127)), dict(residual=f32(5, 128)), dict(residual=half(4, 128)), dict(residual=torch.zeros(5, 128).half()),
           dict(residual=overlapping(5, 128)[0]), dict(residual=elsewhere(half(5, 128))),
           dict(residual=flat[:640].view(5, 128), Y=flat[64:].view(5, 128)), dict(bias=Y[0], Y=Y)]
    for kw in bad:
        for call in (lambda kw: fmpq.fp8_quantize_gemm(layer, X, W, s, workspace=half(8), **kw),
                     lambda kw: fmpq.fp8_gemm(layer, u8(2, 5, 128), f32(2, 8), W, s, 5, workspace=half(8), **kw)):
            with pytest.raises(ValueError):
                call(kw)
                raise AssertionError(f"{kw} was not refused")


def test_the_library_refuses():
    import ctypes

    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    lib = fmpq.load_library()
    z, e = None, fmpq.Epilogue()
    assert lib.fp8_gemm_epilogue(z, z, z, z, z, 1, z, z, 0, 8, z, 0, z) == 1
    assert lib.fp8_gemm_epilogue(z, z, z, z, z, 1, ctypes.addressof(e), z, 0, 8, z, 0, z) == 1
    assert lib.fp8_quantize_gemm_epilogue(z, z, 0, 8, 1, z, z, z, z, z, z, 8, z, 0, z) == 1


@pytest.mark.gpu
def test_the_library_refuses_epilogues(fmpq_mod):  # noqa: F811
    """Bad epilogues on good buffers: an error, and nothing is written."""
    import ctypes

    import torch
    M, K, N = 4, 128, 64
    layer = fmpq_mod.Fp8Layer(K, N)
    X = draw(M, K, torch.float16, 1)
    W = fmpq_mod.fp8_pack_weights(layer, draw(N, K, torch.float16, 2))
    A = fmpq_mod.fp8_quantize(layer, X)
    Y = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
    extra = torch.zeros(4096, dtype=torch.float32, device="cuda").data_ptr()
    for code, kw in [(1, dict(activation=5)), (1, dict(activation=-1)), (1, dict(bias=extra, bias_dtype=1)), (1, dict(bias=extra, bias_dtype=3)),
                     (2, dict(residual=extra, ldr=63)), (3, dict(residual=extra + 1, ldr=64)), (3, dict(bias=extra + 2, bias_dtype=2))]:
        e = fmpq_mod.Epilogue(**kw)
        assert fmpq_mod._lib.fp8_gemm_epilogue(layer.handle, A[0].data_ptr(), A[1].data_ptr(), W[0].data_ptr(), W[1].data_ptr(), M,
                                               ctypes.addressof(e), Y.data_ptr(), 0, N, None, 0, None) == code, kw
        assert fmpq_mod._lib.fp8_quantize_gemm_epilogue(layer.handle, X.data_ptr(), 0, K, M, A[0].data_ptr(), A[1].data_ptr(),
                                                        W[0].data_ptr(), W[1].data_ptr(), ctypes.addressof(e), Y.data_ptr(), N, None, 0,
                                                        None) == code, kw
    torch.cuda.synchronize()
    assert bool((Y == 7).all())
