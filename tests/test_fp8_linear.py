"""E4M3 linear layers with a scale for each block of 128: codes and scales against the definition,
products against 64-bit sums, refusals.

Tolerances. Codes and scales are exact. A product's FP32 sums are off by at most (K + 2 nb + 2) steps of
2^-23 of the sum of the absolute products (every addition and scaling rounds once, at worst by
truncation); the output's rounding by half a step, finfo.eps / 2 of the value (or half the smallest
fp16 number). Over a whole matrix the FP32 part is far smaller than that bound, so the norm of the
error is held to eps / 2 + 1e-5 of the norm.
"""
import ctypes

import pytest

BLOCK = 128


# ---- the definition, in 64 bits on the CPU ----------------------------------------------------

def quantized(x):
    """(codes as values, scales) per row and 128 channels; x [rows, K] any float type."""
    import torch
    rows, K = x.shape
    nb = -(-K // BLOCK)
    b = torch.zeros(rows, nb * BLOCK)
    b[:, :K] = x.float().cpu()
    b = b.view(rows, nb, BLOCK)
    s = b.abs().amax(2) / torch.full((rows, nb), 448.0)
    q = torch.where(s[:, :, None] > 0, b / s[:, :, None], torch.zeros(()))
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).double().view(rows, -1)[:, :K], s


def values(x):
    q, s = quantized(x)
    return q * s.double().repeat_interleave(BLOCK, 1)[:, :x.shape[1]]


def weight_blocks(w):
    """(codes as values, scales [N / 128, nb]) of a matrix quantized per 128 x 128 block."""
    import torch
    N, K = w.shape
    w = w.float().cpu()
    s = torch.zeros(-(-N // BLOCK), -(-K // BLOCK))
    q = torch.zeros(N, K, dtype=torch.float64)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            blk = w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            s[i, j] = (blk.abs().max().view(1) / torch.tensor([448.0]))[0]
            if s[i, j] > 0:
                q[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = (
                    (blk / s[i, j].expand_as(blk)).clamp(-448, 448).to(torch.float8_e4m3fn).double())
    return q, s


def expand(q, s):
    N, K = q.shape
    return q * s.double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def decode_activations(A, rows, K):
    """Codes as values [rows, K] from the packed (swizzled) layout [nb, rows, 128]."""
    import torch
    nb = A.shape[0]
    v = A.cpu().view(torch.float8_e4m3fn).double().view(nb, rows, 8, 16)
    r = torch.arange(rows)[:, None]
    c = torch.arange(8)[None, :]
    v = v[:, r, c ^ (r % 8)]                      # [nb, rows, 8, 16] in channel order
    return v.reshape(nb, rows, BLOCK).permute(1, 0, 2).reshape(rows, nb * BLOCK)


def check_product(Y, x, w):
    """Y against x w^T (x, w: the exact values in 64 bits)."""
    import torch
    Y = Y.cpu()
    K, nb = x.shape[1], -(-x.shape[1] // BLOCK)
    ref, size = x @ w.t(), x.abs() @ w.abs().t()
    eps = torch.finfo(Y.dtype).eps / 2
    tiny = torch.finfo(Y.dtype).smallest_normal * torch.finfo(Y.dtype).eps / 2
    bound = ref.abs() * eps + tiny + (K + 2 * nb + 2) * 2.0 ** -23 * size
    err = (Y.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert float(err.norm()) <= (eps + 1e-5) * float(ref.norm()) + tiny * ref.numel() ** 0.5


# ---- refusals (no GPU) ------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    return fmpq.load_library()


@pytest.mark.parametrize("K,N,experts,gated,code", [
    (0, 128, 1, 0, 2), (128, 0, 1, 0, 2), (70000, 128, 1, 0, 2), (128, 128, 0, 0, 2), (128, 128, 1025, 0, 2),
    (128, 129, 1, 1, 2), (128, 128, 1, 2, 1),
])
def test_layer_sizes_refused(lib, K, N, experts, gated, code):
    out = ctypes.c_void_p()
    assert lib.fp8_layer_create(K, N, experts, gated, ctypes.byref(out)) == code
    assert not out.value


def test_null_arguments_refused(lib):
    z = None
    assert lib.fp8_layer_create(128, 128, 1, 0, None) == 1
    assert lib.fp8_quantize(z, z, 0, 8, 1, z, z, z) == 1
    assert lib.fp8_pack_weights(z, 0, z, 0, 8, z, z, z) == 1
    assert lib.fp8_pack_codes(z, 0, z, 8, z, z) == 1
    assert lib.fp8_unpack_weights(z, 0, z, z, z, z) == 1
    assert lib.fp8_gemm(z, z, z, z, z, 1, z, 0, 8, z, 0, z) == 1
    assert lib.fp8_quantize_gemm(z, z, 0, 8, 1, z, z, z, z, z, 8, z, 0, z) == 1
    assert lib.fp8_device_status(z, None, 0) == 1
    assert lib.fp8_packed_w_bytes(z) == 0 and lib.fp8_gemm_workspace_bytes(z, 4) == 0
    lib.fp8_layer_destroy(z)


# ---- on the GPU -------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def fmpq_mod():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    fmpq.load_library()
    return fmpq


def draw(M, K, dtype, seed, pad=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.rand(K, generator=g) < 0.1] *= 50
    if M > 2:
        x[1] = 0                     # a token of zeros: scale 0
    buf = torch.empty(M, K + pad, dtype=dtype, device="cuda")
    buf[:, :K] = x.to(dtype).cuda()
    return buf[:, :K]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,pad,offset", [
    (1, 1, 0, 0), (1, 128, 0, 0), (3, 127, 1, 0), (7, 129, 0, 0), (130, 520, 8, 0), (64, 1000, 24, 3), (257, 4096, 0, 0),
])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantize_exact(fmpq_mod, M, K, pad, offset, dtype):
    import torch
    X = draw(M, K, getattr(torch, dtype), 7 * M + K, pad)
    if offset:                       # rows that start off the 16-byte boundary
        flat = torch.empty(M * (K + pad) + offset, dtype=X.dtype, device="cuda")
        view = flat[offset:].view(M, K + pad)[:, :K]
        view.copy_(X)
        X = view
    layer = fmpq_mod.Fp8Layer(K, 128)
    A, s = fmpq_mod.fp8_quantize(layer, X)
    q, sr = quantized(X)
    assert torch.equal(s.cpu()[:, :M].t(), sr)
    got = decode_activations(A, M, K)
    assert torch.equal(got[:, :K], q)
    assert bool((got[:, K:] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M,K", [(9, 128), (640, 8192)])
def test_quantize_values_between_two_codes(fmpq_mod, M, K, dtype):
    """Every block holds its absmax and the 126 midpoints of neighbouring codes times its scale, rounded to the
    type, and the values next to them."""
    import torch
    dtype = getattr(torch, dtype)
    g = torch.Generator().manual_seed(M)
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    middles = (codes[1:] + codes[:-1]) / 2
    amax = torch.exp(torch.empty(M, K // BLOCK, 1).uniform_(-6, 6, generator=g)).to(dtype)
    x = ((amax.float() / 448) * middles).to(dtype)
    bits = x.view(torch.int16)       # (a zero has no neighbour below)
    x = (bits + torch.randint(-1, 2, x.shape, generator=g, dtype=torch.int16)).clamp(min=0).view(dtype)
    x = x * (torch.randint(0, 2, x.shape, generator=g) * 2 - 1).to(dtype)
    x = torch.minimum(torch.maximum(x, -amax), amax)
    X = torch.cat([amax, torch.zeros_like(amax), x], 2).reshape(M, K)
    A, s = fmpq_mod.fp8_quantize(fmpq_mod.Fp8Layer(K, 128), X.cuda())
    q, sr = quantized(X)
    assert torch.equal(s.cpu()[:, :M].t(), sr)
    assert torch.equal(decode_activations(A, M, K), q)


@pytest.mark.gpu
def test_quantize_tiny_and_large_values(fmpq_mod):
    import torch
    X = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    X[0, 3] = 3e38
    X[1, :] = 1e-38                  # a scale in the subnormal range
    X[2, 200] = -6e-39
    X[3, :128] = torch.linspace(-1, 1, 128)
    X[4, 0], X[4, 1] = 448.0, 2.0 ** -10     # a tie between 0 and the smallest code
    layer = fmpq_mod.Fp8Layer(256, 128)
    A, s = fmpq_mod.fp8_quantize(layer, X)
    q, sr = quantized(X)
    assert torch.equal(s.cpu()[:, :8].t(), sr)
    assert torch.equal(decode_activations(A, 8, 256), q)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,gated", [(1, 1, False), (130, 200, False), (384, 129, False), (2, 64, True), (300, 257, True)])
def test_weights_pack_and_unpack(fmpq_mod, N, K, gated):
    import torch
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(N + K)).to(torch.bfloat16)
    layer = fmpq_mod.Fp8Layer(K, N, gated=gated)
    Wp, s = fmpq_mod.fp8_pack_weights(layer, w.cuda())
    halves = [w[:N // 2], w[N // 2:]] if gated else [w]
    parts = [weight_blocks(h) for h in halves]
    assert torch.equal(s[0].cpu(), torch.cat([p[1] for p in parts]))
    ref = torch.cat([expand(*p) for p in parts])
    assert torch.equal(fmpq_mod.fp8_unpack_weights(layer, Wp, s).cpu().double(), ref.float().double())
    codes = torch.cat([p[0] for p in parts]).float().to(torch.float8_e4m3fn)
    Wp2, s2 = fmpq_mod.fp8_pack_codes(layer, codes.cuda(), s[0])
    assert torch.equal(Wp2, Wp) and torch.equal(s2[0], s[0])


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [
    (1, 1, 1), (1, 8192, 256), (2, 300, 130), (16, 512, 512), (17, 128, 4004), (31, 2868, 100), (32, 1024, 300),
    (33, 640, 264), (64, 4096, 520), (65, 129, 257), (100, 2000, 1000), (129, 384, 768), (255, 256, 136), (256, 1024, 256),
    (257, 640, 513), (300, 1536, 1300), (515, 2868, 404), (1000, 512, 2304),
    # more tiles than pairs of CTAs
    (64, 200, 20500), (130, 384, 20500), (1000, 256, 5001),
])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_product(fmpq_mod, M, K, N, dtype):
    import torch
    dtype = getattr(torch, dtype)
    X = draw(M, K, dtype, M + K + N, pad=(N % 3) * 4)
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(N)) * 0.02).to(dtype)
    layer = fmpq_mod.Fp8Layer(K, N)
    Wp, s = fmpq_mod.fp8_pack_weights(layer, w.cuda())
    out = torch.full((M, N + 5), 7.0, dtype=dtype, device="cuda")   # a padded output: nothing past N is written
    Y = fmpq_mod.fp8_quantize_gemm(layer, X, Wp, s, Y=out[:, :N])
    check_product(Y, values(X), expand(*weight_blocks(w)))
    assert bool((out[:, N:] == 7.0).all())
    again = fmpq_mod.fp8_gemm(layer, *fmpq_mod.fp8_quantize(layer, X), Wp, s, M, dtype=dtype)
    assert torch.equal(again, Y)     # another call, another output stride: the same sums
    assert fmpq_mod.fp8_device_status(layer) == 0


@pytest.mark.gpu
def test_product_on_streams_and_in_a_graph(fmpq_mod):
    import torch
    layer = fmpq_mod.Fp8Layer(2048, 640)
    w = (torch.randn(640, 2048, generator=torch.Generator().manual_seed(1)) * 0.02).to(torch.bfloat16)
    Wp, s = fmpq_mod.fp8_pack_weights(layer, w.cuda())
    xs = [draw(m, 2048, torch.bfloat16, m) for m in (1, 40, 300)]
    want = [fmpq_mod.fp8_quantize_gemm(layer, x, Wp, s) for x in xs]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, st in zip(xs, side):
        with torch.cuda.stream(st):
            got.append([fmpq_mod.fp8_quantize_gemm(layer, x, Wp, s) for _ in range(3)])
    torch.cuda.synchronize()
    for w_, g in zip(want, got):
        assert all(torch.equal(w_, y) for y in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [fmpq_mod.fp8_quantize_gemm(layer, x, Wp, s) for x in xs]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.gpu
def test_stream_argument(fmpq_mod):
    """stream= (a torch stream or its handle) runs and allocates there: scratch is not reused early."""
    import torch
    layer = fmpq_mod.Fp8Layer(4096, 1024)
    w = (torch.randn(1024, 4096, generator=torch.Generator().manual_seed(2)) * 0.02).to(torch.bfloat16)
    Wp, s = fmpq_mod.fp8_pack_weights(layer, w.cuda())
    xs = [draw(m, 4096, torch.bfloat16, m) for m in (3, 200, 1500)]
    want = [fmpq_mod.fp8_quantize_gemm(layer, x, Wp, s) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for i in range(6):
        x = xs[i % 3]
        got.append(fmpq_mod.fp8_quantize_gemm(layer, x, Wp, s, stream=side if i < 3 else side.cuda_stream))
        junk = torch.full((1 << 22,), float(i), device="cuda")      # work on the current stream meanwhile
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got)) and float(junk[0]) == 5.0


@pytest.mark.gpu
def test_binding_refusals(fmpq_mod):
    import torch
    layer = fmpq_mod.Fp8Layer(256, 128)
    Wp, s = fmpq_mod.fp8_pack_weights(layer, torch.zeros(128, 256, dtype=torch.float16, device="cuda"))
    X = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    for bad in (X.float(), X.cpu(), X[:, :255], X.t(), X[0]):
        with pytest.raises(ValueError):
            fmpq_mod.fp8_quantize_gemm(layer, bad, Wp, s)
    with pytest.raises(ValueError):
        fmpq_mod.fp8_quantize_gemm(layer, X, Wp, s, Y=torch.empty(4, 127, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        fmpq_mod.fp8_pack_codes(layer, torch.zeros(128, 256, device="cuda"), s)
    with pytest.raises(fmpq_mod.FmpqError):
        fmpq_mod.fp8_quantize_gemm(layer, X[:0], Wp, s)
    for kw in (dict(W_packed=Wp[:-16], w_scales=s), dict(W_packed=Wp, w_scales=s[:, :, :1]),
               dict(W_packed=Wp, w_scales=s, A_packed=torch.empty(4, dtype=torch.uint8, device="cuda"), a_scales=s),
               dict(W_packed=Wp, w_scales=s, A_packed=torch.empty(4096, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            fmpq_mod.fp8_quantize_gemm(layer, X, **kw)
    gated = fmpq_mod.Fp8Layer(256, 256, gated=True)
    with pytest.raises(fmpq_mod.FmpqError):
        fmpq_mod.fp8_gemm(gated, *fmpq_mod.fp8_quantize(gated, X), Wp, s, 4)
