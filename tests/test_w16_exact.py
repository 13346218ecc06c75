"""16-bit layers on small whole numbers, where FP32 sums are exact in any order: FP32 outputs equal the 64-bit product, 16-bit outputs its one rounding,
bit for bit. A channel left out or counted twice, a part of K rounded on its way, a second rounding of the output: each shows.

X and W are drawn from -3 .. 3 without 0, so every channel and every block of each part of K counts; K * 9 < 2^24, and biases, residuals and a gated layer's
products stay below 2^24 too (asserted), so no step of the definition rounds.
"""
import pytest

from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)


def whole(shape, dtype, seed, most=3):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(1, most + 1, shape, generator=g, device="cuda")
    return (v * (1 - 2 * torch.randint(0, 2, shape, generator=g, device="cuda"))).to(dtype)


def product(x, w, bias=None, gated=False, residual=None, row_weight=None):
    import torch
    v = x.double() @ w.double().t()
    if bias is not None:
        v = v + bias.double()
    assert float(v.abs().max()) < 2 ** 24
    if gated:
        F = w.shape[0] // 2
        v = v[:, :F] * v[:, F:]
    if row_weight is not None:
        v = v * row_weight.double()[:, None]
    if residual is not None:
        v = v + residual.double()
    assert float(v.abs().max()) < 2 ** 24 and bool((v == v.round()).all())
    return v.float() if v.dtype == torch.float64 else v


def equal(Y, exact):
    import torch
    want = exact.to(Y.dtype)
    assert torch.equal(Y, want), f"{int((Y != want).sum())} of {Y.numel()} differ"


# few units: K in 4 parts, in 2, in 1; rows that are copied first; units of two parts (above 256 rows); several rounds; a rest in a launch of its own, with K in parts
SIZES = [(1, 8192, 1024, 0), (1, 6400, 512, 0), (1, 2048, 512, 0), (16, 8192, 1024, 0), (1, 8192, 8192, 0), (128, 8192, 8192, 0), (257, 4096, 256, 0),
         (40, 4100, 300, 1), (3, 65536, 130, 0), (777, 2048, 5632, 0), (600, 512, 770, 3), (1500, 520, 1030, 0), (300, 4096, 20480, 0), (1, 8192, 28672, 0),
         (2048, 4096, 12288, 0), (520, 2048, 10000, 8), (5, 64, 300, 0), (33, 1, 200, 0), (70, 129, 515, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,pad", SIZES)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_one_matrix(fmpq_mod, M, K, N, pad, dtype):  # noqa: F811
    import torch
    dtype = getattr(torch, dtype)
    X, W = whole((M, K + pad), dtype, M + K)[:, :K], whole((N, K), dtype, N)
    layer = fmpq_mod.W16Layer(K, N, dtype)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    sums = product(X, W)
    equal(fmpq_mod.w16_gemm(layer, X, Wp, dtype=torch.float32), sums)
    equal(fmpq_mod.w16_gemm(layer, X, Wp), sums)
    bias, residual = whole((N,), torch.float32, 5, 2047), whole((M, N), dtype, 6, 255)
    exact = product(X, W, bias, residual=residual)
    equal(fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, residual=residual), exact)
    equal(fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, residual=residual.float(), dtype=torch.float32), exact)
    equal(fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="relu"), product(X, W, bias).clamp_min(0))
    assert fmpq_mod.w16_device_status(layer) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,F", [(1, 4096, 512), (1, 2048, 128), (20, 640, 200), (300, 200, 1000), (700, 1024, 384), (130, 4096, 66), (2000, 512, 1300)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gated(fmpq_mod, M, K, F, dtype):  # noqa: F811
    import torch
    dtype = getattr(torch, dtype)
    X, W = whole((M, K), dtype, M), whole((2 * F, K), dtype, F)
    layer = fmpq_mod.W16Layer(K, 2 * F, dtype, gated=True)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    equal(fmpq_mod.w16_gemm(layer, X, Wp, dtype=torch.float32), product(X, W, gated=True))
    bias, residual = whole((2 * F,), torch.float32, 5, 30), whole((M, F), dtype, 6, 255)
    exact = product(X, W, bias, True, residual)
    equal(fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, residual=residual), exact)
    equal(fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, residual=residual.float(), dtype=torch.float32), exact)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,K,N,gated", [
    ([0] * 30 + [1] + [0] * 34, 6400, 512, False), ([1, 0, 2, 0, 0], 4096, 300, True), ([4, 5], 2048, 520, False),       # K in parts
    ([8, 0, 31, 33, 1, 64], 1404, 2012, False), ([700, 3, 0, 257, 300, 512], 520, 770, False), ([255, 256, 258, 1100, 0, 90], 256, 512, True),
    ([i * 7 % 61 for i in range(128)], 512, 256, True), ([300], 1024, 5000, False)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_groups(fmpq_mod, sizes, K, N, gated, dtype):  # noqa: F811
    import torch
    dtype = getattr(torch, dtype)
    E, rows, out_n = len(sizes), sum(sizes), N // 2 if gated else N
    ends = [sum(sizes[:e]) for e in range(E + 1)]
    X, W = whole((rows, K), dtype, rows), whole((E, N, K), dtype, N)
    bias, residual, weight = whole((E, N), torch.float32, 3, 30), whole((rows, out_n), dtype, 4, 255), whole((rows,), torch.float32, 5, 2)
    layer = fmpq_mod.W16Layer(K, N, dtype, experts=E, gated=gated)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    bare = torch.cat([product(X[ends[e]:ends[e + 1]], W[e], gated=gated) for e in range(E) if sizes[e]])
    full = torch.cat([product(X[at], W[e], bias[e], gated, residual[at], weight[at]) for e, at in
                      ((e, slice(ends[e], ends[e + 1])) for e in range(E) if sizes[e])])
    equal(fmpq_mod.w16_grouped_gemm(layer, X, offsets, Wp), bare)
    equal(fmpq_mod.w16_grouped_gemm(layer, X, offsets, Wp, dtype=torch.float32), bare)
    equal(fmpq_mod.w16_grouped_gemm(layer, X, offsets, Wp, bias=bias, residual=residual, row_weight=weight), full)
    equal(fmpq_mod.w16_grouped_gemm(layer, X, offsets, Wp, bias=bias, residual=residual.float(), row_weight=weight, dtype=torch.float32), full)
    assert fmpq_mod.w16_device_status(layer) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,K,N", [(1, 4, 16, 4096, 256), (50, 3, 8, 300, 136), (600, 2, 5, 1500, 384), (9, 8, 40, 8192, 128)])
def test_experts_on_a_plan(fmpq_mod, T, k, E, K, N):  # noqa: F811
    """Tokens gathered to their experts' rows, whole pair weights, the sum over the slots."""
    import torch
    X, W, weights = whole((T, K), torch.bfloat16, T), whole((E, N, K), torch.bfloat16, N), whole((T, k), torch.float32, 3, 2)
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    ids[T // 2, 0] = -1
    plan = fmpq_mod.moe_plan(ids.cuda(), E)
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16, experts=E)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    D = fmpq_mod.w16_experts_gemm(layer, plan, X, Wp, weights=weights, dtype=torch.float32)
    want = torch.zeros(T, N, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            one = product(X[t.cuda()], W[e], row_weight=weights[t.cuda(), j.cuda()])
            equal(D[plan.row_of[t.cuda(), j.cuda()].long()], one)
            want.index_add_(0, t.cuda(), one)
    equal(fmpq_mod.moe_combine(D, plan), want)


# ---- what these tests would see (no GPU) ------------------------------------------------------

def test_faults_show():
    """On the CPU: a last channel left out, a split K's parts rounded to 16 bits, and an output rounded twice all change the comparison's outputs."""
    import torch
    g = torch.Generator().manual_seed(1)
    draw = lambda *s: torch.randint(1, 4, s, generator=g).double() * (1 - 2 * torch.randint(0, 2, s, generator=g))      # noqa: E731
    x, w = draw(1, 6400), draw(512, 6400)
    sums = x @ w.t()
    assert not torch.equal(sums.float(), (x[:, :-1] @ w[:, :-1].t()).float())
    parts = [x[:, i:i + 1600] @ w[:, i:i + 1600].t() for i in range(0, 6400, 1600)]
    assert torch.equal(sum(p.float() for p in parts), sums.float())
    assert not torch.equal(sum(p.bfloat16().float() for p in parts), sums.float())
    residual = torch.randint(-255, 256, (1, 512), generator=g).double()
    assert not torch.equal((sums.bfloat16().float() + residual.float()).bfloat16(), (sums + residual).bfloat16())
