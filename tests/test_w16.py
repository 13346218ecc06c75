"""Layers kept in 16 bits: products of one matrix and of ragged groups with a matrix each, against 64 bits; refusals.

Tolerances. Products of two 16-bit values are exact in FP32; a sum of K of them on the tensor core is off by at most K + 2 steps
of 2^-23 of the absolute products (every addition at worst truncates), K split in up to 4 parts by 3 more. What follows, and the
output's rounding, as in test_fp8_epilogue; a gated output is act(gate) * up, off by each factor's error times the other and one
rounding; row_weight rounds once.
"""
import pytest

from tests.test_binding_checks import NoLibrary, elsewhere, f32, half, on_gpu, overlapping, plan_of
from tests.test_fp8_epilogue import ACTS, E, act64, padded
from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)


def product64(x, w):
    """The sum and its error bound."""
    x, w = x.cpu().double(), w.cpu().double()
    return x @ w.t(), (x.shape[1] + 5) * 2 * E * (x.abs() @ w.abs().t())


def activated(sum64, off, act, bias):
    v = sum64 if bias is None else sum64 + bias.cpu().double()
    off = off + 2 * E * v.abs()
    a = act64(act, v)
    if act is not None:
        off = 1.13 * off + (16 + 2 * v ** 2 + 5 * 1.6 * (v.abs() + 0.045 * v.abs() ** 3)) * E * a.abs() + 1e-35
    return a, off


def check(Y, x, w, act=None, bias=None, residual=None, row_weight=None, gated=False):
    import torch
    s, off = product64(x, w)
    if gated:
        F = w.shape[0] // 2
        b, bu = (None, None) if bias is None else (bias[:F], bias[F:])
        a, oa = activated(s[:, :F], off[:, :F], act, b)
        u, ou = activated(s[:, F:], off[:, F:], None, bu)
        ref, off = a * u, oa * u.abs() + ou * a.abs() + oa * ou + 2 * E * (a * u).abs()
    else:
        ref, off = activated(s, off, act, bias)
    if row_weight is not None:
        ref = ref * row_weight.cpu().double()[:, None]
        off = off * row_weight.cpu().double().abs()[:, None] + 2 * E * ref.abs()
    if residual is not None:
        ref = ref + residual.cpu().double()
        off = off + 2 * E * ref.abs()
    info = torch.finfo(Y.dtype)
    bound = off * (1 + info.eps) + ref.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2
    err = (Y.cpu().double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def matrix(rows, K, dtype, seed, pad=0, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    out = torch.full((rows, K + pad), 7.0, dtype=dtype)
    out[:, :K] = (torch.randn(rows, K, generator=g) * scale).to(dtype)
    return out.cuda()[:, :K]


# ---- one matrix -------------------------------------------------------------------------------

# one row; K split by 4, by 2; several tiles; odd everything; one channel; rows that need aligning; wide
SIZES = [(1, 2048, 512, 0, 0), (5, 1024, 300, 0, 0), (40, 1536, 4000, 8, 0), (33, 300, 257, 1, 1), (64, 64, 130, 0, 0), (3, 1, 1, 0, 0),
         (130, 200, 6000, 4, 4), (300, 260, 515, 5, 0), (700, 192, 1028, 3, 4), (1500, 512, 770, 0, 0), (257, 4096, 256, 0, 0),
         (300, 128, 20000, 0, 0), (513, 64, 19999, 0, 0),
         # full rounds, and a rest in a launch of its own
         (300, 1024, 20000, 0, 0), (520, 2048, 10000, 8, 0), (1000, 1500, 12345, 0, 1), (2000, 1024, 10240, 0, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,pad,shift", SIZES)
@pytest.mark.parametrize("act", [None, "gelu"])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_one_matrix(fmpq_mod, M, K, N, pad, shift, act, dtype):  # noqa: F811
    import torch
    dtype = getattr(torch, dtype)
    X, W = matrix(M, K, dtype, M + N, pad), matrix(N, K, dtype, N, 0, 2 / K ** 0.5)
    layer = fmpq_mod.W16Layer(K, N, dtype)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    assert torch.equal(Wp, fmpq_mod.w16_pack_weights(layer, W.t().contiguous().t()))    # a checkpoint that holds [K, N]
    bias = matrix(1, N, dtype if N % 2 else torch.float32, 5)[0]
    residual = padded(M, N, dtype, M, pad, shift)
    check(fmpq_mod.w16_gemm(layer, X, Wp), X, W)
    Y = fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation=act, residual=residual)
    check(Y, X, W, act, bias, residual)
    out = torch.full((M, N + 3), 7.0, dtype=dtype, device="cuda")
    fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation=act, residual=residual, Y=out[:, :N])
    assert torch.equal(out[:, :N], Y) and bool((out[:, N:] == 7).all())
    wide = torch.full((M, N + 3), 7.0, device="cuda")
    fmpq_mod.w16_gemm(layer, X, Wp, bias=bias.float(), activation=act, residual=residual.float(), Y=wide[:, :N])
    check(wide[:, :N], X, W, act, bias, residual)
    assert bool((wide[:, N:] == 7).all())
    fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation=act, residual=residual, Y=residual)
    assert torch.equal(residual, Y)
    assert fmpq_mod.w16_device_status(layer) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,F", [(1, 1024, 512), (20, 640, 200), (100, 256, 65), (300, 200, 1000), (600, 512, 384)])
@pytest.mark.parametrize("act", ACTS)
def test_gated(fmpq_mod, M, K, F, act):  # noqa: F811
    import torch
    dtype = torch.bfloat16 if F % 2 else torch.float16
    X, W = matrix(M, K, dtype, M), matrix(2 * F, K, dtype, F, 0, 1.5 / K ** 0.5)
    layer = fmpq_mod.W16Layer(K, 2 * F, dtype, gated=True)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    bias, residual = matrix(1, 2 * F, dtype, 5)[0], matrix(M, F, dtype, 6, 8)
    check(fmpq_mod.w16_gemm(layer, X, Wp, activation=act), X, W, act, gated=True)
    check(fmpq_mod.w16_gemm(layer, X, Wp, activation=act, bias=bias, residual=residual), X, W, act, bias, residual, gated=True)
    check(fmpq_mod.w16_gemm(layer, X, Wp, activation=act, bias=bias.float(), dtype=torch.float32), X, W, act, bias, gated=True)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,gated", [(300, 515, False), (67, 128, False), (1030, 260, False), (9, 5, False), (300, 2 * 516, True), (40, 2 * 66, True)])
def test_rows_of_outputs_lie_anywhere(fmpq_mod, M, N, gated):  # noqa: F811
    """Every start of the first row and step between rows, the residual in step with them or not: the same values, and nothing around them."""
    import torch
    K, dtype = 128, torch.bfloat16    # (K in one part: the sums are the same ones)
    out_n = N // 2 if gated else N
    X, W = matrix(M, K, dtype, M), matrix(N, K, dtype, N, 0, 1.5 / K ** 0.5)
    layer = fmpq_mod.W16Layer(K, N, dtype, gated=gated)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    bias, residual = matrix(1, N, dtype, 5)[0], matrix(M, out_n, dtype, 6)
    plain = fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="silu")
    whole = fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="silu", residual=residual)
    check(whole, X, W, "silu", bias, residual, gated=gated)

    def rows_at(start, step):
        flat = torch.full((start + M * (out_n + step) + 16,), 7.0, dtype=dtype, device="cuda")
        return flat, flat[start:start + M * (out_n + step)].view(M, out_n + step)[:, :out_n]

    for start in range(8):
        for step in range(8):
            for other in (0, 1, 4):    # the residual begins as many elements further
                flat, Y = rows_at(start, step)
                _, r = rows_at((start + other) % 8, step)
                r.copy_(residual)
                fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="silu", residual=r, Y=Y)
                assert torch.equal(Y, whole), (start, step, other)
                fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="silu", residual=r, Y=r)
                assert torch.equal(r, whole), (start, step, other)
                if other == 0:
                    fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="silu", Y=Y)
                    assert torch.equal(Y, plain), (start, step)
                Y.fill_(7.0)
                assert bool((flat == 7).all()), (start, step, other)
    bias = bias.float()
    ref = fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="silu", Y=torch.empty(M, out_n + 9, device="cuda")[:, 1:out_n + 1])
    check(ref, X, W, "silu", bias, gated=gated)
    for step in range(8):    # FP32
        flat = torch.full((M, out_n + step), 7.0, device="cuda")
        assert torch.equal(fmpq_mod.w16_gemm(layer, X, Wp, bias=bias, activation="silu", Y=flat[:, :out_n]), ref), step
        assert bool((flat[:, out_n:] == 7).all()), step


# ---- groups -----------------------------------------------------------------------------------

def group_sizes(kind, E):
    import torch
    g = torch.Generator().manual_seed(E)
    if kind == "one each":
        return [1] * E
    if kind == "all in one":
        return [0] * (E - 1) + [700]
    if kind == "first alone":
        return [300] + [0] * (E - 1)
    if kind == "above 256":     # units of two parts, and a group that is cut
        return [257 + 41 * i % 210 for i in range(E - 1)] + [1100]
    if kind == "odd":
        return [(37 * i + 11) % 90 for i in range(E)]
    return (torch.rand(E, generator=g) ** 3 * 900).int().tolist()     # uneven


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["one each", "all in one", "first alone", "above 256", "odd", "uneven"])
@pytest.mark.parametrize("experts,K,N,gated", [(1, 128, 130, False), (5, 300, 520, False), (9, 256, 256, True), (33, 72, 100, True),
                                               (129, 64, 256, False), (32, 64, 128, False), (512, 72, 64, True)])
def test_groups(fmpq_mod, kind, experts, K, N, gated):  # noqa: F811
    """Every group with its own matrix; rows before, between and behind the groups left as they were."""
    import torch
    dtype = torch.bfloat16 if experts % 2 else torch.float16
    sizes = group_sizes(kind, experts)
    before, behind = 3, 5
    ends = torch.tensor([0] + sizes).cumsum(0) + before
    rows = int(ends[-1]) + behind
    X, out_n = matrix(rows, K, dtype, rows), N // 2 if gated else N
    W = torch.stack([matrix(N, K, dtype, e, 0, 1.5 / K ** 0.5) for e in range(experts)])
    bias = matrix(experts, N, torch.float32, 3)
    residual, weight = matrix(rows, out_n, dtype, 4), matrix(1, rows, torch.float32, 5)[0]
    layer = fmpq_mod.W16Layer(K, N, dtype, experts=experts, gated=gated)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    Y = torch.full((rows, out_n), 7.0, dtype=dtype, device="cuda")
    fmpq_mod.w16_grouped_gemm(layer, X, ends.int().cuda(), Wp, bias=bias, activation="silu", residual=residual, row_weight=weight, Y=Y)
    Z = torch.full((rows, out_n), 7.0, device="cuda")
    fmpq_mod.w16_grouped_gemm(layer, X, ends.int().cuda(), Wp, Y=Z)
    assert fmpq_mod.w16_device_status(layer) == 0
    for e in range(experts):
        at = slice(int(ends[e]), int(ends[e + 1]))
        if sizes[e]:
            check(Y[at], X[at], W[e], "silu", bias[e], residual[at], weight[at], gated)
            check(Z[at], X[at], W[e], None, gated=gated)
    for at in (slice(0, before), slice(rows - behind, rows)):
        assert bool((Y[at] == 7).all()) and bool((Z[at] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(300, 4096, 20480), (1, 8192, 28672), (2048, 2048, 12288)])
def test_rest_of_a_product_in_a_chain(fmpq_mod, M, K, N):  # noqa: F811
    """A residual that every product updates in place, and an input that the kernel before writes: products with a launch for their
    rest, one after another and captured, give what they give with a wait between them."""
    import torch
    X, W = matrix(M, K, torch.bfloat16, 1), matrix(N, K, torch.bfloat16, 2, 0, 0.3 * K ** -0.5)
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    start = matrix(M, N, torch.bfloat16, 3)

    def chain(r, x, wait=False):
        for _ in range(6):
            fmpq_mod.w16_gemm(layer, x, Wp, residual=r, Y=r)
            if wait:
                torch.cuda.synchronize()
            x.copy_(r[:, :K])           # (K <= N)
            if wait:
                torch.cuda.synchronize()
            fmpq_mod.w16_gemm(layer, x, Wp, residual=r, activation="silu", Y=r)
            if wait:
                torch.cuda.synchronize()
            x.mul_(0.5)

    want, x = start.clone(), X.clone()
    chain(want, x, True)
    for _ in range(5):
        got, x = start.clone(), X.clone()
        chain(got, x)
        assert torch.equal(got, want)
    got, x = start.clone(), X.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(got, x)
    for _ in range(5):
        got.copy_(start)
        x.copy_(X)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert bool(torch.isfinite(want).all()) and fmpq_mod.w16_device_status(layer) == 0


@pytest.mark.gpu
def test_calls_in_turn(fmpq_mod):  # noqa: F811
    """Products that split K, that copy their rows and that do both, one after another without a wait."""
    import torch
    cases = []
    for i, (M, K, N, pad) in enumerate([(257, 4096, 256, 0), (130, 200, 6000, 4), (1, 8192, 512, 0), (40, 4100, 300, 1), (300, 60, 64, 0), (33, 2048, 520, 8)]):
        X, W = matrix(M, K, torch.bfloat16, i, pad), matrix(N, K, torch.bfloat16, i + 9, 0, K ** -0.5)
        layer = fmpq_mod.W16Layer(K, N, torch.bfloat16)
        cases.append((layer, X, W, fmpq_mod.w16_pack_weights(layer, W)))
    for turn in range(3):
        order = cases[::-1] if turn % 2 else cases
        got = [fmpq_mod.w16_gemm(layer, X, Wp) for layer, X, W, Wp in order]
        for Y, (layer, X, W, Wp) in zip(got, order):
            check(Y, X, W)


@pytest.mark.gpu
def test_long_rows_of_a_large_buffer(fmpq_mod):  # noqa: F811
    """Rows whose offsets pass 32 bits, in X, Y and the residual; only the rows are read and written."""
    import torch
    rows, K, N, ld = 70, 64, 128, 1 << 26          # 70 rows 2^26 elements apart: 9.4 GB in 16 bits
    W = torch.stack([matrix(N, K, torch.bfloat16, e) for e in range(2)])
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16, experts=2)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)
    X, Y = buf[:, :K], buf[:, 256:256 + N]
    X.copy_(matrix(rows, K, torch.bfloat16, 1))
    Y.copy_(matrix(rows, N, torch.bfloat16, 2))
    residual = Y.clone()
    offsets = torch.tensor([0, 33, 70], dtype=torch.int32, device="cuda")
    fmpq_mod.w16_grouped_gemm(layer, X, offsets, Wp, residual=Y, Y=Y)
    check(Y[:33], X[:33], W[0], residual=residual[:33])
    check(Y[33:], X[33:], W[1], residual=residual[33:])


@pytest.mark.gpu
def test_group_bounds_are_cut_to_the_rows(fmpq_mod):  # noqa: F811
    """Offsets outside [0, rows], and groups that end before they start: nothing outside Y is touched."""
    import torch
    rows, K, N = 40, 64, 128
    X, W = matrix(rows, K, torch.float16, 1), torch.stack([matrix(N, K, torch.float16, e) for e in range(4)])
    layer = fmpq_mod.W16Layer(K, N, torch.float16, experts=4)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    buf = torch.full((rows + 20, N), 7.0, dtype=torch.float16, device="cuda")
    Y = buf[10:-10]
    offsets = torch.tensor([-5, 8, 4, 30, 2 ** 31 - 1], dtype=torch.int32, device="cuda")    # 0-7, none, 4-29, 30-39
    fmpq_mod.w16_grouped_gemm(layer, X, offsets, Wp, Y=Y)
    assert bool((buf[:10] == 7).all()) and bool((buf[-10:] == 7).all())
    check(Y[:8], X[:8], W[0])        # rows 4-7 are the first group's
    check(Y[8:30], X[8:30], W[2])
    check(Y[30:], X[30:], W[3])
    for bad in ([40, 0, 40, 0, 40], [0, 40, 0, 40, 0], [-1] * 5, [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [50] * 5):
        Y.fill_(7)
        fmpq_mod.w16_grouped_gemm(layer, X, torch.tensor(bad, dtype=torch.int32, device="cuda"), Wp, Y=Y)
        assert bool((buf[:10] == 7).all()) and bool((buf[-10:] == 7).all())
        group = next((e for e in range(4) if max(bad[e], 0) < min(bad[e + 1], 40)), None)
        if group is None:
            assert bool((Y == 7).all())
        else:
            check(Y, X, W[group])
    assert fmpq_mod.w16_device_status(layer) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,E,K,N,gated", [(1, 65, 6400, 512, False), (3, 7, 4096, 300, True), (9, 2, 2048, 520, False)])
def test_few_units_of_groups_split_K(fmpq_mod, rows, E, K, N, gated):  # noqa: F811
    import torch
    X, W = matrix(rows, K, torch.bfloat16, 1), torch.stack([matrix(N, K, torch.bfloat16, e, 0, K ** -0.5) for e in range(E)])
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16, experts=E, gated=gated)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    g = torch.Generator().manual_seed(rows)
    for turn in range(4):
        cuts = torch.randint(0, rows + 1, (E - 1,), generator=g).sort().values
        ends = torch.cat([torch.zeros(1), cuts, torch.full((1,), rows)]).int()
        Y = fmpq_mod.w16_grouped_gemm(layer, X, ends.cuda(), Wp, activation="silu")
        for e in range(E):
            at = slice(int(ends[e]), int(ends[e + 1]))
            if ends[e] < ends[e + 1]:
                check(Y[at], X[at], W[e], "silu", gated=gated)
    assert fmpq_mod.w16_device_status(layer) == 0


@pytest.mark.gpu
def test_nan_stays_in_its_rows_and_experts(fmpq_mod):  # noqa: F811
    import torch
    sizes, K, N = [20, 300, 1, 45], 200, 300
    ends = torch.tensor([0] + sizes).cumsum(0)
    X = matrix(366, K, torch.bfloat16, 1)
    W = torch.stack([matrix(N, K, torch.bfloat16, e) for e in range(4)])
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16, experts=4)
    clean = fmpq_mod.w16_grouped_gemm(layer, X, ends.int().cuda(), fmpq_mod.w16_pack_weights(layer, W))
    X, W = X.clone(), W.clone()
    X[5, K - 1], X[320] = float("nan"), float("inf")
    W[3, 7, 0] = float("nan")
    Y = fmpq_mod.w16_grouped_gemm(layer, X, ends.int().cuda(), fmpq_mod.w16_pack_weights(layer, W))
    bad = torch.zeros(366, N, dtype=torch.bool, device="cuda")
    bad[5], bad[320], bad[321:, 7] = True, True, True
    assert bool(Y[5].isnan().all()) and not bool(torch.isfinite(Y[320]).any()) and bool(Y[321:, 7].isnan().all())
    assert torch.equal(Y[~bad], clean[~bad])


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(1, 4096, 1024), (24, 2048, 512), (300, 512, 1000)])
def test_graph_stream_and_repeats(fmpq_mod, M, K, N):  # noqa: F811
    import torch
    X, W = matrix(M, K, torch.bfloat16, 1, 3), matrix(N, K, torch.bfloat16, 2, 0, K ** -0.5)
    layer = fmpq_mod.W16Layer(K, N, torch.bfloat16)
    Wp = fmpq_mod.w16_pack_weights(layer, W)
    ref = fmpq_mod.w16_gemm(layer, X, Wp, activation="silu")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [fmpq_mod.w16_gemm(layer, X, Wp, activation="silu") for _ in range(20)]
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(Y, ref) for Y in outs)
    sides = [torch.cuda.Stream() for _ in range(2)]     # two at once
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    got = [fmpq_mod.w16_gemm(layer, X, Wp, activation="silu", stream=sides[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(Y, ref) for Y in got)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,H,F", [(1, 4, 16, 512, 256), (50, 3, 8, 300, 136), (600, 2, 5, 256, 384)])
def test_routed_experts_in_16_bits(fmpq_mod, T, k, E, H, F):  # noqa: F811
    """Routing, plan, gated product, down product with the weights and the sum over the slots: the library's own steps."""
    import torch
    g = torch.Generator().manual_seed(T)
    X = matrix(T, H, torch.bfloat16, 1)
    up = torch.stack([matrix(2 * F, H, torch.bfloat16, 10 + e, 0, H ** -0.5) for e in range(E)])
    down = torch.stack([matrix(H, F, torch.bfloat16, 50 + e, 0, F ** -0.5) for e in range(E)])
    Lu, Ld = fmpq_mod.W16Layer(H, 2 * F, X.dtype, experts=E, gated=True), fmpq_mod.W16Layer(F, H, X.dtype, experts=E)
    Wu, Wd = fmpq_mod.w16_pack_weights(Lu, up), fmpq_mod.w16_pack_weights(Ld, down)
    ids, w = fmpq_mod.moe_route(torch.randn(T, E, generator=g).cuda(), k)
    plan = fmpq_mod.moe_plan(ids, E)
    buf = torch.full((plan.rows, F + 5), 7.0, dtype=X.dtype, device="cuda")
    hidden = fmpq_mod.w16_experts_gemm(Lu, plan, X, Wu, activation="silu", Y=buf[:, :F])
    D = fmpq_mod.w16_experts_gemm(Ld, plan, hidden, Wd, weights=w, dtype=torch.float32)
    Y = fmpq_mod.moe_combine(D, plan)
    used = torch.zeros(plan.rows, dtype=torch.bool, device="cuda")
    used[plan.row_of.flatten().long()] = True
    assert bool((buf[~used] == 7).all()) and bool((buf[:, F:] == 7).all())
    assert fmpq_mod.w16_device_status(Lu) == 0 and fmpq_mod.w16_device_status(Ld) == 0
    ref = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            x = X[t].cpu().double()
            a = up[e].cpu().double() @ x
            h = a[:F] * torch.sigmoid(a[:F]) * a[F:]
            ref[t] += float(w[t, j]) * (down[e].cpu().double() @ h)
    # the hidden vectors' rounding, half a step each and of either sign, averages over F of them; the output's comes on top
    assert Y.dtype == X.dtype
    assert float((Y.cpu().double() - ref).norm()) <= 2 * 2.0 ** -8 * float(ref.norm())
    for e in range(E):
        at = (ids == e).nonzero()
        if at.numel():
            r = plan.row_of[at[:, 0], at[:, 1]].long()
            check(hidden[r], X[at[:, 0]], up[e], "silu", gated=True)
            check(D[r], hidden[r], down[e], row_weight=w[at[:, 0], at[:, 1]])


# ---- refusals (no GPU) ------------------------------------------------------------------------

@pytest.fixture
def no_gpu(monkeypatch):
    from bit_quantized_gemm_fmpq_gb300 import fmpq
    monkeypatch.setattr(fmpq, "load_library", NoLibrary)
    monkeypatch.setattr(fmpq, "_lib", NoLibrary())
    monkeypatch.setattr(fmpq, "_on", lambda X: 0)
    monkeypatch.setattr(fmpq, "_device", lambda: 0)


def layer_of(K, N, experts=1, gated=False):
    import torch

    from bit_quantized_gemm_fmpq_gb300 import fmpq
    layer = object.__new__(fmpq.W16Layer)
    layer._lib, layer._h, layer._code, layer.dtype = NoLibrary(), None, 0, torch.float16
    layer.K, layer.N, layer.experts, layer.gated, layer.outputs = K, N, experts, gated, N // 2 if gated else N
    pairs = -(-(N // 2) // 128) if gated else -(-N // 256)
    layer._w_bytes = experts * pairs * 2 * -(-K // 64) * 16384
    return layer


def test_the_binding_refuses(no_gpu):
    import torch

    from bit_quantized_gemm_fmpq_gb300 import fmpq
    one, three = layer_of(128, 256), layer_of(128, 256, 3)
    W1 = on_gpu(torch.zeros(one._w_bytes, dtype=torch.uint8))
    W3 = on_gpu(torch.zeros(three._w_bytes, dtype=torch.uint8))
    X, Y = half(6, 128), half(6, 256)
    off = on_gpu(torch.zeros(4, dtype=torch.int32))
    ints = lambda n: on_gpu(torch.zeros(n, dtype=torch.int32))      # noqa: E731
    calls = [
        lambda: fmpq.w16_pack_weights(one, half(256, 127)), lambda: fmpq.w16_pack_weights(one, f32(256, 128)),
        lambda: fmpq.w16_pack_weights(three, half(2, 256, 128)), lambda: fmpq.w16_pack_weights(one, torch.zeros(256, 128).half()),
        lambda: fmpq.w16_pack_weights(one, half(1, 128).expand(256, 128)), lambda: fmpq.w16_pack_weights(one, elsewhere(half(256, 128))),
        lambda: fmpq.w16_gemm(three, X, W3), lambda: fmpq.w16_gemm(one, half(6, 127), W1), lambda: fmpq.w16_gemm(one, f32(6, 128), W1),
        lambda: fmpq.w16_gemm(one, on_gpu(torch.zeros(6, 128, dtype=torch.bfloat16)), W1), lambda: fmpq.w16_gemm(one, overlapping(6, 128)[0], W1),
        lambda: fmpq.w16_gemm(one, X, W1[16:]), lambda: fmpq.w16_gemm(one, X, elsewhere(W1)), lambda: fmpq.w16_gemm(one, elsewhere(X), W1),
        lambda: fmpq.w16_gemm(one, X, W1, dtype=torch.bfloat16), lambda: fmpq.w16_gemm(one, X, W1, Y=half(6, 255)),
        lambda: fmpq.w16_gemm(one, X, W1, Y=overlapping(6, 256)[2]), lambda: fmpq.w16_gemm(one, X, W1, Y=elsewhere(Y)),
        lambda: fmpq.w16_gemm(one, X, W1, bias=half(255)), lambda: fmpq.w16_gemm(one, X, W1, bias=half(3, 256)),
        lambda: fmpq.w16_gemm(one, X, W1, residual=f32(6, 256)), lambda: fmpq.w16_gemm(one, X, W1, residual=half(6, 256), dtype=torch.float32),
        lambda: fmpq.w16_gemm(one, X, W1, activation="swish"), lambda: fmpq.w16_gemm(one, Y[:, :128], W1, Y=Y),
        lambda: fmpq.w16_grouped_gemm(three, X, ints(3), W3), lambda: fmpq.w16_grouped_gemm(three, X, ints(4).long(), W3),
        lambda: fmpq.w16_grouped_gemm(three, X, torch.zeros(4, dtype=torch.int32), W3), lambda: fmpq.w16_grouped_gemm(three, X, ints(8)[::2], W3),
        lambda: fmpq.w16_grouped_gemm(three, X, off, W3, bias=half(256)), lambda: fmpq.w16_grouped_gemm(three, X, off, W3, row_weight=f32(5)),
        lambda: fmpq.w16_grouped_gemm(three, X, off, W3, row_weight=half(6)), lambda: fmpq.w16_grouped_gemm(three, X, elsewhere(off), W3),
        lambda: fmpq.w16_experts_gemm(three, plan_of(5, 1, 3, 40), X, W3), lambda: fmpq.w16_experts_gemm(three, plan_of(6, 1, 4, 40), X, W3),
        lambda: fmpq.w16_experts_gemm(three, plan_of(6, 1, 3, 40), X, W3, weights=f32(6, 2)),
        lambda: fmpq.w16_experts_gemm(three, plan_of(6, 1, 3, 40), X, W3, weights=half(6, 1)),
        lambda: fmpq.w16_experts_gemm(three, plan_of(6, 1, 3, 40), X, W3, Y=half(6, 256)),
        lambda: fmpq.w16_experts_gemm(three, plan_of(6, 1, 3, 40), X, W3, residual=half(6, 256)),
        lambda: fmpq.w16_experts_gemm(three, plan_of(6, 1, 3, 40), half(40, 127), W3),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")


@pytest.mark.parametrize("K,N,experts,gated,dtype,code", [(0, 128, 1, 0, 0, 2), (128, 0, 1, 0, 0, 2), (65537, 8, 1, 0, 0, 2), (8, 8, 0, 0, 0, 2),
                                                          (8, 8, 513, 0, 0, 2), (8, 9, 1, 1, 0, 2), (8, 8, 1, 2, 0, 1), (8, 8, 1, 0, 2, 1)])
def test_layer_sizes_refused(K, N, experts, gated, dtype, code):
    import ctypes

    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    lib, out, z = fmpq.load_library(), ctypes.c_void_p(), None
    assert lib.w16_layer_create(K, N, experts, gated, dtype, ctypes.byref(out)) == code and not out.value
    assert lib.w16_layer_create(8, 8, 1, 0, 0, None) == 1
    assert lib.w16_gemm(z, z, 8, 1, z, z, z, 0, 8, z, 0, z) == 1
    assert lib.w16_grouped_gemm(z, z, 8, 1, z, z, z, z, z, 0, 8, z, 0, z) == 1
    assert lib.w16_experts_gemm(z, z, 1, 1, z, 8, 0, z, z, z, z, 0, 8, z, 0, z) == 1
    assert lib.w16_experts_workspace_bytes(z, z, 8, 1, 1, 1) == 0
    assert lib.w16_pack_weights(z, 0, z, 8, 1, z, z) == 1 and lib.w16_device_status(z, None, 0) == 1
    assert lib.w16_packed_w_bytes(z) == 0 and lib.w16_workspace_bytes(z, z, 7, 3) == 0
    lib.w16_layer_destroy(z)


@pytest.mark.gpu
def test_the_library_refuses(fmpq_mod):  # noqa: F811
    import torch
    layer = fmpq_mod.W16Layer(60, 64, torch.float16)
    X, Wp = matrix(4, 60, torch.float16, 1), fmpq_mod.w16_pack_weights(layer, matrix(64, 60, torch.float16, 2))
    Y = torch.full((4, 64), 7.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(4 * 64 * 2, dtype=torch.uint8, device="cuda").data_ptr()

    def call(ldx=60, M=4, dtype=0, ldy=64, workspace=ws, nbytes=512, y=Y.data_ptr(), x=X.data_ptr()):
        return fmpq_mod._lib.w16_gemm(layer.handle, x, ldx, M, Wp.data_ptr(), None, y, dtype, ldy, workspace, nbytes, None)

    assert fmpq_mod._lib.w16_workspace_bytes(layer.handle, X.data_ptr(), 60, 4) == 512
    for code, kw in [(1, dict(dtype=1)), (1, dict(y=None)), (2, dict(M=0)), (2, dict(M=(1 << 24) + 1)), (2, dict(ldx=59)), (2, dict(ldy=63)),
                     (3, dict(x=X.data_ptr() + 1)), (7, dict(workspace=None)), (7, dict(nbytes=511)), (3, dict(workspace=ws + 8))]:
        assert call(**kw) == code, kw
    torch.cuda.synchronize()
    assert bool((Y == 7).all())
