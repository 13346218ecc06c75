"""Routing to experts and the experts' products against 64-bit forms of their definitions.

Tolerances. Expert ids and the plan are exact. Routing weights: an exponential (2 steps), a sum over at
most 512, a quotient or two and the scale: 16 half steps of 2^-24, and the exponential's argument,
rounded once, up to |logit| half steps more: (16 + 2 max|logit|) 2^-24 of the weight. The hidden vectors: half an E4M3 step (2^-4 of
the value, or half the smallest code, 2^-10 of the scale), the scale's own rounding, and the FP32
sums: (K + 2 nb + 8) 2^-23 of the absolute products for each factor of silu(g) u. The down product as a
linear layer's, its weight one rounding more. The whole: two 16-bit roundings (eps), and codes that
flip because g and u are sums in FP32: within 2^-16 of a value, a flip of at most 2^-3 of it happens
for at most a 2^-11 part, 2^-3 2^-5.5 = 2.8e-3 of the norm at the very worst.
"""
import numpy as np
import pytest

from tests.test_fp8_linear import BLOCK, check_product, decode_activations, expand, values, weight_blocks


# ---- routing in 64 bits -----------------------------------------------------------------------

def route_ref(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    x = logits.astype(np.float64)
    T, E = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        on = x[t] > -np.inf
        if not on.any():
            continue
        if score == "softmax":
            top = x[t].max()
            e = (x[t] == top).astype(float) if np.isinf(top) else np.exp(x[t] - top)
            sc = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                sc = 1.0 / (1.0 + np.exp(-x[t]))
        if bias is None and (groups == 1 or group_top == 1):
            key = x[t].copy()
        else:
            key = sc + (0.0 if bias is None else bias.astype(np.float64))
            key[~on | np.isnan(key)] = -np.inf
        if groups > 1:
            runs = key.reshape(groups, -1)
            val = np.full(groups, -np.inf)
            for g in range(groups):
                best = np.sort(runs[g])[::-1][:group_top]
                if best[0] > -np.inf:
                    val[g] = best[best > -np.inf].sum()
            keep = np.argsort(-val, kind="stable")[:top_groups]
            mask = np.ones(groups, bool)
            mask[keep] = False
            runs[mask] = -np.inf
        order = np.argsort(-key, kind="stable")[:k]
        for j, e_ in enumerate(order):
            if key[e_] > -np.inf:
                ids[t, j], w[t, j] = e_, sc[e_]
        if renormalize and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale


def check_route(fmpq, logits, k, **kw):
    import torch
    bias = kw.get("bias")
    ids, w = fmpq.moe_route(logits, k, **kw)
    ref_kw = dict(kw, bias=None if bias is None else bias.cpu().numpy())
    ri, rw = route_ref(logits.float().cpu().numpy(), k, **ref_kw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    x = logits.float()
    reach = float(x[torch.isfinite(x)].abs().max()) if bool(torch.isfinite(x).any()) else 0.0
    tol = (16 + 2 * reach) * 2.0 ** -24
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - rw) <= tol * np.abs(rw) + 1e-37)


# ---- refusals (no GPU) ------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    return fmpq.load_library()


def test_route_refusals(lib):
    p = 4096   # never read: the arguments are refused first

    def call(logits=p, dtype=0, ldl=64, T=4, E=64, k=4, score=0, bias=None, groups=1, top=1, gtop=1, renorm=1, scale=1.0,
             ids=p, weights=p):
        return lib.moe_route(logits, dtype, ldl, T, E, k, score, bias, groups, top, gtop, renorm, scale, ids, weights, None)

    for kw in (dict(logits=None), dict(ids=None), dict(weights=None), dict(dtype=3), dict(score=2), dict(gtop=3),
               dict(renorm=2), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**kw) == 1, kw
    for kw in (dict(T=0), dict(E=0), dict(E=513, ldl=513), dict(k=0), dict(k=33), dict(E=3, k=4), dict(ldl=63), dict(groups=0),
               dict(groups=5), dict(groups=64), dict(groups=8, top=9), dict(groups=16, top=0), dict(groups=32, top=1)):
        assert call(**kw) == 2, kw
    assert call(logits=p + 1) == 3 and call(ids=p + 2) == 3 and call(bias=p + 2) == 3


def test_plan_refusals(lib):
    p = 4096
    assert lib.moe_plan(None, 4, 2, 8, p, None) == 1
    assert lib.moe_plan(p, 0, 2, 8, p, None) == 2
    assert lib.moe_plan(p, 4, 33, 8, p, None) == 2
    assert lib.moe_plan(p, 4, 2, 1025, p, None) == 2
    assert lib.moe_plan(p, 1 << 22, 2, 8, p, None) == 2
    assert lib.moe_plan(p, 4, 2, 8, p + 4, None) == 3
    assert lib.moe_rows(0, 2, 8) == 0 and lib.moe_plan_bytes(4, 0, 8) == 0
    assert lib.moe_rows(4, 2, 8) == 64 and lib.moe_rows(1, 1, 1) == 8 and lib.moe_rows(100, 2, 3) == 224
    assert lib.moe_combine(p, 0, 8, p, 4, 2, 8, 9, p, 9, None) == 2
    assert lib.moe_combine(p, 2, 8, p, 4, 2, 8, 8, p, 8, None) == 1
    assert lib.moe_quantize(None, p, 4, 2, p, 0, 8, p, p, None) == 1
    assert lib.moe_up(None, p, 4, 2, p, p, p, p, p, p, None) == 1
    assert lib.moe_down(None, p, 4, 2, p, p, p, p, p, p, 0, 8, None) == 1


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


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (9, 32, 32), (33, 60, 4), (100, 64, 6), (70, 128, 8), (50, 256, 8),
                                   (20, 500, 10), (7, 512, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route(fmpq_mod, T, E, k, score, biased):
    import torch
    g = torch.Generator().manual_seed(T * 1000 + E + biased)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        logits = (torch.randn(T, E, generator=g) * 2).to(dtype).cuda()
        bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
        check_route(fmpq_mod, logits, k, score=score, bias=bias, renormalize=bool(T % 2), scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,top_groups,k", [(64, 8, 3, 6), (256, 8, 4, 8), (60, 5, 2, 4), (32, 32, 8, 8), (12, 4, 1, 3),
                                                   (512, 16, 2, 20), (128, 4, 4, 8), (24, 2, 1, 12), (96, 3, 2, 9)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(fmpq_mod, E, groups, top_groups, k, group_top, biased):
    import torch
    g = torch.Generator().manual_seed(E + groups)
    for dtype, score in ((torch.float32, "sigmoid"), (torch.bfloat16, "softmax")):
        x = torch.randn(40, E, generator=g)
        x[torch.rand(40, E, generator=g) < 0.2] = float("-inf")
        x[3, :E // groups] = float("-inf")        # a group with nothing left
        x[5] = float("-inf")
        bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
        check_route(fmpq_mod, x.to(dtype).cuda(), k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                    group_top=group_top)


@pytest.mark.gpu
def test_route_masks_and_ties(fmpq_mod):
    import torch
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(9, 40)
    x[0] = -inf                          # nothing left
    x[1] = nan
    x[2, 1:] = -inf                      # one expert for 4 slots
    x[3, ::2] = nan
    x[4] = torch.arange(40) % 3          # ties: the lowest index
    x[5, 7], x[5, 30] = inf, inf         # two experts share a softmax
    x[6] = -200.0
    x[6, 3] = 200.0
    x[7] = torch.finfo(torch.float32).min
    x[8] = torch.where(torch.arange(40) % 2 == 0, 0.0, -0.0)     # the zeros are equal
    bias = torch.zeros(40)
    bias[2], bias[9], bias[11] = -inf, nan, 1e30
    for renorm in (False, True):
        check_route(fmpq_mod, x.cuda(), 4, renormalize=renorm)
        check_route(fmpq_mod, x.cuda(), 4, bias=bias.cuda(), renormalize=renorm)
        check_route(fmpq_mod, x.cuda(), 4, bias=torch.zeros(40).cuda(), renormalize=renorm)
        check_route(fmpq_mod, x.cuda(), 4, score="sigmoid", renormalize=renorm, groups=8, top_groups=2)
        check_route(fmpq_mod, x.cuda(), 4, score="sigmoid", bias=bias.cuda(), renormalize=renorm, groups=8, top_groups=2,
                    group_top=2)


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups", [(64, 1), (256, 1), (256, 8)])
def test_route_keys_closer_than_fp32(fmpq_mod, E, groups):
    """Biases that cancel the scores: keys differ by a few 1e-8, which only 64 bits order."""
    import torch
    g = torch.Generator().manual_seed(E)
    row = torch.randn(E, generator=g)
    bias = (0.75 - torch.sigmoid(row.double())).float()
    x = row.repeat(6, 1)
    x[3:] += torch.randn(3, E, generator=g) * 1e-6
    check_route(fmpq_mod, x.cuda(), 8, score="sigmoid", bias=bias.cuda(), groups=groups, top_groups=max(1, groups // 2),
                group_top=2)


@pytest.mark.gpu
def test_route_strided_rows(fmpq_mod):
    import torch
    big = torch.randn(30, 71, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    check_route(fmpq_mod, big[:, 3:63], 4)
    check_route(fmpq_mod, big[::3, :64], 4)
    check_route(fmpq_mod, big[4:5, 1:], 8)


def plan_ref(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    start, count, row = np.zeros(E, int), np.zeros(E, int), np.full(T * k, -1)
    at = 0
    for e in range(E):
        mine = np.nonzero(flat == e)[0]
        start[e], count[e] = at, len(mine)
        row[mine] = at + np.arange(len(mine))
        at += (len(mine) + 7) // 8 * 8
    return start, count, row.reshape(T, k), at


def draw_ids(T, k, E, seed, skew=0.0, dropped=0.1):
    rng = np.random.default_rng(seed)
    p = np.exp(skew * rng.random(E) * 4)
    ids = np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < dropped] = -1
    return ids


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (5, 2, 7), (128, 8, 64), (129, 8, 64), (700, 6, 1024), (3000, 4, 33)])
def test_plan(fmpq_mod, T, k, E):
    import torch
    ids = draw_ids(T, k, E, T + E)
    if T > 4:
        ids[2, 0] = E          # outside: no expert
        ids[3] = ids[3, 0]     # one expert in every slot
        ids[4] = -1
    plan = fmpq_mod.moe_plan(torch.from_numpy(ids).cuda(), E)
    start, count, row, used = plan_ref(ids, E)
    assert np.array_equal(plan.start.cpu().numpy(), start)
    assert np.array_equal(plan.count.cpu().numpy(), count)
    assert np.array_equal(plan.row_of.cpu().numpy(), row)
    assert used <= plan.rows
    pair_of = plan.buffer.cpu().numpy()[2 * E + T * k:2 * E + T * k + plan.rows]
    there = row.reshape(-1) >= 0
    assert np.array_equal(pair_of[row.reshape(-1)[there]], np.nonzero(there)[0])


def experts_case(T, k, E, H, F, N, dtype, seed, skew=0.0, dropped=0.1):
    import torch
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, H, generator=g).to(dtype)
    up = (torch.randn(E, 2 * F, H, generator=g) / H ** 0.5).to(dtype)
    down = (torch.randn(E, N, F, generator=g) / F ** 0.5).to(dtype)
    ids = torch.from_numpy(draw_ids(T, k, E, seed, skew, dropped))
    w = torch.rand(T, k, generator=g) + 0.1
    return X, up, down, ids, w


CASES = [
    (1, 1, 1, 128, 128, 128, 0.0, 0.0), (1, 4, 8, 256, 128, 130, 0.0, 0.0), (5, 2, 3, 1, 1, 1, 0.0, 0.2),
    (40, 2, 6, 300, 140, 260, 1.0, 0.1), (17, 1, 2, 512, 256, 384, 0.0, 0.0), (200, 3, 4, 129, 127, 256, 1.0, 0.1),
    (700, 2, 3, 256, 200, 264, 1.0, 0.0), (600, 1, 1, 128, 130, 72, 0.0, 0.0), (30, 2, 4, 256, 128, 128, 0.0, 1.0),
    (130, 8, 32, 384, 384, 512, 0.5, 0.0),
    # more tiles than pairs of CTAs: several a pair, for many tokens an expert and for few
    (700, 2, 3, 256, 2560, 5200, 0.0, 0.0), (64, 4, 16, 256, 1280, 2600, 0.5, 0.1),
    (160, 2, 4, 256, 200, 264, 0.0, 0.0), (150, 4, 7, 200, 1300, 2500, 0.3, 0.1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,H,F,N,skew,dropped", CASES)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_experts_step_by_step(fmpq_mod, T, k, E, H, F, N, skew, dropped, dtype):
    import torch
    dtype = getattr(torch, dtype)
    X, up, down, ids, w = experts_case(T, k, E, H, F, N, dtype, T + E + F, skew, dropped)
    Lu, Ld = fmpq_mod.Fp8Layer(H, 2 * F, experts=E, gated=True), fmpq_mod.Fp8Layer(F, N, experts=E)
    Wu, su = fmpq_mod.fp8_pack_weights(Lu, up.cuda())
    Wd, sd = fmpq_mod.fp8_pack_weights(Ld, down.cuda())
    plan = fmpq_mod.moe_plan(ids.cuda(), E)
    A, sa = fmpq_mod.moe_quantize(Lu, plan, X.cuda())
    Hq, sh = fmpq_mod.moe_up(Lu, plan, A, sa, Wu, su)
    D = fmpq_mod.moe_down(Ld, plan, Hq, sh, Wd, sd, weights=w.cuda(), dtype=dtype)
    Y = fmpq_mod.moe_combine(D, plan)
    assert fmpq_mod.fp8_device_status(Lu) == 0 and fmpq_mod.fp8_device_status(Ld) == 0

    x64 = values(X)
    a64 = decode_activations(A, plan.rows, H)[:, :H] * sa.cpu().double()[:, :plan.rows].t().repeat_interleave(BLOCK, 1)[:, :H]
    h_codes = decode_activations(Hq, plan.rows, F)
    h_scale = sh.cpu().double()[:, :plan.rows].t()
    h64 = (h_codes * h_scale.repeat_interleave(BLOCK, 1))[:, :F]
    row_of = plan.row_of.cpu().long()
    nb = -(-H // BLOCK)
    total = torch.zeros(T, N, dtype=torch.float64)
    whole = torch.zeros(T, N, dtype=torch.float64)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        rows = row_of[t, j]
        assert torch.equal(a64[rows], x64[t])
        wg, wu = (expand(*weight_blocks(up[e, i * F:(i + 1) * F])) for i in (0, 1))
        wd = expand(*weight_blocks(down[e]))
        g, u = x64[t] @ wg.t(), x64[t] @ wu.t()
        slack = (H + 2 * nb + 8) * 2.0 ** -23
        dg, du = slack * (x64[t].abs() @ wg.abs().t()), slack * (x64[t].abs() @ wu.abs().t())
        h = g * torch.sigmoid(g) * u
        # |silu'| <= 1.1, |silu(g)| <= |g|
        fp32 = 1.1 * dg * (u.abs() + du) + g.abs() * du + 2.0 ** -20 * h.abs()
        bound = h.abs() * 2.0 ** -4 * (1 + 2.0 ** -20) + 2.0 ** -10 * h_scale[rows].repeat_interleave(BLOCK, 1)[:, :F] + 1.1 * fp32 + 1e-300
        assert bool(((h64[rows] - h).abs() <= bound).all())
        for b in range(h_scale.shape[1]):
            cols = slice(b * BLOCK, min((b + 1) * BLOCK, F))
            top = h[:, cols].abs().amax(1) / 448
            near = (h_scale[rows, b] - top).abs() <= 2.0 ** -22 * top + fp32[:, cols].amax(1) / 448 + 1e-44
            assert bool(near.all())
        assert bool((h_codes[rows][:, F:] == 0).all())
        check_product(D[rows.cuda()], h64[rows] * w[t, j].double()[:, None], wd)
        total.index_add_(0, t, D.cpu().double()[rows])
        whole.index_add_(0, t, (values(h) @ wd.t()) * w[t, j].double()[:, None])
    eps = torch.finfo(dtype).eps
    got = Y.cpu().double()
    assert bool(((got - total).abs() <= total.abs() * eps / 2 + 8 * k * 2.0 ** -24 * total.abs().max() + 1e-7).all())
    assert float((got - whole).norm()) <= (eps + 2.8e-3) * float(whole.norm())
    again = fmpq_mod.moe_experts(Lu, Ld, X.cuda(), ids.cuda(), w.cuda(), Wu, su, Wd, sd)
    assert torch.equal(again, Y)


@pytest.mark.gpu
@pytest.mark.parametrize("turn", [0, 5])
def test_experts_tiles_and_small_rests(fmpq_mod, turn):
    """Tiles of 256 rows and every kind of rest, for many experts, the last of them with and without any."""
    import torch
    E, H, F, N = 512, 1024, 512, 2048
    shares = [0, 1, 40, 64, 65, 130, 255, 256, 257, 300, 320, 321, 513, 600]
    share = [shares[(e + turn) % len(shares)] for e in range(E)]
    g = torch.Generator(device="cuda").manual_seed(turn)
    ids = torch.repeat_interleave(torch.arange(E), torch.tensor(share))
    T = ids.numel()
    ids = ids[torch.randperm(T, generator=torch.Generator().manual_seed(turn))].int().cuda()[:, None]
    X = torch.randn(T, H, device="cuda", generator=g).half()
    w = torch.rand(T, 1, device="cuda", generator=g) + 0.1

    def weights(layer, rows, cols):
        codes = torch.randn(E, rows, cols, device="cuda", generator=g).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        scales = (torch.rand(E, rows // BLOCK, cols // BLOCK, device="cuda", generator=g) + 0.5) / (100 * cols ** 0.5)
        return codes, scales, fmpq_mod.fp8_pack_codes(layer, codes, scales)
    Lu, Ld = fmpq_mod.Fp8Layer(H, 2 * F, experts=E, gated=True), fmpq_mod.Fp8Layer(F, N, experts=E)
    cu, su, Wu = weights(Lu, 2 * F, H)
    cd, sd, Wd = weights(Ld, N, F)
    plan = fmpq_mod.moe_plan(ids, E)
    A, sa = fmpq_mod.moe_quantize(Lu, plan, X)
    Hq, sh = fmpq_mod.moe_up(Lu, plan, A, sa, *Wu)
    D = fmpq_mod.moe_down(Ld, plan, Hq, sh, *Wd, weights=w, dtype=torch.float16)
    Y = fmpq_mod.moe_combine(D, plan)
    assert fmpq_mod.fp8_device_status(Lu) == 0 and fmpq_mod.fp8_device_status(Ld) == 0
    again = fmpq_mod.moe_experts(Lu, Ld, X, ids, w, *Wu, *Wd)
    assert torch.equal(Y, again)

    def decoded(codes, scales, channels):
        v = decode_activations(codes, plan.rows, channels).cuda()
        return v, scales.double()[:, :plan.rows].t().repeat_interleave(BLOCK, 1)

    def matrix(codes, scales):
        return codes.double() * scales.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
    (a, a_scale), (h_codes, h_scale) = decoded(A, sa, H), decoded(Hq, sh, F)
    row_of = plan.row_of.long()[:, 0]
    assert torch.equal(Y.cpu(), (D[row_of].float() + 0.0).half().cpu())   # one expert a token
    slack, eps = (H + 2 * (H // BLOCK) + 8) * 2.0 ** -23, torch.finfo(torch.float16).eps / 2
    for e in range(E):
        t = (ids[:, 0] == e).nonzero()[:, 0]
        assert t.numel() == share[e]
        r = row_of[t]
        x = a[r] * a_scale[r]
        wg, wu = matrix(cu[e], su[e]).split(F)
        u, gate = x @ wu.t(), x @ wg.t()
        dg, du = slack * (x.abs() @ wg.abs().t()), slack * (x.abs() @ wu.abs().t())
        h = gate * torch.sigmoid(gate) * u
        fp32 = 1.1 * dg * (u.abs() + du) + gate.abs() * du + 2.0 ** -20 * h.abs()
        hq = h_codes[r] * h_scale[r]
        bound = h.abs() * 2.0 ** -4 * (1 + 2.0 ** -20) + 2.0 ** -10 * h_scale[r] + 1.1 * fp32 + 1e-300
        assert bool(((hq - h).abs() <= bound).all()), (e, share[e])
        x, wd = hq * w[t].double(), matrix(cd[e], sd[e])
        ref, size = x @ wd.t(), x.abs() @ wd.abs().t()
        bound = ref.abs() * eps + 2.0 ** -25 + (F + 2 * (F // BLOCK) + 2) * 2.0 ** -23 * size
        assert bool(((D[r].double() - ref).abs() <= bound).all()), (e, share[e])


@pytest.mark.gpu
def test_experts_in_a_graph_and_on_a_stream(fmpq_mod):
    import torch
    X, up, down, ids, w = experts_case(50, 2, 6, 256, 256, 256, torch.bfloat16, 3)
    Lu, Ld = fmpq_mod.Fp8Layer(256, 512, experts=6, gated=True), fmpq_mod.Fp8Layer(256, 256, experts=6)
    Wu, su = fmpq_mod.fp8_pack_weights(Lu, up.cuda())
    Wd, sd = fmpq_mod.fp8_pack_weights(Ld, down.cuda())
    x, logits = X.cuda(), torch.randn(50, 6, generator=torch.Generator().manual_seed(9)).cuda()

    def step():
        i, p = fmpq_mod.moe_route(logits, 2)
        return fmpq_mod.moe_experts(Lu, Ld, x, i, p, Wu, su, Wd, sd)

    want = step()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        assert torch.equal(step(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    logits.copy_(torch.randn(50, 6, generator=torch.Generator().manual_seed(10)))
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    assert torch.equal(replayed, step())      # the replay routes the new logits
    assert not torch.equal(replayed, want)


@pytest.mark.gpu
def test_experts_binding_refusals(fmpq_mod):
    import torch
    Lu, Ld = fmpq_mod.Fp8Layer(128, 256, experts=2, gated=True), fmpq_mod.Fp8Layer(128, 128, experts=2)
    Wu, su = fmpq_mod.fp8_pack_weights(Lu, torch.zeros(2, 256, 128, dtype=torch.float16, device="cuda"))
    Wd, sd = fmpq_mod.fp8_pack_weights(Ld, torch.zeros(2, 128, 128, dtype=torch.float16, device="cuda"))
    X = torch.zeros(3, 128, dtype=torch.float16, device="cuda")
    ids = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(3, 1, device="cuda")
    ok = (Lu, Ld, X, ids, w, Wu, su, Wd, sd)
    fmpq_mod.moe_experts(*ok)
    for at, bad in ((0, Ld), (2, X[:2]), (2, X.float()), (3, ids.long()), (4, w.half()), (4, w[:2])):
        args = list(ok)
        args[at] = bad
        with pytest.raises((ValueError, fmpq_mod.FmpqError)):
            fmpq_mod.moe_experts(*args)
    with pytest.raises(ValueError):
        fmpq_mod.moe_route(X[0], 1)
    with pytest.raises(fmpq_mod.FmpqError):
        fmpq_mod.moe_route(X, 200)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 40, 700])
def test_example_step(fmpq_mod, tokens):
    """The example's captured step: two bf16 roundings and flipped codes (see the head of this file)."""
    from examples import routed_experts
    assert routed_experts.main(tokens) <= 2.0 ** -7 + 2.8e-3
