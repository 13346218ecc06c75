"""The routed experts' outputs are summed in FP32 and rounded once; SwiGLU is good to a few FP32 roundings.

Tolerances. Y against the 64-bit sum over a token's slots of w down(h), h the values of the hidden codes: half a
step of the type (finfo.eps / 2 of the value, or half the smallest fp16 number), and (F + 2 nb + k + 2) steps of 2^-23
of the absolute products for the FP32 sums, each addition and scaling one step at worst. The hidden scale where gate
and up are exact: the exponential 2 steps of 2^-23, the sum in the denominator, the quotient, the product and the
division by 448 half a step each: 4 steps of 2^-23.
"""
import pytest

from tests.test_fp8_linear import BLOCK, decode_activations, expand, weight_blocks
from tests.test_moe import draw_ids, fmpq_mod  # noqa: F401  (the fixture)


def run_steps(fmpq, X, up, down, ids, w):
    """moe_experts' output, and the hidden values of every row in 64 bits with the rows of the pairs."""
    E, F = down.shape[0], down.shape[2]
    Lu, Ld = fmpq.Fp8Layer(X.shape[1], 2 * F, experts=E, gated=True), fmpq.Fp8Layer(F, down.shape[1], experts=E)
    Wu, Wd = fmpq.fp8_pack_weights(Lu, up.cuda()), fmpq.fp8_pack_weights(Ld, down.cuda())
    plan = fmpq.moe_plan(ids.cuda(), E)
    Hq, sh = fmpq.moe_up(Lu, plan, *fmpq.moe_quantize(Lu, plan, X.cuda()), *Wu)
    h = decode_activations(Hq, plan.rows, F) * sh.cpu().double()[:, :plan.rows].t().repeat_interleave(BLOCK, 1)
    Y = fmpq.moe_experts(Lu, Ld, X.cuda(), ids.cuda(), w.cuda(), *Wu, *Wd)
    assert fmpq.fp8_device_status(Lu) == 0 and fmpq.fp8_device_status(Ld) == 0
    return Y.cpu(), h[:, :F], plan.row_of.cpu().long()


def check_sum(Y, h, row_of, down, ids, w):
    import torch
    T, k = ids.shape
    N, F = down.shape[1:]
    ref, size = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    for e in range(down.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            hw, wd = h[row_of[t, j]] * w[t, j].double()[:, None], expand(*weight_blocks(down[e]))
            ref.index_add_(0, t, hw @ wd.t())
            size.index_add_(0, t, hw.abs() @ wd.abs().t())
    info = torch.finfo(Y.dtype)
    bound = ref.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2 + (F + 2 * -(-F // BLOCK) + k + 2) * 2.0 ** -23 * size
    assert bool(torch.isfinite(Y).all())
    err = (Y.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,H,F,N", [(1, 8, 16, 256, 128, 260), (37, 5, 9, 200, 140, 136), (700, 4, 6, 128, 256, 520),
                                         (90, 3, 4, 130, 129, 131), (600, 2, 3, 256, 2560, 5201)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_experts_outputs_are_rounded_once(fmpq_mod, T, k, E, H, F, N, dtype):  # noqa: F811
    import torch
    dtype = getattr(torch, dtype)
    g = torch.Generator().manual_seed(T + F)
    X = torch.randn(T, H, generator=g).to(dtype)
    up = (torch.randn(E, 2 * F, H, generator=g) / H ** 0.5).to(dtype)
    down = (torch.randn(E, N, F, generator=g) / F ** 0.5).to(dtype)
    ids = torch.from_numpy(draw_ids(T, k, E, T + E))
    w = torch.rand(T, k, generator=g) + 0.1
    Y, h, row_of = run_steps(fmpq_mod, X, up, down, ids, w)
    check_sum(Y, h, row_of, down, ids, w)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 600])
def test_slots_past_the_types_range_may_cancel(fmpq_mod, T):  # noqa: F811
    """Two experts of opposite signs: each slot's product is past fp16's 65504, the token's sum is not."""
    import torch
    g = torch.Generator().manual_seed(T)
    H, F, N = 128, 128, 256
    X = (torch.rand(T, H, generator=g) + 1).half()
    up = (torch.rand(1, 2 * F, H, generator=g) * 0.5).half().repeat(2, 1, 1)
    down = (torch.rand(1, N, F, generator=g) + 0.5).half()
    down = torch.cat([down, -down])
    ids = torch.tensor([0, 1], dtype=torch.int32).repeat(T, 1)
    w = torch.tensor([1.0, 1.0 - 2.0 ** -6]).repeat(T, 1)
    Y, h, row_of = run_steps(fmpq_mod, X, up, down, ids, w)
    assert float((h[row_of[:, 0]] @ down[0].double().t()).min()) > 65504     # a slot alone
    check_sum(Y, h, row_of, down, ids, w)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [128, 6000])   # tiles of 64 and of 256 tokens
@pytest.mark.parametrize("sign", [1, -1])
def test_swiglu_scale(fmpq_mod, T, sign):  # noqa: F811
    """Tokens with one channel and weights in one row make gate and up exact: the hidden scale is
    fl32(|silu(g) u| / 448) to 4 steps of 2^-23, for gates up to 49 in size."""
    import torch
    channel = torch.arange(T) % 128
    X = torch.zeros(T, 128)
    X[torch.arange(T), channel] = 448.0
    up = torch.zeros(1, 256, 128)
    codes = torch.arange(128, dtype=torch.uint8).clamp(max=126).view(torch.float8_e4m3fn).float()
    gates = sign * codes.flip(0) * 2.0 ** -12      # a block of E4M3 codes with the scale 2^-12
    up[0, 0] = gates
    up[0, 128] = 448 * 2.0 ** -12
    layer = fmpq_mod.Fp8Layer(128, 256, gated=True)
    W = fmpq_mod.fp8_pack_weights(layer, up.half().cuda())
    plan = fmpq_mod.moe_plan(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1)
    _, scales = fmpq_mod.moe_up(layer, plan, *fmpq_mod.moe_quantize(layer, plan, X.bfloat16().cuda()), *W)
    gate, lin = (448.0 * gates).double()[channel], 49.0
    ref = (gate * torch.sigmoid(gate) * lin).abs() / 448
    got = scales[0].cpu().double()[plan.row_of.cpu().long()[:, 0]]
    assert bool(((got - ref).abs() <= ref * 4 * 2.0 ** -23 + 2.0 ** -149).all()), float(((got - ref).abs() / ref.clamp_min(1e-300)).max() * 2 ** 23)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,F,N,pad", [(20, 3, 4, 128, 130, 0), (20, 2, 3, 256, 264, 1), (600, 2, 3, 2560, 5201, 3), (600, 2, 3, 2560, 5200, 0)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_steps_with_rows_of_16_or_32_bits(fmpq_mod, T, k, E, F, N, pad, dtype):  # noqa: F811
    """D is FP32 unless a 16-bit one is passed: that one holds the FP32 rows rounded, and Y is the sum of either, rounded."""
    import torch
    dtype = getattr(torch, dtype)
    g = torch.Generator().manual_seed(T + N)
    X = torch.randn(T, 128, generator=g).to(dtype).cuda()
    Lu, Ld = fmpq_mod.Fp8Layer(128, 2 * F, experts=E, gated=True), fmpq_mod.Fp8Layer(F, N, experts=E)
    Wu = fmpq_mod.fp8_pack_weights(Lu, (torch.randn(E, 2 * F, 128, generator=g) / 12).to(dtype).cuda())
    Wd = fmpq_mod.fp8_pack_weights(Ld, (torch.randn(E, N, F, generator=g) / F ** 0.5).to(dtype).cuda())
    ids, w = torch.from_numpy(draw_ids(T, k, E, T)).cuda(), (torch.rand(T, k, generator=g) + 0.1).cuda()
    plan = fmpq_mod.moe_plan(ids, E)
    H = fmpq_mod.moe_up(Lu, plan, *fmpq_mod.moe_quantize(Lu, plan, X), *Wu)
    wide = torch.full((plan.rows, N + pad), 7.0, device="cuda")       # rows of any stride, nothing past N written
    D = fmpq_mod.moe_down(Ld, plan, *H, *Wd, weights=w, dtype=dtype, D=wide[:, :N])
    assert bool((wide[:, N:] == 7.0).all())
    narrow = torch.empty((plan.rows, N + pad), dtype=dtype, device="cuda")[:, :N]
    fmpq_mod.moe_down(Ld, plan, *H, *Wd, weights=w, D=narrow)
    rows = plan.row_of.long().reshape(-1)
    used = rows[rows >= 0]
    assert torch.equal(narrow[used], D[used].to(dtype))
    for rows_of in (D, narrow):
        total = torch.zeros(T, N, device="cuda")
        for j in range(k):                                            # in slot order, FP32
            r = plan.row_of[:, j].long()
            total += torch.where((r >= 0)[:, None], rows_of[r.clamp(min=0)].float(), torch.zeros((), device="cuda"))
        Y = fmpq_mod.moe_combine(rows_of, plan)
        assert Y.dtype == dtype and torch.equal(Y, total.to(dtype))
    assert torch.equal(fmpq_mod.moe_combine(D, plan), fmpq_mod.moe_experts(Lu, Ld, X, ids, w, *Wu, *Wd))
    with pytest.raises(ValueError):
        fmpq_mod.moe_down(Ld, plan, *H, *Wd, weights=w, dtype=torch.float32)
    with pytest.raises(ValueError):
        fmpq_mod.moe_down(Ld, plan, *H, *Wd, D=narrow, dtype=torch.float16 if dtype == torch.bfloat16 else torch.bfloat16)


def test_combine_refusals():
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    lib, p = fmpq.load_library(), 4096   # never read: the arguments are refused first
    assert lib.moe_combine_f32(None, 8, p, 4, 2, 8, 8, p, 0, 8, None) == 1
    assert lib.moe_combine_f32(p, 8, p, 4, 2, 8, 8, p, 2, 8, None) == 1       # Y has 16 bits
    assert lib.moe_combine_f32(p, 7, p, 4, 2, 8, 8, p, 0, 8, None) == 2
    assert lib.moe_combine_f32(p + 2, 8, p, 4, 2, 8, 8, p, 0, 8, None) == 3
