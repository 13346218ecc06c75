"""The norms between two blocks with gate, residual sum and quantizer (block_norm), against 64 bits.

Tolerances, with e = 2^-24 (half a step of FP32) and sizes of what is summed. r: the gate's product and the sum round
once each; a norm of X before it adds its own error. A row's sum is at most 66 additions deep in a thread (the long rows':
8 of 8 channels and one a vector) and 10 in the tree; mean, mean square, square root, the difference, the two products and the
bias round once each: fewer than 100 e of the sizes below in all, first order in e.
  size of norm(v): |w| inv (A + mean A + |d| inv^2 mean(|d| (A + mean A))) + |b|, A the size of v (at least |v|), d = v - c:
  an error of v's elements moves the element, the mean and the mean square.
The 16-bit outputs round once more, half a step of the type. A scale is within the largest error of its block over 448, and
a step of its own rounding; a code is between those of the smallest and the largest value that the errors allow.
"""
import ctypes

import pytest

from tests.test_binding_checks import NoLibrary, elsewhere, f32, half, layer_of, on_gpu, overlapping
from tests.test_fp8_linear import decode_activations, fmpq_mod  # noqa: F401  (the fixture)

BLOCK = 128
E = 2.0 ** -24


# ---- the definition, in 64 bits ---------------------------------------------------------------

def norm(kind, v, size, w, b, eps, offset):
    import torch
    c = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros(v.shape[0], 1, dtype=torch.float64)
    d = v - c
    inv = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    w = torch.ones(v.shape[1], dtype=torch.float64) if w is None else offset + w.cpu().double()
    b = torch.zeros(v.shape[1], dtype=torch.float64) if b is None else b.cpu().double()
    moved = size + (size.mean(1, keepdim=True) if kind == "layer" else 0)
    grown = w.abs() * inv * (moved + d.abs() * inv ** 2 * (d.abs() * moved).mean(1, keepdim=True)) + b.abs()
    return d * inv * w + b, grown


def define(X, residual=None, kind="rms", eps=1e-6, post_norm=False, post_weight=None, post_bias=None, gate=None,
           residual_scale=1.0, pre_norm=True, weight=None, bias=None, weight_offset=0.0):
    """(r, its size, y, its size)"""
    r = X.cpu().double()
    size = r.abs()
    if post_norm:
        r, size = norm(kind, r, size, post_weight, post_bias, eps, weight_offset)
    if gate is not None:
        g = gate.cpu().double()
        g = g[None] if g.dim() == 1 else g.repeat_interleave(X.shape[0] // g.shape[0], 0)
        r, size = r * g, size * g.abs()
    if residual is not None:
        add = residual_scale * residual.cpu().double()
        r, size = r + add, size + add.abs()
    y, grown = norm(kind, r, size, weight, bias, eps, weight_offset) if pre_norm else (None, None)
    return r, size, y, grown


def check16(got, ref, size):
    import torch
    info = torch.finfo(got.dtype)
    err = (got.cpu().double() - ref).abs()
    bound = ref.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2 + 100 * E * size * (1 + info.eps)
    assert bool((err <= bound).all()), float((err / bound).max())


def check_codes(A, s, y, size):
    import torch
    M, K = y.shape
    nb = -(-K // BLOCK)
    code, s = decode_activations(A, M, K), s.cpu().double()[:, :M].t()      # [M, nb * 128], [M, nb]
    y, off = torch.nn.functional.pad(y, (0, -K % BLOCK)), torch.nn.functional.pad(100 * E * size, (0, -K % BLOCK))
    top, most = y.abs().view(M, nb, BLOCK).amax(2) / 448, off.view(M, nb, BLOCK).amax(2) / 448
    assert bool(((s - top).abs() <= most + 2 * E * top + 2.0 ** -149).all())
    wide = s.repeat_interleave(BLOCK, 1)
    safe = torch.where(wide > 0, wide, torch.ones(()).double())

    def e4m3(v):
        v = torch.where(wide > 0, v / safe, torch.zeros(()).double())
        return (v * (1 + 2 * E * v.sign())).clamp(-448, 448)

    def rounded(v, up):   # (through FP32: the next value outwards first, so that no second rounding moves a code inwards)
        f = v.float()
        f = torch.nextafter(f, torch.full_like(f, float("inf") if up else float("-inf")))
        return f.clamp(-448, 448).to(torch.float8_e4m3fn).double()

    assert bool((code >= rounded(e4m3(y - off), False)).all()) and bool((code <= rounded(e4m3(y + off), True)).all())


# ---- on the GPU -------------------------------------------------------------------------------

def draw(M, K, dtype, seed, pad=0, amp=1.0, mean=0.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    out = torch.full((M, K + pad), 7.0, dtype=dtype)
    loud = torch.where(torch.rand(K, generator=g) < 0.02, 20.0, 1.0)
    out[:, :K] = (torch.randn(M, K, generator=g) * loud * amp + mean).to(dtype)
    return out.cuda()[:, :K]


def vectors(K, dtype, seed, n=4):
    import torch
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(K, generator=g) * 0.2 + (i % 2 == 0)).to(dtype).cuda() for i in range(n)]


SIZES = [(1, 8192, 0), (1, 1, 0), (3, 5, 1), (2, 127, 1), (5, 128, 0), (7, 129, 8), (400, 64, 0), (310, 250, 0), (33, 4096, 8),
         (350, 1024, 1), (320, 2868, 4), (305, 8192, 0), (305, 12000, 0), (2, 20000, 0), (3, 16385, 1), (1, 65536, 0),
         (1000, 512, 0), (5000, 520, 8), (700, 1000, 0), (2500, 2048, 0), (400, 16384, 0), (310, 28672, 0),
         (306, 20008, 8), (400, 5913, 1), (310, 21703, 3), (1300, 771, 0), (600, 513, 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,pad", SIZES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_all_of_it(fmpq_mod, M, K, pad, kind, dtype):  # noqa: F811
    """Both norms, a gate for each channel, the residual, 16 bits and codes."""
    import torch
    dtype = getattr(torch, dtype)
    X, residual = draw(M, K, dtype, M + K, pad, 0.5, 0.3), draw(M, K, dtype, M + K + 1, pad, 2.0)
    w, b, pw, pb = vectors(K, dtype if K % 16 else torch.float32, K)
    gate, = vectors(K, torch.float32 if K % 3 == 0 else dtype, K + 9, 1)
    if kind == "rms":
        b = pb = None
    layer = fmpq_mod.Fp8Layer(K, 16)
    Y = torch.full((M, K + pad), 7.0, dtype=dtype, device="cuda")
    kw = dict(kind=kind, eps=1e-5, post_norm=True, post_weight=pw, post_bias=pb, gate=gate, residual_scale=0.75, weight=w, bias=b,
              weight_offset=0.5)
    out = fmpq_mod.block_norm(X, residual, layer=layer, Y=Y[:, :K], **kw)
    r, size, y, grown = define(X, residual, **kw)
    check16(out.R, r, size)
    check16(out.Y, y, grown)
    check_codes(out.A_packed, out.a_scales, y, grown)
    assert bool((Y[:, K:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 4096), (6, 300), (400, 260), (3, 17000)])
@pytest.mark.parametrize("case", ["norm", "residual", "gate", "gate_batch", "gate_token", "post_only", "sum_only", "no_weight"])
def test_parts_alone(fmpq_mod, M, K, case):  # noqa: F811
    import torch
    dtype = torch.bfloat16
    X, residual = draw(M, K, dtype, K, 0, 0.5), draw(M, K, dtype, K + 1, 0, 2.0)
    w, pw = vectors(K, dtype, K, 2)
    g = torch.Generator().manual_seed(M)
    groups = 3 if M % 3 == 0 else 1
    kw, res = {
        "norm": (dict(weight=w), None),
        "residual": (dict(weight=w), residual),
        "gate": (dict(weight=w, gate=torch.randn(K, generator=g).cuda()), None),
        "gate_batch": (dict(weight=w, gate=torch.randn(groups, K + 8, generator=g).to(dtype).cuda()[:, :K]), residual),
        "gate_token": (dict(weight=w, gate=torch.randn(M, K, generator=g).cuda()), residual),
        "post_only": (dict(post_norm=True, post_weight=pw, pre_norm=False), residual),
        "sum_only": (dict(pre_norm=False, residual_scale=-1.5), residual),
        "no_weight": (dict(post_norm=True), residual),
    }[case]
    out = fmpq_mod.block_norm(X, res, **kw)
    r, size, y, grown = define(X, res, **kw)
    assert (out.R is None) == (case == "norm") and (out.Y is None) == (not kw.get("pre_norm", True))
    if out.R is not None:
        check16(out.R, r, size)
    if out.Y is not None:
        check16(out.Y, y, grown)
    assert out.A_packed is None and out.a_scales is None


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(2, 1024), (400, 1024), (2, 20000), (400, 2048), (320, 17000)])
def test_any_alignment_gives_the_same(fmpq_mod, M, K):  # noqa: F811
    """Weights, rows and outputs that start 2, 8 and 16 bytes into their buffers."""
    import torch
    X, residual = draw(M, K, torch.bfloat16, 1), draw(M, K, torch.bfloat16, 2)
    w, pw, gate = vectors(K, torch.bfloat16, 3, 3)
    layer = fmpq_mod.Fp8Layer(K, 16)
    ref = fmpq_mod.block_norm(X, residual, weight=w, post_norm=True, post_weight=pw, gate=gate, layer=layer)

    def at(v, shift):
        out = torch.empty(v.numel() + shift, dtype=v.dtype, device="cuda")[shift:].view(v.shape)
        return out.copy_(v)

    for shift in (1, 4, 8):
        for moved in range(4):
            a = [at(v, shift if i == moved else 0) for i, v in enumerate((X, residual, w, gate))]
            R = at(X, shift if moved == 0 else 0)
            out = fmpq_mod.block_norm(a[0], a[1], weight=a[2], post_norm=True, post_weight=pw, gate=a[3], layer=layer, R=R)
            # another kernel sums in another order: both are within 100 e of the same value, so 200 e = 1.2e-5 of each other.
            # R then differs by a bf16 step (2^-8) where the value is that near to a border, 1.2e-5 / 2^-8 = 0.3% of them: 2.2e-4 in
            # norm; a code where it is that near to one of E4M3's, at least 2^-4 apart: 2e-4 of them, and as many for the scale
            assert float((out.R.float() - ref.R.float()).norm()) <= 2.2e-4 * float(ref.R.float().norm())
            assert float((out.a_scales - ref.a_scales)[:, :M].abs().max()) <= 1.2e-5 * float(ref.a_scales[:, :M].max())
            assert float((out.A_packed != ref.A_packed).float().mean()) <= 4e-4


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 512), (333, 1024), (2, 17000), (700, 1003), (700, 2003), (400, 9001)])
def test_in_place(fmpq_mod, M, K):  # noqa: F811
    """R in the residual's buffer and Y in X's, or R in X's: the same values as in buffers of their own."""
    import torch
    X, residual = draw(M, K, torch.float16, 1), draw(M, K, torch.float16, 2)
    w, = vectors(K, torch.float16, 3, 1)
    ref = fmpq_mod.block_norm(X, residual, weight=w, post_norm=True)
    a, b = X.clone(), residual.clone()
    out = fmpq_mod.block_norm(a, b, weight=w, post_norm=True, R=b, Y=a)
    assert torch.equal(b, ref.R) and torch.equal(a, ref.Y) and out.R is b and out.Y is a
    a = X.clone()
    fmpq_mod.block_norm(a, residual, weight=w, post_norm=True, R=a)
    assert torch.equal(a, ref.R)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(9, 256), (9, 4096), (9, 17000), (400, 4096), (400, 2003), (330, 17003)])
def test_zeros_nan_and_infinity_stay_in_their_rows(fmpq_mod, M, K):  # noqa: F811
    import torch
    X, residual = draw(M, K, torch.bfloat16, 1), draw(M, K, torch.bfloat16, 2)
    layer = fmpq_mod.Fp8Layer(K, 16)
    Y = torch.empty_like(X)
    kw = dict(weight=vectors(K, torch.bfloat16, 3, 1)[0], layer=layer, post_norm=True)
    clean = fmpq_mod.block_norm(X, residual, Y=Y, **kw)
    X, residual, Z = X.clone(), residual.clone(), torch.empty_like(X)
    X[1], residual[1] = 0, 0
    X[3, K - 1] = float("nan")
    residual[5, 0] = float("inf")
    out = fmpq_mod.block_norm(X, residual, Y=Z, **kw)
    rest = [m for m in range(M) if m not in (1, 3, 5)]
    assert torch.equal(Z[rest], Y[rest]) and torch.equal(out.R[rest], clean.R[rest])
    assert torch.equal(out.a_scales[:, rest], clean.a_scales[:, rest]) and torch.equal(out.A_packed[:, rest], clean.A_packed[:, rest])
    assert bool((Z[1] == 0).all()) and bool((out.R[1] == 0).all()) and bool((out.a_scales[:, 1] == 0).all())
    assert bool((out.A_packed[:, 1] == 0).all())
    assert bool(Z[3].isnan().all()) and bool(out.a_scales[:, 3].isnan().all())
    assert float(out.R[5, 0]) == float("inf") and bool(Z[5, 0].isnan())


@pytest.mark.gpu
def test_graph_and_stream(fmpq_mod):  # noqa: F811
    import torch
    M, K = 40, 1024
    X, residual = draw(M, K, torch.bfloat16, 1), draw(M, K, torch.bfloat16, 2)
    w, = vectors(K, torch.bfloat16, 3, 1)
    ref = fmpq_mod.block_norm(X, residual, weight=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = fmpq_mod.block_norm(X, residual, weight=w, stream=side)
    side.synchronize()
    assert torch.equal(out.Y, ref.Y) and torch.equal(out.R, ref.R)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fmpq_mod.block_norm(X, residual, weight=w)
    X.copy_(draw(M, K, torch.bfloat16, 5))
    graph.replay()
    ref = fmpq_mod.block_norm(X, residual, weight=w)
    torch.cuda.synchronize()
    assert torch.equal(out.Y, ref.Y) and torch.equal(out.R, ref.R)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 1000), (37, 512), (400, 2868)])
def test_codes_feed_the_product(fmpq_mod, M, K):  # noqa: F811
    """fp8_gemm on the codes: the sum of their values' products, within the output's half step and FP32's sums."""
    import torch
    X = draw(M, K, torch.float16, K)
    layer = fmpq_mod.Fp8Layer(K, 200)
    W = fmpq_mod.fp8_pack_weights(layer, draw(200, K, torch.float16, 4))
    out = fmpq_mod.block_norm(X, layer=layer, weight=vectors(K, torch.float16, 5, 1)[0])
    assert out.R is None and out.Y is None
    got = fmpq_mod.fp8_gemm(layer, out.A_packed, out.a_scales, *W, M).double().cpu()
    x = (decode_activations(out.A_packed, M, K) * out.a_scales.cpu().double()[:, :M].t().repeat_interleave(BLOCK, 1))[:, :K]
    ref = x @ fmpq_mod.fp8_unpack_weights(layer, *W).cpu().double().t()
    assert float((got - ref).norm()) <= (2.0 ** -11 + 1e-5) * float(ref.norm())


# ---- refusals (no GPU) ------------------------------------------------------------------------

@pytest.fixture
def no_gpu(monkeypatch):
    from bit_quantized_gemm_fmpq_gb300 import fmpq
    monkeypatch.setattr(fmpq, "load_library", NoLibrary)
    monkeypatch.setattr(fmpq, "_lib", NoLibrary())
    monkeypatch.setattr(fmpq, "_on", lambda X: 0)
    monkeypatch.setattr(fmpq, "_device", lambda: 0)


def test_the_binding_refuses(no_gpu):
    import torch

    from bit_quantized_gemm_fmpq_gb300 import fmpq
    X, r, w = half(6, 64), half(6, 64), half(64)
    buf = half(6, 128)
    flat = half(6 * 64 + 64)
    shifted = (flat[:384].view(6, 64), flat[64:].view(6, 64))
    calls = [
        lambda: fmpq.block_norm(f32(6, 64)), lambda: fmpq.block_norm(half(64)), lambda: fmpq.block_norm(torch.zeros(6, 64).half()),
        lambda: fmpq.block_norm(X, half(6, 63)), lambda: fmpq.block_norm(X, on_gpu(torch.zeros(6, 64, dtype=torch.bfloat16))),
        lambda: fmpq.block_norm(X, kind="batch"), lambda: fmpq.block_norm(X, weight=half(63)),
        lambda: fmpq.block_norm(X, weight=half(1, 64)), lambda: fmpq.block_norm(X, weight=half(128)[::2]),
        lambda: fmpq.block_norm(X, weight=w, bias=f32(64)), lambda: fmpq.block_norm(X, weight=elsewhere(w)),
        lambda: fmpq.block_norm(X, post_weight=w), lambda: fmpq.block_norm(X, r, pre_norm=False, weight=w),
        lambda: fmpq.block_norm(X, gate=half(4, 64)), lambda: fmpq.block_norm(X, gate=half(6, 63)),
        lambda: fmpq.block_norm(X, gate=half(1, 64).expand(6, 64)), lambda: fmpq.block_norm(X, gate=torch.zeros(64).half()),
        lambda: fmpq.block_norm(X, layer=layer_of(65, 8)), lambda: fmpq.block_norm(X, A_packed=half(8)),
        lambda: fmpq.block_norm(X, R=half(6, 63)), lambda: fmpq.block_norm(X, Y=f32(6, 64)),
        lambda: fmpq.block_norm(overlapping(6, 64)[0]), lambda: fmpq.block_norm(X, overlapping(6, 64)[1]),
        lambda: fmpq.block_norm(X, r, R=r, Y=r), lambda: fmpq.block_norm(shifted[0], r, R=shifted[1]),
        lambda: fmpq.block_norm(buf[:, :64], r, Y=buf[:, 32:96]), lambda: fmpq.block_norm(X, r, weight=r[0], Y=r),
        lambda: fmpq.block_norm(X, gate=r, Y=r),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")


def test_column_ranges_of_one_buffer_are_apart(no_gpu):
    from bit_quantized_gemm_fmpq_gb300 import fmpq
    buf = half(6, 192)
    fmpq._apart(buf[:, 64:128], "R", buf[:, :64], buf[:, 128:])
    fmpq._apart(buf[:, :64], "R", buf[:, 64:])
    fmpq._apart(half(6, 8), "R", None, half(6, 8))


def test_the_library_refuses():
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    lib = fmpq.load_library()

    def status(**kw):
        a = fmpq.BlockNormArgs()
        base = dict(X=4096, ldx=64, M=4, K=64, Y=8192, ldy=64, eps=1e-6, residual_scale=1.0, pre_norm=1)
        for name, v in {**base, **kw}.items():
            setattr(a, name, v)
        return lib.fmpq_block_norm(ctypes.addressof(a), None)

    assert lib.fmpq_block_norm(None, None) == 1
    for kw in (dict(X=None), dict(dtype=2), dict(param_dtype=1), dict(kind=2), dict(eps=0.0), dict(eps=float("nan")),
               dict(Y=None), dict(pre_norm=0), dict(post_norm=2), dict(post_weight=64), dict(A_packed=4096),
               dict(gate=64, gate_tokens=1, gate_dtype=1, ldg=64), dict(residual_scale=float("inf"))):
        assert status(**kw) == 1, kw
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(K=0), dict(K=65537, ldx=65537, ldy=65537), dict(ldx=63), dict(ldy=63),
               dict(residual=4096, ldr=63), dict(R=4096, ldo=2), dict(gate=64, gate_tokens=0, ldg=64), dict(gate=64, gate_tokens=1, ldg=63)):
        assert status(**kw) == 2, kw
    for kw in (dict(X=4097), dict(Y=8193), dict(weight=4097), dict(A_packed=4098, a_scales=4096), dict(weight=4098, param_dtype=2)):
        assert status(**kw) == 3, kw
