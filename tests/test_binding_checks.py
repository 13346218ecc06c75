"""What the Python binding of the E4M3 layers and the routed experts refuses before the library sees a pointer. No GPU:
CPU tensors that claim to be on one stand in for the arguments, and a library that must not be called for the real one."""
import pytest
import torch

from bit_quantized_gemm_fmpq_gb300 import fmpq


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


class OnAnother(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 1


def on_gpu(t):
    return t.as_subclass(OnGpu)


class NoLibrary:
    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):    # a size, computed on the host
                return 64
            raise AssertionError(f"{name} was reached")
        return call


def layer_of(K, N, experts=1, gated=False):
    layer = object.__new__(fmpq.Fp8Layer)
    layer._lib, layer._h = NoLibrary(), None
    layer.K, layer.N, layer.experts, layer.gated = K, N, experts, gated
    layer.nb = -(-K // 128)
    layer.scale_rows = 2 * -(-(N // 2) // 128) if gated else -(-N // 128)
    pairs = -(-(N // 2) // 128) if gated else -(-N // 256)
    layer._w_bytes, layer._w_scales = experts * pairs * 2 * layer.nb * 128 * 128, experts * layer.scale_rows * layer.nb
    layer._workspaces, layer._workspace_bytes = {}, {}
    return layer


def weights_of(layer):
    return (on_gpu(torch.zeros(layer._w_bytes, dtype=torch.uint8)),
            on_gpu(torch.zeros(layer.experts, layer.scale_rows, layer.nb)))


def plan_of(T, k, experts, rows):
    plan = object.__new__(fmpq.MoePlan)
    plan.T, plan.k, plan.experts, plan.rows, plan.dtype = T, k, experts, rows, torch.float16
    plan.buffer = on_gpu(torch.zeros(2 * experts + T * k + rows, dtype=torch.int32))
    return plan


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(fmpq, "load_library", NoLibrary)
    monkeypatch.setattr(fmpq, "_lib", NoLibrary())
    monkeypatch.setattr(fmpq, "_on", lambda X: 0)
    monkeypatch.setattr(fmpq, "_device", lambda: 0, raising=False)
    monkeypatch.setattr(fmpq, "_stream", lambda s: 0)


def half(*shape):
    return on_gpu(torch.zeros(*shape, dtype=torch.float16))


def overlapping(M, K):
    """M rows of K that share storage: one row repeated, and windows one element apart."""
    return [half(1, K).expand(M, K), half(M + K).as_strided((M, K), (1, 1)), half(M * K).as_strided((M, K), (K - 1, 1))]


# ---- rows that overlap ------------------------------------------------------------------------

def test_row_stride():
    assert fmpq._ld(half(4, 8)) == 8 and fmpq._ld(half(4, 8)[:, :5]) == 8
    assert fmpq._ld(half(8, 6)[::2]) == 12 and fmpq._ld(half(1, 8).expand(1, 8)) == 8
    assert fmpq._ld(half(9)[2:].as_strided((1, 7), (3, 1))) == 7      # one row: any stride
    for X in overlapping(3, 8):
        with pytest.raises(ValueError):
            fmpq._ld(X)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_overlapping_rows_are_refused(which):
    layer, M = layer_of(256, 128), 5
    W, s = weights_of(layer)
    X = overlapping(M, 256)[which]
    A, a = on_gpu(torch.zeros(2, M, 128, dtype=torch.uint8)), on_gpu(torch.zeros(2, 8))
    calls = [
        lambda: fmpq.fp8_quantize(layer, X, A, a),
        lambda: fmpq.fp8_quantize_gemm(layer, X, W, s, A, a, Y=half(M, 128), workspace=half(8)),
        lambda: fmpq.fp8_quantize_gemm(layer, half(M, 256), W, s, A, a, Y=overlapping(M, 128)[which], workspace=half(8)),
        lambda: fmpq.fp8_gemm(layer, A, a, W, s, M, Y=overlapping(M, 128)[which], workspace=half(8)),
        lambda: fmpq.fp8_pack_weights(layer, overlapping(128, 256)[which]),
        lambda: fmpq.fp8_pack_codes(layer, on_gpu(torch.zeros(1, 256, dtype=torch.uint8)).expand(128, 256), s),
        lambda: fmpq.moe_route(X, 2),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    up, down, T, k = layer_of(256, 256, 3, True), layer_of(128, 256, 3), M, 2
    plan = plan_of(T, k, 3, 40)
    H, h = on_gpu(torch.zeros(1, 40, 128, dtype=torch.uint8)), on_gpu(torch.zeros(1, 40))
    ids, w = on_gpu(torch.zeros(T, k, dtype=torch.int32)), on_gpu(torch.zeros(T, k))
    calls = [
        lambda: fmpq.moe_quantize(up, plan, X, on_gpu(torch.zeros(2, 40, 128, dtype=torch.uint8)), on_gpu(torch.zeros(2, 40))),
        lambda: fmpq.moe_experts(up, down, X, ids, w, *weights_of(up), *weights_of(down)),
        lambda: fmpq.moe_down(down, plan, H, h, *weights_of(down), D=overlapping(40, 256)[which]),
        lambda: fmpq.moe_combine(overlapping(40, 256)[which], plan),
        lambda: fmpq.moe_combine(half(40, 256), plan, Y=overlapping(T, 256)[which]),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()


# ---- buffers that the caller passes -----------------------------------------------------------

def u8(*shape):
    return on_gpu(torch.zeros(*shape, dtype=torch.uint8))


def f32(*shape):
    return on_gpu(torch.zeros(*shape))


@pytest.mark.parametrize("bad", [
    (u8(1, 5, 128), f32(2, 8)), (u8(2, 5, 128)[:, :, :127], f32(2, 8)), (u8(2, 5, 128), f32(2, 5)), (u8(2, 5, 128), f32(1, 8)),
    (u8(2, 5, 128), f32(8, 2).t()), (u8(5, 2, 128).transpose(0, 1), f32(2, 8)),
    (None, f32(2, 4)), (u8(4), None),
])
def test_buffers_of_the_quantizers_are_large_enough(bad):
    layer = layer_of(256, 128)
    with pytest.raises(ValueError):
        fmpq.fp8_quantize(layer, half(5, 256), *bad)
    up = layer_of(256, 256, 3, True)
    with pytest.raises(ValueError):
        fmpq.moe_quantize(up, plan_of(2, 1, 3, 5), half(2, 256), *bad)


@pytest.mark.parametrize("bad", [(u8(1, 40, 128), None), (None, f32(1, 40)), (u8(2, 39, 128), None), (None, f32(2, 39)),
                                 (u8(40, 2, 128).transpose(0, 1), f32(2, 40))])
def test_buffers_of_the_hidden_vectors_are_large_enough(bad):
    up, plan = layer_of(128, 300, 3, True), plan_of(5, 2, 3, 40)     # 150 hidden channels: two blocks
    with pytest.raises(ValueError):
        fmpq.moe_up(up, plan, u8(1, 40, 128), f32(1, 40), *weights_of(up), *bad)


# ---- types, and tensors that are not on the GPU -----------------------------------------------

def calls_with_weights(W, s):
    """Every call that reads packed weights, each with W and s made for its own layer."""
    plain, down, up = layer_of(256, 128), layer_of(256, 128, 3), layer_of(256, 256, 3, True)
    A, a = u8(2, 40, 128), f32(2, 40)
    plan, ids, w = plan_of(5, 2, 3, 40), on_gpu(torch.zeros(5, 2, dtype=torch.int32)), f32(5, 2)
    square = layer_of(128, 256, 3)
    return [lambda: fmpq.fp8_unpack_weights(plain, W(plain), s(plain)),
            lambda: fmpq.fp8_gemm(plain, A, a, W(plain), s(plain), 5),
            lambda: fmpq.fp8_quantize_gemm(plain, half(5, 256), W(plain), s(plain)),
            lambda: fmpq.moe_up(up, plan, A, a, W(up), s(up)),
            lambda: fmpq.moe_down(down, plan, A, a, W(down), s(down)),
            lambda: fmpq.moe_experts(up, square, half(5, 256), ids, w, *weights_of(up), W(square), s(square)),
            lambda: fmpq.moe_experts(up, square, half(5, 256), ids, w, W(up), s(up), *weights_of(square))]


@pytest.mark.parametrize("W,s", [
    (lambda L: weights_of(L)[0], lambda L: weights_of(L)[1].half()),                       # fp16 scales of the right count
    (lambda L: weights_of(L)[0], lambda L: weights_of(L)[1].as_subclass(torch.Tensor)),    # on the host
    (lambda L: weights_of(L)[0].as_subclass(torch.Tensor), lambda L: weights_of(L)[1]),
    (lambda L: on_gpu(torch.zeros(2 * L._w_bytes, dtype=torch.uint8))[::2], lambda L: weights_of(L)[1]),
    (lambda L: on_gpu(torch.zeros(L._w_bytes, dtype=torch.int16)), lambda L: weights_of(L)[1]),
    (lambda L: weights_of(L)[0][16:], lambda L: weights_of(L)[1]),
    (lambda L: weights_of(L)[0], lambda L: f32(L.experts, L.scale_rows, L.nb + 1)),
])
def test_weights_are_of_the_layers_types(W, s):
    for call in calls_with_weights(W, s):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("bad", [
    (u8(2, 40, 128), f32(2, 40).half()), (on_gpu(torch.zeros(2, 40, 128, dtype=torch.int16)), f32(2, 40)),
    (torch.zeros(2, 40, 128, dtype=torch.uint8), f32(2, 40)), (u8(2, 40, 128), torch.zeros(2, 40)),
])
def test_activations_are_of_the_layers_types(bad):
    plain, down, up = layer_of(256, 128), layer_of(256, 128, 3), layer_of(256, 300, 3, True)
    plan = plan_of(5, 2, 3, 40)
    for call in (lambda: fmpq.fp8_quantize(plain, half(40, 256), *bad), lambda: fmpq.moe_quantize(up, plan, half(5, 256), *bad),
                 lambda: fmpq.fp8_gemm(plain, *bad, *weights_of(plain), 40),
                 lambda: fmpq.fp8_quantize_gemm(plain, half(40, 256), *weights_of(plain), *bad),
                 lambda: fmpq.moe_up(up, plan, *bad, *weights_of(up)),
                 lambda: fmpq.moe_up(up, plan, u8(2, 40, 128), f32(2, 40), *weights_of(up), *bad),
                 lambda: fmpq.moe_down(down, plan, *bad, *weights_of(down))):
        with pytest.raises(ValueError):
            call()


def test_outputs_and_workspaces_on_the_host_are_refused():
    with pytest.raises(ValueError):
        fmpq.moe_route(f32(5, 8), 2, ids=torch.zeros(5, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        fmpq.moe_route(f32(5, 8), 2, weights=torch.zeros(5, 2))
    plain = layer_of(256, 128)
    W, s = weights_of(plain)
    for ws in (torch.zeros(64, dtype=torch.uint8), on_gpu(torch.zeros(128, dtype=torch.uint8))[::2]):
        with pytest.raises(ValueError):
            fmpq.fp8_gemm(plain, u8(2, 5, 128), f32(2, 8), W, s, 5, workspace=ws)
        with pytest.raises(ValueError):
            fmpq.fp8_quantize_gemm(plain, half(5, 256), W, s, workspace=ws)


# ---- tensors of another GPU than the current one ----------------------------------------------

def elsewhere(t):
    return t.as_subclass(OnAnother)


def test_tensors_of_another_gpu_are_refused():
    plain, down, up = layer_of(256, 128), layer_of(128, 256, 3), layer_of(256, 256, 3, True)
    plan, ids, w = plan_of(5, 2, 3, 40), on_gpu(torch.zeros(5, 2, dtype=torch.int32)), f32(5, 2)
    A, a, H, h = u8(2, 40, 128), f32(2, 40), u8(1, 40, 128), f32(1, 40)
    W, X = weights_of, half(5, 256)
    far = lambda L: (elsewhere(weights_of(L)[0]), weights_of(L)[1])     # noqa: E731
    far_X, far_ids, far_w = elsewhere(half(5, 256)), elsewhere(ids), elsewhere(f32(5, 2))
    codes = on_gpu(torch.zeros(128, 256, dtype=torch.uint8))
    scales = f32(1, 2)
    calls = [
        lambda: fmpq.fp8_pack_weights(plain, elsewhere(half(128, 256))),
        lambda: fmpq.fp8_pack_codes(plain, elsewhere(codes), scales),
        lambda: fmpq.fp8_pack_codes(plain, codes, elsewhere(f32(1, 2))),
        lambda: fmpq.fp8_unpack_weights(plain, *far(plain)),
        lambda: fmpq.fp8_quantize(plain, far_X, A, a),
        lambda: fmpq.fp8_quantize(plain, X, elsewhere(u8(2, 40, 128)), a),
        lambda: fmpq.fp8_gemm(plain, A, a, *far(plain), 5),
        lambda: fmpq.fp8_gemm(plain, A, elsewhere(f32(2, 40)), *W(plain), 5),
        lambda: fmpq.fp8_gemm(plain, A, a, *W(plain), 5, Y=elsewhere(half(5, 128))),
        lambda: fmpq.fp8_gemm(plain, A, a, *W(plain), 5, workspace=elsewhere(u8(64))),
        lambda: fmpq.fp8_quantize_gemm(plain, far_X, *W(plain)),
        lambda: fmpq.fp8_quantize_gemm(plain, X, *far(plain)),
        lambda: fmpq.moe_route(elsewhere(f32(5, 8)), 2),
        lambda: fmpq.moe_route(f32(5, 8), 2, bias=elsewhere(f32(8))),
        lambda: fmpq.moe_route(f32(5, 8), 2, ids=far_ids),
        lambda: fmpq.moe_route(f32(5, 8), 2, weights=far_w),
        lambda: fmpq.moe_plan(far_ids, 3, plan),
        lambda: fmpq.moe_quantize(up, plan, far_X, A, a),
        lambda: fmpq.moe_up(up, plan, A, a, *far(up)),
        lambda: fmpq.moe_down(down, plan, H, h, *W(down), weights=far_w),
        lambda: fmpq.moe_down(down, plan, elsewhere(u8(1, 40, 128)), h, *W(down)),
        lambda: fmpq.moe_combine(elsewhere(half(40, 256)), plan),
        lambda: fmpq.moe_combine(half(40, 256), plan, Y=elsewhere(half(5, 256))),
        lambda: fmpq.moe_experts(up, down, far_X, ids, w, *W(up), *W(down)),
        lambda: fmpq.moe_experts(up, down, X, far_ids, w, *W(up), *W(down)),
        lambda: fmpq.moe_experts(up, down, X, ids, far_w, *W(up), *W(down)),
        lambda: fmpq.moe_experts(up, down, X, ids, w, *far(up), *W(down)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")


def test_a_plan_of_another_gpu_is_refused():
    plan = plan_of(5, 2, 3, 40)
    plan.buffer = elsewhere(plan.buffer)
    up, down = layer_of(256, 256, 3, True), layer_of(128, 256, 3)
    for call in (lambda: fmpq.moe_quantize(up, plan, half(5, 256), u8(2, 40, 128), f32(2, 40)),
                 lambda: fmpq.moe_up(up, plan, u8(2, 40, 128), f32(2, 40), *weights_of(up)),
                 lambda: fmpq.moe_down(down, plan, u8(1, 40, 128), f32(1, 40), *weights_of(down)),
                 lambda: fmpq.moe_plan(on_gpu(torch.zeros(5, 2, dtype=torch.int32)), 3, plan),
                 lambda: fmpq.moe_combine(half(40, 256), plan)):
        with pytest.raises(ValueError):
            call()


# ---- after a timeout --------------------------------------------------------------------------

@pytest.mark.parametrize("code,kept", [(0, True), (5, False)])
@pytest.mark.parametrize("clear", [False, True])
def test_workspaces_are_not_reused_after_an_error(code, kept, clear):
    """A product that gave up leaves counters in its workspace that the next one would take for its own."""
    class Library:
        def fp8_device_status(self, handle, status, do_clear):
            status._obj.value = code
            return 0

    layer = layer_of(8192, 256)
    layer._lib = Library()
    layer._workspaces = {(64, 0): u8(64)}
    assert fmpq.fp8_device_status(layer, clear) == code
    assert bool(layer._workspaces) == kept
