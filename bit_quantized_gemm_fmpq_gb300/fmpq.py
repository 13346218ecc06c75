"""Thin Python binding of the C ABI in include/fmpq.h (argument marshalling only).

Every function here forwards to the CUDA library built in-tree
(bit_quantized_gemm_fmpq_gb300/_build/libfmpq_gb300.so); all the arithmetic runs in its
kernels. Torch is used only to own device memory and to supply the current CUDA stream.
If the library is missing, the first call raises ``FmpqLibraryMissing``: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading
from typing import NamedTuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfmpq_gb300.so")
BLOCK = 128
TILE_N = 256

_lib = None
_lock = threading.Lock()

STATUS = {
    0: "FMPQ_OK", 1: "FMPQ_ERR_INVALID_ARG", 2: "FMPQ_ERR_UNSUPPORTED_SHAPE", 3: "FMPQ_ERR_MISALIGNED",
    4: "FMPQ_ERR_CUDA", 5: "FMPQ_ERR_TIMEOUT", 6: "FMPQ_ERR_DEVICE", 7: "FMPQ_ERR_WORKSPACE",
}

# C-ABI symbols and their ctypes signatures (restype, argtypes)
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "fmpq_layout_create": (_I32, [_I32, _P, _P, ctypes.POINTER(_P)]),
    "fmpq_layout_destroy": (None, [_P]),
    "fmpq_layout_k": (_I32, [_P]),
    "fmpq_layout_num_blocks": (_I32, [_P]),
    "fmpq_layout_num_int8_blocks": (_I32, [_P]),
    "fmpq_packed_a_bytes": (_SZ, [_P, _I64]),
    "fmpq_packed_w_bytes": (_SZ, [_P, _I64]),
    "fmpq_quantize": (_I32, [_P, _P, _I64, _I64, _P, _P, _P]),
    "w4_pack_weights": (_I32, [_P, _P, _I64, _I64, _P, _P, _P]),
    "w4_unpack_weights": (_I32, [_P, _P, _I64, _P, _P]),
    "w4ax_gemm_workspace_bytes": (_SZ, [_P, _I64, _I64]),
    "w4ax_gemm": (_I32, [_P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _P]),
    "w4ax_gemm_noalloc": (_I32, [_P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P]),
    "w4ax_gemm_fault_test": (_I32, [_P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _I32, ctypes.c_uint32, _P]),
    "w4ax_gemm_partials": (_I32, [_P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "fmpq_device_status": (_I32, [_P, ctypes.POINTER(_I32), _I32]),
    "fmpq_rmsnorm_quantize": (_I32, [_P, _P, _I64, _I64, _P, ctypes.c_float, _P, _P, _P]),
    "fmpq_swiglu_quantize": (_I32, [_P, _P, _I64, _P, _I64, _I64, _P, _P, _P]),
    "fmpq_variant_gemm_workspace_bytes": (_SZ, [_P, _I64, _I64]),
    "fmpq_quantize_asym": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P]),
    "w4_weight_sums": (_I32, [_P, _P, _P, _I64, _P, _P]),
    "w4ax_gemm_asym": (_I32, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _P]),
    "qoq_pack_weights": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    "qoq_unpack_weights": (_I32, [_P, _P, _I64, _P, _P]),
    "qoq_quantize": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P]),
    "qoq_gemm": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _P]),
    "qoq_gemm_partials": (_I32, [_P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "fmpq_layout_create_select": (_I32, [_I32, _I32, _P, _P, ctypes.POINTER(_P)]),
    "fmpq_outlier_gemm_fp16": (_I32, [_P, _P, _I64, _I64, _P, _I32, _P, _I64, _I64, _P, _P, _I64, _P]),
    "fmpq_quantize_split": (_I32, [_P, _P, _I64, _I64, _P, _I32, _I32, _P, _P, _P, _P, _P]),
    "fmpq_quantize_gemm": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _I64, _P, _I64, _P]),
    "fmpq_outlier_product_fp16": (_I32, [_P, _P, _I64, _I32, _P, _I64, _I64, _P, _I64, _P]),
    "fmpq_channel_absmax": (_I32, [_P, _I64, _I64, _I32, _P, _P]),
    "fmpq_plan_layout": (_I32, [_I32, _P, _I32, _P, _P]),
    "fmpq_plan_layout_budget": (_I32, [_I32, _P, _P, _I64, _I64, ctypes.c_double, _P, _P, _P, _P]),
    "fmpq_outlier_blocks": (_I32, [_I32, ctypes.c_double]),
    "fp8_layer_create": (_I32, [_I32, _I32, _I32, _I32, ctypes.POINTER(_P)]),
    "fp8_layer_destroy": (None, [_P]),
    "fp8_device_status": (_I32, [_P, ctypes.POINTER(_I32), _I32]),
    "fp8_packed_w_bytes": (_SZ, [_P]),
    "fp8_weight_scale_count": (_SZ, [_P]),
    "fp8_packed_a_bytes": (_SZ, [_P, _I64]),
    "fp8_a_scale_count": (_SZ, [_P, _I64]),
    "fp8_pack_weights": (_I32, [_P, _I32, _P, _I32, _I64, _P, _P, _P]),
    "fp8_pack_codes": (_I32, [_P, _I32, _P, _I64, _P, _P]),
    "fp8_unpack_weights": (_I32, [_P, _I32, _P, _P, _P, _P]),
    "fp8_quantize": (_I32, [_P, _P, _I32, _I64, _I64, _P, _P, _P]),
    "fp8_gemm_workspace_bytes": (_SZ, [_P, _I64]),
    "fp8_gemm": (_I32, [_P, _P, _P, _P, _P, _I64, _P, _I32, _I64, _P, _SZ, _P]),
    "fp8_quantize_gemm": (_I32, [_P, _P, _I32, _I64, _I64, _P, _P, _P, _P, _P, _I64, _P, _SZ, _P]),
    "fp8_gemm_epilogue": (_I32, [_P, _P, _P, _P, _P, _I64, _P, _P, _I32, _I64, _P, _SZ, _P]),
    "fp8_quantize_gemm_epilogue": (_I32, [_P, _P, _I32, _I64, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _SZ, _P]),
    "fmpq_block_norm": (_I32, [_P, _P]),
    "fmpq_block_norm_fault_test": (_I32, [_P, _I64, ctypes.c_uint32, _P]),
    "moe_route": (_I32, [_P, _I32, _I64, _I64, _I32, _I32, _I32, _P, _I32, _I32, _I32, _I32, ctypes.c_float, _P, _P, _P]),
    "moe_rows": (_I64, [_I64, _I32, _I32]),
    "moe_plan_bytes": (_SZ, [_I64, _I32, _I32]),
    "moe_plan": (_I32, [_P, _I64, _I32, _I32, _P, _P]),
    "moe_quantize": (_I32, [_P, _P, _I64, _I32, _P, _I32, _I64, _P, _P, _P]),
    "moe_up": (_I32, [_P, _P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "moe_down": (_I32, [_P, _P, _I64, _I32, _P, _P, _P, _P, _P, _P, _I32, _I64, _P]),
    "moe_experts_bytes": (_SZ, [_P, _P, _I64, _I32]),
    "moe_experts": (_I32, [_P, _P, _P, _I32, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _SZ, _P]),
    "moe_combine_f32": (_I32, [_P, _I64, _P, _I64, _I32, _I32, _I32, _P, _I32, _I64, _P]),
    "moe_combine": (_I32, [_P, _I32, _I64, _P, _I64, _I32, _I32, _I32, _P, _I64, _P]),
    "w16_layer_create": (_I32, [_I32, _I32, _I32, _I32, _I32, ctypes.POINTER(_P)]),
    "w16_layer_destroy": (None, [_P]),
    "w16_device_status": (_I32, [_P, ctypes.POINTER(_I32), _I32]),
    "w16_packed_w_bytes": (_SZ, [_P]),
    "w16_pack_weights": (_I32, [_P, _I32, _P, _I64, _I64, _P, _P]),
    "w16_workspace_bytes": (_SZ, [_P, _P, _I64, _I64]),
    "w16_gemm": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _I32, _I64, _P, _SZ, _P]),
    "w16_gemm_fault_test": (_I32, [_P, _P, _I64, _I64, _P, _P, _I64, _I32, _I32, ctypes.c_uint32, _P]),
    "w16_grouped_gemm": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P, _I32, _I64, _P, _SZ, _P]),
    "w16_experts_workspace_bytes": (_SZ, [_P, _P, _I64, _I64, _I32, _I32]),
    "w16_experts_gemm": (_I32, [_P, _P, _I64, _I32, _P, _I64, _I32, _P, _P, _P, _P, _I32, _I64, _P, _SZ, _P]),
    "fmpq_status_string": (ctypes.c_char_p, [_I32]),
    "fmpq_version": (_I32, []),
}


class FmpqLibraryMissing(RuntimeError):
    pass


class FmpqError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")
        self.code = code


def load_library():
    """Load the in-tree CUDA library (raises FmpqLibraryMissing when it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise FmpqLibraryMissing(
                    f"{LIB_PATH} is missing: build it with `python -m bit_quantized_gemm_fmpq_gb300.build`")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype = res
                f.argtypes = args
            _lib = lib
    return _lib


def _check(fn: str, code: int):
    if code != 0:
        raise FmpqError(fn, code)


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


class Layout:
    """Owns an fmpq_layout* (channel permutation + outlier-block mask) on the current device."""

    def __init__(self, K: int, perm, mask):
        lib = load_library()
        perm = np.ascontiguousarray(perm, dtype=np.int32)
        mask = np.ascontiguousarray(mask, dtype=np.uint8)
        if perm.shape != (K,) or mask.shape != (K // BLOCK,):
            raise ValueError("perm must have K entries and mask K/128 entries")
        h = ctypes.c_void_p()
        _check("fmpq_layout_create", lib.fmpq_layout_create(K, perm.ctypes.data, mask.ctypes.data, ctypes.byref(h)))
        self._h = h
        self._lib = lib
        self.K = K
        self.nb = K // BLOCK
        self.mask = mask.copy()
        self.perm = perm.copy()
        self._workspaces = {}

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.fmpq_layout_destroy(self._h)
            self._h = ctypes.c_void_p()
        self._workspaces = {}

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def n8(self) -> int:
        return int(self._lib.fmpq_layout_num_int8_blocks(self._h))

    def packed_a_bytes(self, M: int) -> int:
        return int(self._lib.fmpq_packed_a_bytes(self._h, M))

    def packed_w_bytes(self, N: int) -> int:
        return int(self._lib.fmpq_packed_w_bytes(self._h, N))

    def workspace_bytes(self, M: int, N: int) -> int:
        return int(self._lib.w4ax_gemm_workspace_bytes(self._h, M, N))

    def workspace(self, M: int, N: int, variant: bool = False):
        """A zero-initialised, reusable workspace tensor for (M, N) (cached per size); variant:
        for the quantization variants' GEMMs."""
        import torch
        nbytes = (int(self._lib.fmpq_variant_gemm_workspace_bytes(self._h, M, N)) if variant
                  else self.workspace_bytes(M, N))
        if nbytes == 0:
            return None
        ws = self._workspaces.get(nbytes)
        if ws is None:
            ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
            self._workspaces[nbytes] = ws
        return ws


# ---- the C-ABI entry points, same names ---------------------------------------------------

def fmpq_layout_create(K: int, perm, mask) -> Layout:
    return Layout(K, perm, mask)


def fmpq_quantize(layout: Layout, X, A_packed=None, a_scales=None, stream=None):
    """X: fp16 CUDA tensor [M, >=K] (row stride multiple of 8). Returns (A_packed u8, a_scales fp16 [nb, M])."""
    import torch
    M = X.shape[0]
    if A_packed is None:
        A_packed = torch.empty(layout.packed_a_bytes(M), dtype=torch.uint8, device=X.device)
    if a_scales is None:
        a_scales = torch.empty((layout.nb, M), dtype=torch.float16, device=X.device)
    _check("fmpq_quantize", layout._lib.fmpq_quantize(layout.handle, _ptr(X), X.stride(0), M, _ptr(A_packed),
                                                        _ptr(a_scales), _stream(stream)))
    return A_packed, a_scales


def fmpq_swiglu_quantize(layout: Layout, G_perm, U_perm, A_packed=None, a_scales=None, stream=None):
    """SwiGLU (silu(g) * u, rounded once to fp16) fused with the activation quantizer; G_perm and
    U_perm fp16 [M, >=K] in the layout's permuted channel order."""
    import torch
    M = G_perm.shape[0]
    if A_packed is None:
        A_packed = torch.empty(layout.packed_a_bytes(M), dtype=torch.uint8, device=G_perm.device)
    if a_scales is None:
        a_scales = torch.empty((layout.nb, M), dtype=torch.float16, device=G_perm.device)
    _check("fmpq_swiglu_quantize", load_library().fmpq_swiglu_quantize(
        layout.handle, _ptr(G_perm), G_perm.stride(0), _ptr(U_perm), U_perm.stride(0), M, _ptr(A_packed),
        _ptr(a_scales), _stream(stream)))
    return A_packed, a_scales


def fmpq_rmsnorm_quantize(layout: Layout, X, gamma_perm, eps: float, A_packed=None, a_scales=None, stream=None):
    """RMSNorm of X fused with the activation quantizer (gamma in the permuted channel order)."""
    import torch
    M = X.shape[0]
    if A_packed is None:
        A_packed = torch.empty(layout.packed_a_bytes(M), dtype=torch.uint8, device=X.device)
    if a_scales is None:
        a_scales = torch.empty((layout.nb, M), dtype=torch.float16, device=X.device)
    _check("fmpq_rmsnorm_quantize", load_library().fmpq_rmsnorm_quantize(
        layout.handle, _ptr(X), X.stride(0), M, _ptr(gamma_perm), ctypes.c_float(eps), _ptr(A_packed),
        _ptr(a_scales), _stream(stream)))
    return A_packed, a_scales


def w4_pack_weights(layout: Layout, W, W_packed=None, w_scales=None, stream=None):
    """W: fp16 CUDA tensor [N, >=K]. Returns (W_packed u8, w_scales fp16 [nb, N])."""
    import torch
    N = W.shape[0]
    if W_packed is None:
        W_packed = torch.empty(layout.packed_w_bytes(N), dtype=torch.uint8, device=W.device)
    if w_scales is None:
        w_scales = torch.empty((layout.nb, N), dtype=torch.float16, device=W.device)
    _check("w4_pack_weights", layout._lib.w4_pack_weights(layout.handle, _ptr(W), W.stride(0), N, _ptr(W_packed),
                                                            _ptr(w_scales), _stream(stream)))
    return W_packed, w_scales


def w4_unpack_weights(layout: Layout, W_packed, N: int, stream=None):
    import torch
    Wq = torch.empty((N, layout.K), dtype=torch.int8, device=W_packed.device)
    _check("w4_unpack_weights", layout._lib.w4_unpack_weights(layout.handle, _ptr(W_packed), N, _ptr(Wq),
                                                                _stream(stream)))
    return Wq


def w4ax_gemm(layout: Layout, A_packed, a_scales, W_packed, w_scales, M: int, N: int, Y=None, workspace=None,
              stream=None):
    """Returns Y fp16 [M, N] (or writes into the given Y [M, >=N])."""
    import torch
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=A_packed.device)
    if workspace is None:
        workspace = layout.workspace(M, N)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check("w4ax_gemm", layout._lib.w4ax_gemm(layout.handle, _ptr(A_packed), _ptr(a_scales), _ptr(W_packed),
                                                _ptr(w_scales), M, N, _ptr(Y), Y.stride(0), _ptr(workspace),
                                                ws_bytes, _stream(stream)))
    return Y


def fmpq_quantize_gemm(layout: Layout, X, W_packed, w_scales, N: int, A_packed=None, a_scales=None, Y=None,
                       workspace=None, stream=None):
    """fmpq_quantize then w4ax_gemm in one call (the GEMM's prologue and weight stream overlap the
    quantizer). Returns Y (fp16 [M, N])."""
    import torch
    M = X.shape[0]
    if A_packed is None:
        A_packed = torch.empty(layout.packed_a_bytes(M), dtype=torch.uint8, device=X.device)
    if a_scales is None:
        a_scales = torch.empty((layout.nb, M), dtype=torch.float16, device=X.device)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    if workspace is None:
        workspace = layout.workspace(M, N)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check("fmpq_quantize_gemm", layout._lib.fmpq_quantize_gemm(
        layout.handle, _ptr(X), X.stride(0), M, _ptr(A_packed), _ptr(a_scales), _ptr(W_packed), _ptr(w_scales), N,
        _ptr(Y), Y.stride(0), _ptr(workspace), ws_bytes, _stream(stream)))
    return Y


def w4ax_gemm_fault_test(layout: Layout, A_packed, a_scales, W_packed, w_scales, M: int, N: int, withhold_copy: int,
                         poll_limit: int, Y=None, workspace=None, stream=None):
    """Debug/test of failure detection: w4ax_gemm with one packed weight copy of the first CTA
    withheld and every device wait bounded by poll_limit polls; records FMPQ_ERR_TIMEOUT."""
    import torch
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=A_packed.device)
    if workspace is None:
        workspace = layout.workspace(M, N)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check("w4ax_gemm_fault_test", layout._lib.w4ax_gemm_fault_test(
        layout.handle, _ptr(A_packed), _ptr(a_scales), _ptr(W_packed), _ptr(w_scales), M, N, _ptr(Y), Y.stride(0),
        _ptr(workspace), ws_bytes, int(withhold_copy), int(poll_limit), _stream(stream)))
    return Y


def w4ax_gemm_noalloc(layout: Layout, A_packed, a_scales, W_packed, w_scales, M: int, N: int, Y=None,
                      stream=None):
    """w4ax_gemm without a workspace argument: for callers that cannot allocate device memory,
    the library's own fixed device array serves as the split-K workspace."""
    import torch
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=A_packed.device)
    _check("w4ax_gemm_noalloc", layout._lib.w4ax_gemm_noalloc(layout.handle, _ptr(A_packed), _ptr(a_scales),
                                                                _ptr(W_packed), _ptr(w_scales), M, N, _ptr(Y),
                                                                Y.stride(0), _stream(stream)))
    return Y


def w4ax_gemm_partials(layout: Layout, A_packed, W_packed, M: int, N: int, m0: int, mcount: int, n0: int,
                       ncount: int, stream=None):
    """Exact per-block integer partial sums P int32 [mcount, ncount, nb] from the GEMM's tensor-core path."""
    import torch
    P = torch.zeros((mcount, ncount, layout.nb), dtype=torch.int32, device=A_packed.device)
    _check("w4ax_gemm_partials", layout._lib.w4ax_gemm_partials(layout.handle, _ptr(A_packed), _ptr(W_packed), M, N,
                                                                  m0, mcount, n0, ncount, _ptr(P), _stream(stream)))
    return P


def fmpq_device_status(layout: Layout, clear: bool = True) -> int:
    code = ctypes.c_int32(0)
    _check("fmpq_device_status", layout._lib.fmpq_device_status(layout.handle, ctypes.byref(code), int(clear)))
    return int(code.value)


def fmpq_version() -> int:
    return int(load_library().fmpq_version())


# ---------------------------------------------------------------------- calibration (offline)

def fmpq_channel_absmax(X, out=None, stream=None):
    """Per-channel absolute maximum of fp16 X [T][K] (rows may be strided): uint32 [K] of fp16
    bit patterns, computed on the GPU."""
    import torch
    T, K = X.shape
    if out is None:
        out = torch.empty(K, dtype=torch.int32, device=X.device)
    _check("fmpq_channel_absmax", load_library().fmpq_channel_absmax(_ptr(X), X.stride(0), T, K, _ptr(out),
                                                                         _stream(stream)))
    return out


def fmpq_plan_layout(absmax, n8: int):
    """Host planner: (perm int32 [K], mask uint8 [K/128]) from per-channel statistics."""
    a = np.ascontiguousarray(np.asarray(absmax).astype(np.uint32))
    K = a.size
    perm = np.empty(K, dtype=np.int32)
    mask = np.empty(K // BLOCK, dtype=np.uint8)
    _check("fmpq_plan_layout", load_library().fmpq_plan_layout(K, a.ctypes.data, n8, perm.ctypes.data,
                                                                   mask.ctypes.data))
    return perm, mask


def fmpq_plan_layout_budget(absmax, X_calib, eps: float):
    """Host planner with an error budget: the fewest INT8 blocks whose layout keeps the largest
    relative quantization error of the calibration tokens X_calib (fp16 [T, K], host) within
    eps. Returns (n8, err, perm int32 [K], mask uint8 [K/128])."""
    a = np.ascontiguousarray(np.asarray(absmax).astype(np.uint32))
    Xc = np.ascontiguousarray(np.asarray(X_calib, dtype=np.float16))
    T, K = Xc.shape
    perm = np.empty(K, dtype=np.int32)
    mask = np.empty(K // BLOCK, dtype=np.uint8)
    n8 = np.zeros(1, dtype=np.int32)
    err = np.zeros(1, dtype=np.float64)
    _check("fmpq_plan_layout_budget", load_library().fmpq_plan_layout_budget(
        K, a.ctypes.data, Xc.ctypes.data, T, K, float(eps), n8.ctypes.data, err.ctypes.data, perm.ctypes.data,
        mask.ctypes.data))
    return int(n8[0]), float(err[0]), perm, mask


def fmpq_outlier_blocks(K: int, fraction: float) -> int:
    n8 = int(load_library().fmpq_outlier_blocks(K, fraction))
    if n8 < 0:
        raise ValueError("K must be a multiple of 128 in [128, 32768] and fraction in [0, 1]")
    return n8


# ---------------------------------------------------------------------- outlier split (QUIK)

def select_layout(K: int, K_in: int, select, mask) -> "Layout":
    """A Layout over K channels selected (distinct indices < K_in) from rows of K_in channels."""
    lib = load_library()
    sel = np.ascontiguousarray(select, dtype=np.int32)
    mask = np.ascontiguousarray(mask, dtype=np.uint8)
    if sel.shape != (K,) or mask.shape != (K // BLOCK,):
        raise ValueError("select must have K entries and mask K/128 entries")
    h = ctypes.c_void_p()
    _check("fmpq_layout_create_select",
           lib.fmpq_layout_create_select(K, K_in, sel.ctypes.data, mask.ctypes.data, ctypes.byref(h)))
    lay = Layout.__new__(Layout)
    lay._h = h
    lay._lib = lib
    lay.K = K
    lay.nb = K // BLOCK
    lay.mask = mask.copy()
    lay.perm = sel.copy()
    lay._workspaces = {}
    return lay


def fmpq_outlier_gemm_fp16(layout: "Layout", X, cols, W_out, Y, X_out=None, stream=None):
    """Y += X[:, cols] @ W_out^T in FP16 (the outlier path of an outlier split); `layout` is the
    base part's layout (its device status word records device-side timeouts)."""
    import torch
    M = X.shape[0]
    n_out = cols.numel()
    N = W_out.shape[0]
    if X_out is None:
        X_out = torch.empty((M, n_out), dtype=torch.float16, device=X.device)
    _check("fmpq_outlier_gemm_fp16", load_library().fmpq_outlier_gemm_fp16(
        layout.handle, _ptr(X), X.stride(0), M, _ptr(cols), n_out, _ptr(W_out), W_out.stride(0), N, _ptr(X_out), _ptr(Y),
        Y.stride(0), _stream(stream)))
    return Y


def fmpq_quantize_split(layout: "Layout", X, cols, asym: bool = False, A_packed=None, a_scales=None, a_zeros=None,
                        X_out=None, stream=None):
    """The quantizer (symmetric, or asymmetric with asym=True) that also splits off X[:, cols]
    into X_out in the same pass. Returns (A_packed, a_scales, a_zeros or None, X_out)."""
    import torch
    M = X.shape[0]
    n_out = cols.numel()
    if A_packed is None:
        A_packed = torch.empty(layout.packed_a_bytes(M), dtype=torch.uint8, device=X.device)
    if a_scales is None:
        a_scales = torch.empty((layout.nb, M), dtype=torch.float16, device=X.device)
    if asym and a_zeros is None:
        a_zeros = torch.empty((layout.nb, M), dtype=torch.float16, device=X.device)
    if X_out is None:
        X_out = torch.empty((M, n_out), dtype=torch.float16, device=X.device)
    _check("fmpq_quantize_split", layout._lib.fmpq_quantize_split(
        layout.handle, _ptr(X), X.stride(0), M, _ptr(cols), n_out, 1 if asym else 0, _ptr(A_packed), _ptr(a_scales),
        _ptr(a_zeros if asym else None), _ptr(X_out), _stream(stream)))
    return A_packed, a_scales, (a_zeros if asym else None), X_out


def fmpq_outlier_product_fp16(layout: "Layout", X_out, W_out, Y, stream=None):
    """Y = fp16(Y + fp16(X_out @ W_out^T)) with X_out already split off (fmpq_quantize_split)."""
    M, n_out = X_out.shape
    N = W_out.shape[0]
    _check("fmpq_outlier_product_fp16", load_library().fmpq_outlier_product_fp16(
        layout.handle, _ptr(X_out), M, n_out, _ptr(W_out), W_out.stride(0), N, _ptr(Y), Y.stride(0), _stream(stream)))
    return Y


# ---- quantization variants: QUIK asymmetric activations, QoQ progressive group quantization

def _gemm_ws(layout: Layout, M: int, N: int, workspace):
    if workspace is None:
        workspace = layout.workspace(M, N, variant=True)
    return workspace, (workspace.numel() if workspace is not None else 0)


def fmpq_quantize_asym(layout: Layout, X, A_packed=None, a_scales=None, a_zeros=None, stream=None):
    """Asymmetric 4-bit activations. Returns (A_packed u8, a_scales fp16 [nb, M], a_zeros fp16 [nb, M])."""
    import torch
    M = X.shape[0]
    if A_packed is None:
        A_packed = torch.empty(layout.packed_a_bytes(M), dtype=torch.uint8, device=X.device)
    if a_scales is None:
        a_scales = torch.empty((layout.nb, M), dtype=torch.float16, device=X.device)
    if a_zeros is None:
        a_zeros = torch.empty((layout.nb, M), dtype=torch.float16, device=X.device)
    _check("fmpq_quantize_asym", layout._lib.fmpq_quantize_asym(layout.handle, _ptr(X), X.stride(0), M, _ptr(A_packed),
                                                                  _ptr(a_scales), _ptr(a_zeros), _stream(stream)))
    return A_packed, a_scales, a_zeros


def w4_weight_sums(layout: Layout, W_packed, w_scales, N: int, out=None, stream=None):
    """w_sums fp32 [nb, N] = w_scales * (sum of each block's weight codes)."""
    import torch
    if out is None:
        out = torch.empty((layout.nb, N), dtype=torch.float32, device=W_packed.device)
    _check("w4_weight_sums", layout._lib.w4_weight_sums(layout.handle, _ptr(W_packed), _ptr(w_scales), N, _ptr(out),
                                                          _stream(stream)))
    return out


def w4ax_gemm_asym(layout: Layout, A_packed, a_scales, a_zeros, W_packed, w_scales, w_sums, M: int, N: int,
                   Y=None, workspace=None, stream=None):
    import torch
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=A_packed.device)
    workspace, ws_bytes = _gemm_ws(layout, M, N, workspace)
    _check("w4ax_gemm_asym", layout._lib.w4ax_gemm_asym(
        layout.handle, _ptr(A_packed), _ptr(a_scales), _ptr(a_zeros), _ptr(W_packed), _ptr(w_scales), _ptr(w_sums),
        M, N, _ptr(Y), Y.stride(0), _ptr(workspace), ws_bytes, _stream(stream)))
    return Y


def qoq_pack_weights(layout: Layout, W, W_packed=None, stream=None):
    """Returns (W_packed u8, ch_scales fp16 [N], grp_scales u8 [nb, N], grp_zeros u8 [nb, N])."""
    import torch
    N = W.shape[0]
    if W_packed is None:
        W_packed = torch.empty(layout.packed_w_bytes(N), dtype=torch.uint8, device=W.device)
    s1 = torch.empty(N, dtype=torch.float16, device=W.device)
    s2 = torch.empty((layout.nb, N), dtype=torch.uint8, device=W.device)
    z2 = torch.empty((layout.nb, N), dtype=torch.uint8, device=W.device)
    _check("qoq_pack_weights", layout._lib.qoq_pack_weights(layout.handle, _ptr(W), W.stride(0), N, _ptr(W_packed),
                                                              _ptr(s1), _ptr(s2), _ptr(z2), _stream(stream)))
    return W_packed, s1, s2, z2


def qoq_unpack_weights(layout: Layout, W_packed, N: int, stream=None):
    import torch
    q4 = torch.empty((N, layout.K), dtype=torch.uint8, device=W_packed.device)
    _check("qoq_unpack_weights", layout._lib.qoq_unpack_weights(layout.handle, _ptr(W_packed), N, _ptr(q4),
                                                                  _stream(stream)))
    return q4


def qoq_quantize(layout: Layout, X, A_packed=None, a_scales=None, a_sums=None, stream=None):
    """Per-token INT8 activations. Returns (A_packed u8, a_scales fp16 [M], a_sums int32 [nb, M])."""
    import torch
    M = X.shape[0]
    if A_packed is None:
        A_packed = torch.empty(layout.packed_a_bytes(M), dtype=torch.uint8, device=X.device)
    if a_scales is None:
        a_scales = torch.empty(M, dtype=torch.float16, device=X.device)
    if a_sums is None:
        a_sums = torch.empty((layout.nb, M), dtype=torch.int32, device=X.device)
    _check("qoq_quantize", layout._lib.qoq_quantize(layout.handle, _ptr(X), X.stride(0), M, _ptr(A_packed),
                                                      _ptr(a_scales), _ptr(a_sums), _stream(stream)))
    return A_packed, a_scales, a_sums


def qoq_gemm(layout: Layout, A_packed, a_scales, a_sums, W_packed, ch_scales, grp_scales, grp_zeros, M: int,
             N: int, Y=None, workspace=None, stream=None):
    import torch
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=A_packed.device)
    workspace, ws_bytes = _gemm_ws(layout, M, N, workspace)
    _check("qoq_gemm", layout._lib.qoq_gemm(
        layout.handle, _ptr(A_packed), _ptr(a_scales), _ptr(a_sums), _ptr(W_packed), _ptr(ch_scales),
        _ptr(grp_scales), _ptr(grp_zeros), M, N, _ptr(Y), Y.stride(0), _ptr(workspace), ws_bytes, _stream(stream)))
    return Y


def qoq_gemm_partials(layout: Layout, A_packed, W_packed, M: int, N: int, m0: int, mcount: int, n0: int,
                      ncount: int, stream=None):
    import torch
    P = torch.zeros((mcount, ncount, layout.nb), dtype=torch.int32, device=A_packed.device)
    _check("qoq_gemm_partials", layout._lib.qoq_gemm_partials(layout.handle, _ptr(A_packed), _ptr(W_packed), M, N,
                                                                m0, mcount, n0, ncount, _ptr(P), _stream(stream)))
    return P


# ---- E4M3 linear layers: a scale for each block of 128 ------------------------------------
# Every call below also takes stream=: it then runs, and allocates, as under torch.cuda.stream(stream).
# Tensors are on torch's current GPU, which is the layer's.

def _on_stream(call):
    """Run a call under its `stream` argument (a torch stream or a raw handle), so that its buffers come from
    that stream's memory and are not given to other work before it is done."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        import torch
        with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
            return call(*args, **kw)
    return wrapped


_DTYPES = {}


def _dtype_code(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    code = _DTYPES.get(t)
    if code is None:
        raise ValueError(f"unsupported dtype {t}")
    return code


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


_current_device = None


def _device() -> int:
    global _current_device
    if _current_device is None:
        import torch
        _current_device = torch._C._cuda_getDevice
    return _current_device()


def _here(a, b=None) -> bool:
    """Whether the tensors are on the current GPU (a host tensor's device is -1)."""
    device = _device()
    return a.get_device() == device and (b is None or b.get_device() == device)


def _codes_and_scales(codes, scales) -> bool:
    return (_here(codes, scales) and codes.element_size() == 1 and _dtype_code(scales.dtype) == 2 and
            codes.is_contiguous() and scales.is_contiguous())


def _need_activations(codes, scales, nb: int, rows: int, what: str):
    """Codes [nb, rows, 128] and scales [nb, rows rounded up to 4], or larger."""
    _need(_codes_and_scales(codes, scales) and codes.numel() >= nb * rows * BLOCK and
          scales.numel() >= nb * ((rows + 3) // 4 * 4), f"{what} must be contiguous bytes and fp32 on the current GPU, large enough for the rows")


def _rows16(X, what: str, fp32: bool = False) -> int:
    """A 16-bit (fp32: or FP32) CUDA matrix whose rows are contiguous (any row stride). Returns its dtype code."""
    code = _dtype_code(X.dtype)
    if not (X.dim() == 2 and (code < 2 or fp32) and _here(X)):
        raise ValueError(f"{what} must be a 2-D {'fp32, ' if fp32 else ''}fp16 or bf16 tensor on the current GPU")
    if X.shape[1] > 1 and X.stride(1) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return code


def _ld(X) -> int:
    """Row stride in elements (a single row may have any). Rows that share storage (an expanded tensor, windows that
    overlap) are refused: the kernels take rows one after another."""
    rows, width = X.shape
    if rows <= 1:
        return width
    ld = X.stride(0)
    if ld < width:
        raise ValueError("the rows of a matrix must not overlap (an expanded tensor needs .contiguous())")
    return ld


def _extent(t):
    """First and last byte address of a matrix, exclusive."""
    at, size = t.data_ptr(), t.element_size()
    return at, at + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * size


def _apart(out, what: str, *inputs, same=()):
    """Refuse an output that shares memory with an input, unless it is in `same` and has its very rows. Column ranges of
    one buffer are apart."""
    lo, hi = _extent(out)
    for t in inputs:
        if t is None:
            continue
        a, b = _extent(t)
        if hi <= a or b <= lo:
            continue
        rows = out.shape[0] <= 1 or out.stride(0) == t.stride(0)
        if lo == a and rows and out.dtype == t.dtype and any(t is x for x in same):
            continue
        if rows and t.dim() == out.dim() == 2 and out.element_size() == t.element_size() and out.shape[0] > 1:
            ld = out.stride(0) * out.element_size()
            gap = (a - lo) % ld     # t's columns start this many bytes behind out's, and end before out's next row
            if gap >= out.shape[1] * out.element_size() and gap + t.shape[1] * t.element_size() <= ld:
                continue
        raise ValueError(f"{what} must not overlap an input")


class Epilogue(ctypes.Structure):
    """fmpq_epilogue of include/fmpq.h."""
    _fields_ = [("bias", _P), ("residual", _P), ("ldr", _I64), ("bias_dtype", _I32), ("activation", _I32)]


ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


_pack_epilogue = struct.Struct("@PPqii").pack    # Epilogue, faster than by its fields


def _epilogue(bias, activation, residual, shape, biases, code: int, Y=None):
    """The bytes of a product's epilogue with outputs of `shape` and the type `code`, or None where nothing is asked for.
    Y: the output that was passed, if one was."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be None, 'relu', 'silu', 'gelu' or 'gelu_tanh'")
    b_ptr = b_code = r_ptr = ldr = 0
    if bias is not None:
        if not (bias.shape == biases and _here(bias) and bias.is_contiguous()):
            raise ValueError(f"bias must be a contiguous tensor {list(biases)} on the current GPU")
        b_ptr, b_code = bias.data_ptr(), _dtype_code(bias.dtype)
        _need(b_code == code or b_code == 2, "bias must be of the output's type or fp32")
    if residual is not None:
        _need(_rows16(residual, "residual", fp32=True) == code and residual.shape == shape,
              "residual must have the output's shape and type")
        r_ptr, ldr = residual.data_ptr(), _ld(residual)
    if Y is not None:
        _apart(Y, "Y", residual, bias, same=(residual,))
    if b_ptr == 0 and r_ptr == 0 and act == 0:
        return None
    return _pack_epilogue(b_ptr, r_ptr, ldr, b_code, act)


def _on(X) -> int:
    """torch's current stream for X's device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(X.get_device())


class Fp8Layer:
    """Owns an fp8_layer*: `experts` E4M3 weight matrices [N, K] with 128 x 128 block scales (one: a
    linear layer); gated: N = 2F rows, F gate rows then F up rows (for moe_up)."""

    def __init__(self, K: int, N: int, experts: int = 1, gated: bool = False):
        lib = load_library()
        h = ctypes.c_void_p()
        _check("fp8_layer_create", lib.fp8_layer_create(K, N, experts, int(gated), ctypes.byref(h)))
        self._h = h
        self._lib = lib
        self.K, self.N, self.experts, self.gated = K, N, experts, bool(gated)
        self.nb = -(-K // BLOCK)
        self.scale_rows = 2 * -(-(N // 2) // BLOCK) if gated else -(-N // BLOCK)
        self._workspaces = {}
        self._workspace_bytes = {}
        self._w_bytes = int(lib.fp8_packed_w_bytes(h))
        self._w_scales = int(lib.fp8_weight_scale_count(h))

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.fp8_layer_destroy(self._h)
            self._h = ctypes.c_void_p()
        self._workspaces = {}

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def packed_w_bytes(self) -> int:
        return self._w_bytes

    def check_weights(self, W_packed, w_scales):
        _need(_codes_and_scales(W_packed, w_scales) and W_packed.numel() == self._w_bytes and w_scales.numel() == self._w_scales,
              "W_packed and w_scales must be this layer's (fp8_pack_weights, fp8_pack_codes)")

    def check_activations(self, A_packed, a_scales, rows: int):
        _need_activations(A_packed, a_scales, self.nb, rows, "A_packed and a_scales")

    def activations(self, rows: int, device):
        """Buffers for `rows` rows of quantized activations: codes uint8 [nb, rows, 128] (swizzled) and
        scales fp32 [nb, rows rounded up to 4]."""
        import torch
        return (torch.empty((self.nb, rows, BLOCK), dtype=torch.uint8, device=device),
                torch.empty((self.nb, (rows + 3) // 4 * 4), dtype=torch.float32, device=device))

    def workspace(self, M: int):
        """fp8_gemm's workspace for M rows: zeroed, reused by later calls on the same stream; one that a
        stream capture creates belongs to that graph alone."""
        import torch
        nbytes = self._workspace_bytes.get(M)
        if nbytes is None:
            nbytes = self._workspace_bytes[M] = int(self._lib.fp8_gemm_workspace_bytes(self._h, M))
        if nbytes == 0:
            return None
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        key = (nbytes, torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
        ws = self._workspaces.get(key)
        if ws is None:
            ws = self._workspaces[key] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        return ws


@_on_stream
def fp8_pack_weights(layer: Fp8Layer, W):
    """Quantize W (fp16 or bf16, [N, K], or [experts, N, K]) per 128 x 128 block. Returns (W_packed u8,
    w_scales fp32 [experts, scale rows, nb])."""
    import torch
    W3 = W if W.dim() == 3 else W[None]
    _need(W3.shape == (layer.experts, layer.N, layer.K), "W must be [experts, N, K] (or [N, K])")
    Wp = torch.empty(layer.packed_w_bytes(), dtype=torch.uint8, device=W.device)
    ws = torch.empty((layer.experts, layer.scale_rows, layer.nb), dtype=torch.float32, device=W.device)
    for e in range(layer.experts):
        _rows16(W3[e], "W")
        _check("fp8_pack_weights", layer._lib.fp8_pack_weights(layer.handle, e, _ptr(W3[e]), _dtype_code(W.dtype),
                                                               _ld(W3[e]), _ptr(Wp), _ptr(ws), _stream(None)))
    return Wp, ws


@_on_stream
def fp8_pack_codes(layer: Fp8Layer, codes, scales):
    """Lay out an E4M3 checkpoint: codes float8_e4m3fn (or its bytes) [experts, N, K] or [N, K], scales
    fp32 [experts, scale rows, nb] or [scale rows, nb] (value = code * scale). Returns (W_packed u8,
    w_scales)."""
    import torch
    C = codes if codes.dim() == 3 else codes[None]
    S = scales if scales.dim() == 3 else scales[None]
    _need(codes.dtype in (torch.float8_e4m3fn, torch.uint8) and _here(codes), "codes must be float8_e4m3fn on the current GPU")
    _need(C.shape == (layer.experts, layer.N, layer.K), "codes must be [experts, N, K] (or [N, K])")
    _need(S.shape == (layer.experts, layer.scale_rows, layer.nb) and S.dtype == torch.float32 and _here(S),
          "scales must be fp32 on the current GPU, [experts, scale rows, blocks of K]")
    _need(C.shape[2] <= 1 or C.stride(2) == 1, "codes must have contiguous rows")
    Wp = torch.empty(layer.packed_w_bytes(), dtype=torch.uint8, device=codes.device)
    for e in range(layer.experts):
        _check("fp8_pack_codes", layer._lib.fp8_pack_codes(layer.handle, e, _ptr(C[e]), _ld(C[e]), _ptr(Wp),
                                                           _stream(None)))
    return Wp, S.contiguous()


@_on_stream
def fp8_unpack_weights(layer: Fp8Layer, W_packed, w_scales, expert: int = 0):
    import torch
    layer.check_weights(W_packed, w_scales)
    W = torch.empty((layer.N, layer.K), dtype=torch.float32, device=W_packed.device)
    _check("fp8_unpack_weights", layer._lib.fp8_unpack_weights(layer.handle, expert, _ptr(W_packed), _ptr(w_scales),
                                                               _ptr(W), _stream(None)))
    return W


@_on_stream
def fp8_quantize(layer: Fp8Layer, X, A_packed=None, a_scales=None):
    """X fp16 or bf16 [M, K], any row stride. Returns (A_packed u8, a_scales fp32), see
    Fp8Layer.activations."""
    _rows16(X, "X")
    _need(X.shape[1] == layer.K, "X must be [M, K]")
    M = X.shape[0]
    if A_packed is None or a_scales is None:
        A, s = layer.activations(M, X.device)
        A_packed, a_scales = A if A_packed is None else A_packed, s if a_scales is None else a_scales
    layer.check_activations(A_packed, a_scales, M)
    _check("fp8_quantize", layer._lib.fp8_quantize(layer.handle, _ptr(X), _dtype_code(X.dtype), _ld(X), M,
                                                   _ptr(A_packed), _ptr(a_scales), _stream(None)))
    return A_packed, a_scales


def _workspace_of(layer: Fp8Layer, M: int, workspace):
    """The pointer and the bytes of the workspace passed, or of the layer's own."""
    if workspace is None:
        workspace = layer.workspace(M)
        return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _need(_here(workspace) and workspace.is_contiguous(), "workspace must be a contiguous tensor on the current GPU")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


@_on_stream
def fp8_gemm(layer: Fp8Layer, A_packed, a_scales, W_packed, w_scales, M: int, dtype=None, Y=None, workspace=None,
             bias=None, activation=None, residual=None):
    """Y [M, N] (fp16 by default) of quantized activations and packed weights: act(product + bias) + residual, rounded
    once. bias [N] (Y's type or fp32); activation None, "relu", "silu", "gelu" or "gelu_tanh"; residual [M, N] of Y's
    type, which may be Y."""
    import torch
    epilogue = None
    if bias is not None or activation is not None or residual is not None:
        code = _dtype_code(Y.dtype if Y is not None else dtype or torch.float16)
        epilogue = _epilogue(bias, activation, residual, (M, layer.N), (layer.N,), code, Y)
    if Y is None:
        Y = torch.empty((M, layer.N), dtype=dtype or torch.float16, device=A_packed.device)
    _rows16(Y, "Y")
    _need(Y.shape == (M, layer.N), "Y must be [M, N]")
    if not layer.gated:  # the library refuses a gated one
        layer.check_weights(W_packed, w_scales)
        layer.check_activations(A_packed, a_scales, M)
    w_ptr, w_bytes = _workspace_of(layer, M, workspace)
    if epilogue is not None:
        _check("fp8_gemm", layer._lib.fp8_gemm_epilogue(
            layer.handle, _ptr(A_packed), _ptr(a_scales), _ptr(W_packed), _ptr(w_scales), M, epilogue, _ptr(Y),
            _dtype_code(Y.dtype), _ld(Y), w_ptr, w_bytes, _stream(None)))
        return Y
    _check("fp8_gemm", layer._lib.fp8_gemm(layer.handle, _ptr(A_packed), _ptr(a_scales), _ptr(W_packed), _ptr(w_scales), M,
                                           _ptr(Y), _dtype_code(Y.dtype), _ld(Y), w_ptr, w_bytes,
                                           _stream(None)))
    return Y


@_on_stream
def fp8_quantize_gemm(layer: Fp8Layer, X, W_packed, w_scales, A_packed=None, a_scales=None, Y=None, workspace=None,
                      bias=None, activation=None, residual=None):
    """The layer on X (fp16 or bf16 [M, K]) in one call: Y [M, N] of X's type; bias, activation and residual as
    fp8_gemm takes them."""
    import torch
    code = _rows16(X, "X")
    M, K = X.shape
    _need(K == layer.K, "X must be [M, K]")
    layer.check_weights(W_packed, w_scales)
    _need((A_packed is None) == (a_scales is None), "pass both A_packed and a_scales, or neither")
    if A_packed is not None:
        layer.check_activations(A_packed, a_scales, M)
        a_ptr, s_ptr = A_packed.data_ptr(), a_scales.data_ptr()
    else:
        # one scratch buffer: codes, then scales
        codes = layer.nb * M * BLOCK
        scratch = torch.empty(codes + layer.nb * ((M + 3) // 4 * 16), dtype=torch.uint8, device=X.device)
        a_ptr = scratch.data_ptr()
        s_ptr = a_ptr + codes
    epilogue = None
    if bias is not None or activation is not None or residual is not None:
        epilogue = _epilogue(bias, activation, residual, (M, layer.N), (layer.N,), code, Y)
    if Y is None:
        Y = torch.empty((M, layer.N), dtype=X.dtype, device=X.device)
    else:
        _need(_rows16(Y, "Y") == code and Y.shape == (M, layer.N), "Y must be [M, N] of X's type")
    w_ptr, w_bytes = _workspace_of(layer, M, workspace)
    if epilogue is not None:
        _check("fp8_quantize_gemm", layer._lib.fp8_quantize_gemm_epilogue(
            layer._h, X.data_ptr(), code, _ld(X), M, a_ptr, s_ptr, W_packed.data_ptr(), w_scales.data_ptr(),
            epilogue, Y.data_ptr(), _ld(Y), w_ptr, w_bytes, _on(X)))
        return Y
    _check("fp8_quantize_gemm", layer._lib.fp8_quantize_gemm(
        layer._h, X.data_ptr(), code, _ld(X), M, a_ptr, s_ptr, W_packed.data_ptr(), w_scales.data_ptr(), Y.data_ptr(),
        _ld(Y), w_ptr, w_bytes, _on(X)))
    return Y


def fp8_device_status(layer: Fp8Layer, clear: bool = True) -> int:
    """The layer's status word (0, or 5 after a wait that gave up). After an error the layer's own workspaces are
    dropped, new ones being zeroed; one that the caller passes has to be zeroed by the caller."""
    code = ctypes.c_int32(0)
    _check("fp8_device_status", layer._lib.fp8_device_status(layer.handle, ctypes.byref(code), int(clear)))
    if code.value != 0:
        layer._workspaces = {}
    return int(code.value)


# ---- between two blocks: norms, gate, residual sum, quantizer -----------------------------

class BlockNormArgs(ctypes.Structure):
    """fmpq_block_norm_args of include/fmpq.h."""
    _fields_ = [("X", _P), ("ldx", _I64), ("residual", _P), ("ldr", _I64), ("gate", _P), ("ldg", _I64), ("gate_tokens", _I64),
                ("post_weight", _P), ("post_bias", _P), ("weight", _P), ("bias", _P), ("R", _P), ("ldo", _I64), ("Y", _P),
                ("ldy", _I64), ("A_packed", _P), ("a_scales", _P), ("M", _I64), ("K", _I32), ("dtype", _I32),
                ("param_dtype", _I32), ("gate_dtype", _I32), ("kind", _I32), ("post_norm", _I32), ("pre_norm", _I32),
                ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class BlockNorm(NamedTuple):
    """What block_norm wrote (None: not asked for)."""
    R: object
    Y: object
    A_packed: object
    a_scales: object


_NORMS = {"rms": 0, "layer": 1}


_pack_block_norm = struct.Struct("@PqPqPqqPPPPPqPqPPqiiiiiiifff").pack    # BlockNormArgs, faster than by its fields


def _vector(v, K: int, what: str, code: int, seen):
    """A contiguous vector [K] on the current GPU, of X's type (code) or fp32, and of the type of those before it (seen).
    Returns its pointer and dtype code."""
    _need(v.dim() == 1 and v.shape[0] == K and (K == 1 or v.stride(0) == 1) and _here(v),
          f"{what} must be a contiguous tensor [K] on the current GPU")
    mine = _dtype_code(v.dtype)
    _need((mine == code or mine == 2) and (seen is None or mine == seen),
          "weights and biases must all be of X's type, or all fp32")
    return v.data_ptr(), mine


@_on_stream
def block_norm(X, residual=None, kind: str = "rms", eps: float = 1e-6, post_norm: bool = False, post_weight=None,
               post_bias=None, gate=None, residual_scale: float = 1.0, pre_norm: bool = True, weight=None, bias=None,
               weight_offset: float = 0.0, layer: "Fp8Layer" = None, R=None, Y=None, A_packed=None,
               a_scales=None) -> BlockNorm:
    """The norms between two blocks, fused with the gate, the residual sum and the E4M3 quantizer, for X [M, K] (fp16
    or bf16): u = X, or its norm (post_norm); r = residual_scale * residual + gate * u; y = norm(r) of the unrounded r
    (pre_norm). kind: "rms" or "layer". gate: [K], or [G, K] with G dividing M, each row for M / G rows of X. Weights
    and biases [K]: all of X's type or all fp32; a norm multiplies by weight_offset + weight.

    Returns (R, Y, A_packed, a_scales). R is r (None where r is X itself and no R is passed). With a layer y comes as the
    codes and scales that fp8_gemm takes for that layer, and as Y only where a Y is passed; without one it comes as Y.
    R may be residual or X, Y may be X or residual. A NaN makes its row's norm NaN, and so does an infinity in a layer norm; in an RMS norm an
    infinity's own channel is NaN and the row's others are 0 times their weight, plus their bias."""
    import torch
    code = _rows16(X, "X")
    M, K = X.shape
    norm = _NORMS.get(kind)
    _need(norm is not None, "kind must be 'rms' or 'layer'")
    _need(post_norm or (post_weight is None and post_bias is None), "post_weight and post_bias need post_norm")
    _need(pre_norm or (weight is None and bias is None and layer is None and Y is None),
          "weight, bias, layer and Y need pre_norm")
    param = None
    w_ptr = b_ptr = pw_ptr = pb_ptr = 0
    if weight is not None:
        w_ptr, param = _vector(weight, K, "weight", code, param)
    if bias is not None:
        b_ptr, param = _vector(bias, K, "bias", code, param)
    if post_weight is not None:
        pw_ptr, param = _vector(post_weight, K, "post_weight", code, param)
    if post_bias is not None:
        pb_ptr, param = _vector(post_bias, K, "post_bias", code, param)
    res_ptr = ldr = gate_ptr = ldg = gate_tokens = gate_code = 0
    if residual is not None:
        _need(_rows16(residual, "residual") == code and residual.shape == X.shape, "residual must be [M, K] of X's type")
        res_ptr, ldr = residual.data_ptr(), _ld(residual)
    if gate is not None:
        rows = gate if gate.dim() == 2 else gate[None]
        groups = rows.shape[0]
        _need(gate.dim() in (1, 2) and _here(gate) and rows.shape[1] == K and (K == 1 or rows.stride(1) == 1) and
              groups >= 1 and M % groups == 0, "gate must be [K], or [G, K] with G dividing M, on the current GPU")
        gate_ptr, gate_code = gate.data_ptr(), _dtype_code(gate.dtype)
        _need(gate_code in (code, 2), "gate must be of X's type or fp32")
        gate_tokens, ldg = M // groups, rows.stride(0) if groups > 1 else K
        _need(ldg >= K, "the rows of a gate must not overlap")
    r_ptr = ldo = y_ptr = ldy = a_ptr = s_ptr = 0
    if R is not None:
        _need(_rows16(R, "R") == code and R.shape == X.shape, "R must be [M, K] of X's type")
        _apart(R, "R", X, residual, gate, post_weight, post_bias, weight, bias, same=(X, residual))
        r_ptr, ldo = R.data_ptr(), _ld(R)
    elif post_norm or residual is not None or gate is not None or not pre_norm:
        R = torch.empty((M, K), dtype=X.dtype, device=X.device)
        r_ptr, ldo = R.data_ptr(), K
    if Y is not None:
        _need(_rows16(Y, "Y") == code and Y.shape == X.shape, "Y must be [M, K] of X's type")
        _apart(Y, "Y", X, residual, gate, post_weight, post_bias, weight, bias, same=(X, residual))
        _apart(Y, "Y (and R)", R)
        y_ptr, ldy = Y.data_ptr(), _ld(Y)
    elif pre_norm and layer is None:
        Y = torch.empty((M, K), dtype=X.dtype, device=X.device)
        y_ptr, ldy = Y.data_ptr(), K
    if layer is not None:
        _need(layer.K == K, "the layer must take K channels")
        if A_packed is None and a_scales is None:
            A_packed, a_scales = layer.activations(M, X.device)
        else:
            if A_packed is None or a_scales is None:
                A, s = layer.activations(M, X.device)
                A_packed, a_scales = A if A_packed is None else A_packed, s if a_scales is None else a_scales
            layer.check_activations(A_packed, a_scales, M)
            for out, what in ((A_packed, "A_packed"), (a_scales, "a_scales")):
                _apart(out, what, X, residual, gate, post_weight, post_bias, weight, bias, R, Y)
        a_ptr, s_ptr = A_packed.data_ptr(), a_scales.data_ptr()
    else:
        _need(A_packed is None and a_scales is None, "A_packed and a_scales need a layer")
    args = _pack_block_norm(X.data_ptr(), _ld(X), res_ptr, ldr, gate_ptr, ldg, gate_tokens, pw_ptr, pb_ptr, w_ptr, b_ptr, r_ptr,
                            ldo, y_ptr, ldy, a_ptr, s_ptr, M, K, code, code if param is None else param, gate_code, norm,
                            bool(post_norm), bool(pre_norm), eps, residual_scale, weight_offset)
    _check("fmpq_block_norm", (_lib or load_library()).fmpq_block_norm(args, _on(X)))
    return BlockNorm(R, Y, A_packed, a_scales)


# ---- routing to experts -------------------------------------------------------------------

_SCORES = {"softmax": 0, "sigmoid": 1}


@_on_stream
def moe_route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
              group_top: int = 1, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None):
    """The top-k experts of each token from the router's logits [T, E] (fp32, fp16 or bf16): ids int32
    [T, k] (by falling key, -1: none) and weights fp32 [T, k]. score: "softmax" or "sigmoid"; bias: fp32
    [E], added for the choice only; groups: keep the top_groups runs of E / groups experts with the
    largest sum of their group_top best keys; renormalize: weights sum to `scale`."""
    import torch
    sigmoid = _SCORES.get(score)
    _need(sigmoid is not None, "score must be 'softmax' or 'sigmoid'")
    _need(logits.dim() == 2 and _here(logits), "logits must be a 2-D tensor on the current GPU")
    T, E = logits.shape
    _need(E <= 1 or logits.stride(1) == 1, "logits must have contiguous rows")
    b_ptr = None
    if bias is not None:
        _need(_here(bias) and bias.dtype == torch.float32 and bias.shape == (E,) and (E == 1 or bias.stride(0) == 1),
              "bias must be a contiguous fp32 tensor [E] on the current GPU")
        b_ptr = bias.data_ptr()
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    else:
        _need(_here(ids) and ids.shape == (T, k) and ids.dtype == torch.int32 and ids.is_contiguous(),
              "ids must be a contiguous int32 tensor [T, k] on the current GPU")
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    else:
        _need(_here(weights) and weights.shape == (T, k) and weights.dtype == torch.float32 and weights.is_contiguous(),
              "weights must be a contiguous fp32 tensor [T, k] on the current GPU")
    _check("moe_route", (_lib or load_library()).moe_route(
        logits.data_ptr(), _dtype_code(logits.dtype), _ld(logits), T, E, k, sigmoid, b_ptr, groups, top_groups, group_top,
        1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), _on(logits)))
    return ids, weights


class MoePlan:
    """The (token, slot) pairs sorted by expert (moe_plan): sizes, the device buffer, and the type of the sums over a
    token's slots (moe_down's dtype)."""

    def __init__(self, T: int, k: int, experts: int, device):
        import torch
        lib = load_library()
        nbytes = int(lib.moe_plan_bytes(T, k, experts))
        if nbytes == 0:
            raise FmpqError("moe_plan_bytes", 2)
        self.T, self.k, self.experts = T, k, experts
        self.dtype = torch.float16
        self.rows = int(lib.moe_rows(T, k, experts))
        self.buffer = torch.empty(nbytes // 4, dtype=torch.int32, device=device)

    @property
    def start(self):
        return self.buffer[:self.experts]

    @property
    def count(self):
        return self.buffer[self.experts:2 * self.experts]

    @property
    def row_of(self):
        return self.buffer[2 * self.experts:2 * self.experts + self.T * self.k].view(self.T, self.k)


@_on_stream
def moe_plan(ids, experts: int, plan=None) -> MoePlan:
    """Sort the pairs of ids (int32 [T, k]) by expert; ids outside [0, experts) belong to none."""
    import torch
    _need(_here(ids) and ids.dim() == 2 and ids.dtype == torch.int32 and ids.is_contiguous(),
          "ids must be a contiguous int32 tensor [T, k] on the current GPU")
    T, k = ids.shape
    plan = MoePlan(T, k, experts, ids.device) if plan is None else plan
    _need((plan.T, plan.k, plan.experts) == (T, k, experts) and _here(plan.buffer), "the plan was made for other sizes, or on another GPU")
    _check("moe_plan", load_library().moe_plan(_ptr(ids), T, k, experts, _ptr(plan.buffer), _stream(None)))
    return plan


@_on_stream
def moe_quantize(layer: Fp8Layer, plan: MoePlan, X, A_packed=None, a_scales=None):
    """Quantize each token of X [T, K] once into its experts' rows."""
    _rows16(X, "X")
    _need(X.shape == (plan.T, layer.K) and plan.experts == layer.experts and _here(plan.buffer), "X must be [T, K], the plan the layer's")
    if A_packed is None or a_scales is None:
        A, s = layer.activations(plan.rows, X.device)
        A_packed, a_scales = A if A_packed is None else A_packed, s if a_scales is None else a_scales
    layer.check_activations(A_packed, a_scales, plan.rows)
    _check("moe_quantize", layer._lib.moe_quantize(layer.handle, _ptr(plan.buffer), plan.T, plan.k, _ptr(X),
                                                   _dtype_code(X.dtype), _ld(X), _ptr(A_packed), _ptr(a_scales),
                                                   _stream(None)))
    return A_packed, a_scales


@_on_stream
def moe_up(layer: Fp8Layer, plan: MoePlan, A_packed, a_scales, W_packed, w_scales, H_packed=None, h_scales=None):
    """SwiGLU of the gated layer's products, quantized: codes uint8 [F / 128, rows, 128] and scales."""
    import torch
    _need(layer.gated and plan.experts == layer.experts and _here(plan.buffer), "moe_up needs a gated layer and its plan")
    layer.check_weights(W_packed, w_scales)
    layer.check_activations(A_packed, a_scales, plan.rows)
    fb = -(-(layer.N // 2) // BLOCK)
    if H_packed is None:
        H_packed = torch.empty((fb, plan.rows, BLOCK), dtype=torch.uint8, device=A_packed.device)
    if h_scales is None:
        h_scales = torch.empty((fb, (plan.rows + 3) // 4 * 4), dtype=torch.float32, device=A_packed.device)
    _need_activations(H_packed, h_scales, fb, plan.rows, "H_packed and h_scales")
    _check("moe_up", layer._lib.moe_up(layer.handle, _ptr(plan.buffer), plan.T, plan.k, _ptr(A_packed), _ptr(a_scales),
                                       _ptr(W_packed), _ptr(w_scales), _ptr(H_packed), _ptr(h_scales), _stream(None)))
    return H_packed, h_scales


@_on_stream
def moe_down(layer: Fp8Layer, plan: MoePlan, A_packed, a_scales, W_packed, w_scales, weights=None, dtype=None, D=None):
    """Every row's product with its expert, times its pair's weight: D [plan.rows, N] in FP32, for moe_combine to sum
    and to round to dtype (fp16 by default). A D that is passed may have 16 bits: each row is then rounded, which halves
    the bytes and costs a rounding a slot."""
    import torch
    _need(plan.experts == layer.experts and not layer.gated and _here(plan.buffer), "moe_down needs a plain layer and its plan")
    layer.check_weights(W_packed, w_scales)
    layer.check_activations(A_packed, a_scales, plan.rows)
    if weights is not None:
        _need(_here(weights) and weights.dtype == torch.float32 and weights.shape == (plan.T, plan.k) and
              weights.is_contiguous(), "weights must be contiguous fp32 [T, k] on the current GPU")
    if D is None:
        D = torch.empty((plan.rows, layer.N), dtype=torch.float32, device=A_packed.device)
    _rows16(D, "D", fp32=True)
    _need(D.shape == (plan.rows, layer.N), "D must be [rows, N]")
    dtype = dtype or (D.dtype if D.dtype != torch.float32 else torch.float16)
    _need(_dtype_code(dtype) < 2 and D.dtype in (torch.float32, dtype), "dtype must be fp16 or bf16, and a 16-bit D of it")
    plan.dtype = dtype
    _check("moe_down", layer._lib.moe_down(layer.handle, _ptr(plan.buffer), plan.T, plan.k, _ptr(weights), _ptr(A_packed),
                                           _ptr(a_scales), _ptr(W_packed), _ptr(w_scales), _ptr(D), _dtype_code(D.dtype),
                                           _ld(D), _stream(None)))
    return D


@_on_stream
def moe_combine(D, plan: MoePlan, Y=None):
    """Y [T, N]: the sum of D's rows of each token, rounded once; of moe_down's dtype (or of a 16-bit D's)."""
    import torch
    code = _rows16(D, "D", fp32=True)
    _need(D.shape[0] == plan.rows and _here(plan.buffer), "D must be [rows, N], the plan on its GPU")
    if Y is None:
        Y = torch.empty((plan.T, D.shape[1]), dtype=plan.dtype if code == 2 else D.dtype, device=D.device)
    y_code = _rows16(Y, "Y")
    _need(Y.shape == (plan.T, D.shape[1]) and (code == 2 or y_code == code), "Y must be [T, N], of a 16-bit D's type")
    sizes = (_ptr(plan.buffer), plan.T, plan.k, plan.experts, D.shape[1])
    if code == 2:
        _check("moe_combine_f32", load_library().moe_combine_f32(_ptr(D), _ld(D), *sizes, _ptr(Y), y_code, _ld(Y), _stream(None)))
    else:
        _check("moe_combine", load_library().moe_combine(_ptr(D), code, _ld(D), *sizes, _ptr(Y), _ld(Y), _stream(None)))
    return Y


@_on_stream
def moe_experts(up: Fp8Layer, down: Fp8Layer, X, ids, weights, W_up, s_up, W_down, s_down):
    """The routed feed-forward on X [T, K]: for each token the sum over its slots of weights[t, j] *
    down(silu(gate(x)) * up(x)) with expert ids[t, j] (-1: none). up: a gated layer [2F, K]; down: [N, F]
    with the same experts. ids and weights as moe_route returns them. Y [T, N] of X's type."""
    import torch
    _need(up.gated and not down.gated and up.experts == down.experts and up.N == 2 * down.K,
          "up must be the gated layer [2F, K] and down the plain layer [N, F] of the same experts")
    code = _rows16(X, "X")
    T, K = X.shape
    _need(_here(ids, weights) and ids.dim() == 2 and ids.dtype == torch.int32 and ids.is_contiguous() and ids.shape[0] == T and
          K == up.K, "ids must be a contiguous int32 tensor [T, k] for X [T, K], ids and weights on the current GPU")
    _need(weights.dtype == torch.float32 and weights.shape == ids.shape and weights.is_contiguous(),
          "weights must be contiguous fp32 [T, k]")
    up.check_weights(W_up, s_up)
    down.check_weights(W_down, s_down)
    k = ids.shape[1]
    sizes = up._workspace_bytes
    nbytes = sizes.get((T, k, down.N))
    if nbytes is None:
        nbytes = sizes[(T, k, down.N)] = int(up._lib.moe_experts_bytes(up._h, down._h, T, k))
        if nbytes == 0:
            del sizes[(T, k, down.N)]
            raise FmpqError("moe_experts", 2)
    scratch = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    Y = torch.empty((T, down.N), dtype=X.dtype, device=X.device)
    _check("moe_experts", up._lib.moe_experts(
        up._h, down._h, X.data_ptr(), code, _ld(X), T, k, ids.data_ptr(), weights.data_ptr(), W_up.data_ptr(),
        s_up.data_ptr(), W_down.data_ptr(), s_down.data_ptr(), Y.data_ptr(), down.N, scratch.data_ptr(), nbytes,
        _on(X)))
    return Y


# ---- layers kept in 16 bits ---------------------------------------------------------------

class W16Layer:
    """Owns a w16_layer*: `experts` weight matrices [N, K] in fp16 or bf16 (one: a linear layer); gated: N = 2F rows, F
    gate rows then F up rows, and outputs act(gate) * up of F columns."""

    def __init__(self, K: int, N: int, dtype, experts: int = 1, gated: bool = False):
        lib = load_library()
        h = ctypes.c_void_p()
        code = _dtype_code(dtype)
        _check("w16_layer_create", lib.w16_layer_create(K, N, experts, int(gated), code, ctypes.byref(h)))
        self._h = h
        self._lib = lib
        self.K, self.N, self.experts, self.gated, self.dtype = K, N, experts, bool(gated), dtype
        self.outputs = N // 2 if gated else N
        self._code = code
        self._w_bytes = int(lib.w16_packed_w_bytes(h))

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.w16_layer_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def packed_w_bytes(self) -> int:
        return self._w_bytes


def w16_device_status(layer: W16Layer, clear: bool = True) -> int:
    """The layer's status word (0, or 5 after a wait that gave up)."""
    code = ctypes.c_int32(0)
    _check("w16_device_status", layer._lib.w16_device_status(layer.handle, ctypes.byref(code), int(clear)))
    return int(code.value)


@_on_stream
def w16_pack_weights(layer: W16Layer, W):
    """Lay out W [experts, N, K] (or [N, K]) of the layer's type, of any strides: a checkpoint that holds [K, N] passes its
    transpose. Returns W_packed u8."""
    import torch
    W3 = W if W.dim() == 3 else W[None]
    _need(W3.shape == (layer.experts, layer.N, layer.K) and W.dtype == layer.dtype and _here(W),
          "W must be [experts, N, K] (or [N, K]) of the layer's type on the current GPU")
    strides = [s if n > 1 else 1 for s, n in zip(W3.stride()[1:], W3.shape[1:])]
    _need(min(strides) >= 1, "W must not be an expanded tensor")
    Wp = torch.empty(layer.packed_w_bytes(), dtype=torch.uint8, device=W.device)
    for e in range(layer.experts):
        _check("w16_pack_weights", layer._lib.w16_pack_weights(layer.handle, e, W3[e].data_ptr(), *strides, Wp.data_ptr(), _on(W)))
    return Wp


def _w16_product(layer, X, W_packed, rows: int, call, workspace_bytes, bias, activation, residual, dtype, Y, inputs=()):
    """What the three products share: checks, epilogue, output and workspace; then call(Y's pointer, code and stride, epilogue,
    workspace's pointer and bytes)."""
    import torch
    _need(_here(W_packed) and W_packed.element_size() == 1 and W_packed.is_contiguous() and W_packed.numel() == layer._w_bytes,
          "W_packed must be this layer's (w16_pack_weights)")
    shape = (rows, layer.outputs)
    code = layer._code if Y is None and dtype is None else _dtype_code(dtype if Y is None else Y.dtype)
    _need(code == layer._code or code == 2, "the output's type must be the layer's or fp32")
    epilogue = None
    if bias is not None or activation is not None or residual is not None:
        if bias is not None and bias.dim() == 1 and layer.experts == 1:
            bias = bias[None]
        epilogue = _epilogue(bias, activation, residual, shape, (layer.experts, layer.N), code, Y)
    if Y is None:
        Y = torch.empty(shape, dtype=layer.dtype if dtype is None else dtype, device=X.device)
        ldy = layer.outputs
    else:
        _need(_rows16(Y, "Y", fp32=True) == code and Y.shape == shape, "Y must be [rows, N] ([rows, N / 2] of a gated layer)")
        _apart(Y, "Y", X, *inputs)
        ldy = _ld(Y)
    nbytes = workspace_bytes()
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=X.device) if nbytes else None
    call(Y.data_ptr(), code, ldy, epilogue, workspace.data_ptr() if nbytes else None, nbytes)
    return Y


def _w16_rows(layer, X) -> int:
    """Row stride of X [rows, K] of the layer's type."""
    _need(_rows16(X, "X") == layer._code and X.shape[1] == layer.K, "X must be [rows, K] of the layer's type")
    return _ld(X)


@_on_stream
def w16_gemm(layer: W16Layer, X, W_packed, bias=None, activation=None, residual=None, dtype=None, Y=None):
    """Y [M, N] (a gated layer: [M, N / 2]) of X [M, K] in the layer's type, or in fp32 (dtype, or a Y that is passed):
    act(X W^T + bias) + residual; gated: act(gate + bias) * (up + bias) + residual. bias [N] or [1, N], of Y's type or fp32;
    activation as fp8_gemm takes it; residual of Y's shape and type, which may be Y."""
    _need(layer.experts == 1, "w16_gemm takes a layer of one matrix (w16_grouped_gemm, w16_experts_gemm: experts)")
    ld, M, lib, x_ptr = _w16_rows(layer, X), X.shape[0], layer._lib, X.data_ptr()

    def call(y_ptr, code, ldy, epilogue, ws, nbytes):
        _check("w16_gemm", lib.w16_gemm(layer._h, x_ptr, ld, M, W_packed.data_ptr(), epilogue, y_ptr, code, ldy, ws, nbytes, _on(X)))

    return _w16_product(layer, X, W_packed, M, call, lambda: _w16_workspace(layer, x_ptr, ld, M), bias, activation, residual, dtype, Y)


def _w16_workspace(layer, x_ptr: int, ld: int, rows: int) -> int:
    return int(layer._lib.w16_workspace_bytes(layer._h, x_ptr, ld, rows)) if ld % 8 or x_ptr % 16 else 0


@_on_stream
def w16_grouped_gemm(layer: W16Layer, X, offsets, W_packed, bias=None, activation=None, residual=None, row_weight=None,
                     dtype=None, Y=None):
    """As w16_gemm, the rows of X in groups with a matrix each: group e is rows offsets[e] to offsets[e + 1] - 1 (int32
    [experts + 1] on the GPU, cut to X's rows). bias [experts, N]; row_weight fp32 [rows] scales a row's outputs before the
    residual. Rows of no group are not written."""
    import torch
    ld, rows, lib, x_ptr = _w16_rows(layer, X), X.shape[0], layer._lib, X.data_ptr()
    _need(_here(offsets) and offsets.dtype == torch.int32 and offsets.shape == (layer.experts + 1,) and offsets.is_contiguous(),
          "offsets must be contiguous int32 [experts + 1] on the current GPU")
    _need(row_weight is None or (_here(row_weight) and row_weight.dtype == torch.float32 and row_weight.shape == (rows,) and
                                 row_weight.is_contiguous()), "row_weight must be contiguous fp32 [rows] on the current GPU")
    r_ptr = row_weight.data_ptr() if row_weight is not None else None

    def call(y_ptr, code, ldy, epilogue, ws, nbytes):
        _check("w16_grouped_gemm", lib.w16_grouped_gemm(layer._h, x_ptr, ld, rows, offsets.data_ptr(), W_packed.data_ptr(), epilogue,
                                                        r_ptr, y_ptr, code, ldy, ws, nbytes, _on(X)))

    return _w16_product(layer, X, W_packed, rows, call, lambda: _w16_workspace(layer, x_ptr, ld, rows), bias, activation, residual, dtype,
                        Y, (row_weight,))


@_on_stream
def w16_experts_gemm(layer: W16Layer, plan: MoePlan, X, W_packed, weights=None, bias=None, activation=None, residual=None,
                     dtype=None, Y=None):
    """The rows of a plan, each with its expert's matrix: Y [plan.rows, N] ([plan.rows, N / 2] of a gated layer), as
    w16_grouped_gemm. X [T, K]: each token goes to its experts' rows; or X [plan.rows, K], such a product's output. weights
    fp32 [T, k] scale each row's outputs by its pair's. Rows of no pair are not written. With dtype=torch.float32 it makes the D
    that moe_combine sums (into X's type)."""
    import torch
    _need(plan.experts == layer.experts and _here(plan.buffer), "the plan must be of this layer's experts, on the current GPU")
    ld, lib, x_ptr = _w16_rows(layer, X), layer._lib, X.data_ptr()
    gather = X.shape[0] != plan.rows     # (a plan has more rows than tokens)
    _need(not gather or X.shape[0] == plan.T, "X must be [T, K] or [plan.rows, K]")
    _need(weights is None or (_here(weights) and weights.dtype == torch.float32 and weights.shape == (plan.T, plan.k) and
                              weights.is_contiguous()), "weights must be contiguous fp32 [T, k] on the current GPU")
    w_ptr = weights.data_ptr() if weights is not None else None

    def need():
        return int(lib.w16_experts_workspace_bytes(layer._h, x_ptr, ld, plan.T, plan.k, int(gather)))

    def call(y_ptr, code, ldy, epilogue, ws, nbytes):
        _check("w16_experts_gemm", lib.w16_experts_gemm(
            layer._h, plan.buffer.data_ptr(), plan.T, plan.k, x_ptr, ld, int(gather), W_packed.data_ptr(), epilogue, w_ptr, y_ptr,
            code, ldy, ws, nbytes, _on(X)))

    Y = _w16_product(layer, X, W_packed, plan.rows, call, need, bias, activation, residual, dtype, Y, (weights,))
    plan.dtype = layer.dtype
    return Y
