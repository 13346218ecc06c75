// What a product does to its FP32 sums before it rounds them: bias, activation, residual.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.h"

namespace fmpq {
namespace epi {

__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// v Phi(v) = max(v, 0) - |v| (1 - Phi(|v|)), and 1 - Phi(a) = e^(-a^2 / 2) G(a): nothing cancels, so the relative error is that of the
// factors. G(a) = erfcx(a / sqrt 2) / 2 as t times a polynomial of degree 8 in t = 1 / (1 + 0.27 a), good to 3.9e-8 relative over
// [0, 20] with these constants (4e-7 evaluated in FP32; tests/test_activations.py); beyond 20 the product is 0 in any case. erfcf takes three times the instructions: 515 tokens
// x 4004 outputs of an E4M3 product 29.5 us, in this form 20.7.
__device__ __forceinline__ float gelu(float v) {
    const float a = fminf(fabsf(v), 20.0f), t = reciprocal_fast(fmaf(a, 0.27f, 1.0f));
    float g = 0.029064413f;
    g = fmaf(g, t, -0.12700377f);
    g = fmaf(g, t, 0.17089249f);
    g = fmaf(g, t, -0.070522867f);
    g = fmaf(g, t, 0.10876805f);
    g = fmaf(g, t, 0.071631014f);
    g = fmaf(g, t, 0.10192257f);
    g = fmaf(g, t, 0.10752644f);
    g = fmaf(g, t, 0.10772167f);
    const float tail = g * t * exp2_fast(a * a * -0.72134752f);
    return fmaf(-a, tail, fmaf(0.5f, fabsf(v), 0.5f * v));   // (0.5 |v| + 0.5 v: max(v, 0) that keeps NaN)
}
// The activations in FP32, off by fewer than |v| + 8 steps of 2^-23 of the value (v^2 + 8 gelu, 3 |v| + |v|^3 / 4 + 8 gelu_tanh):
// what the argument's rounding and the hardware's exponential cost. Values below 1.1e-36 in magnitude may come out as 0 (the quotient by more than
// 2^126 is). An argument of -inf gives NaN but for relu, as inf * 0 does.
__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case kActRelu: return v < 0.0f ? 0.0f : v;
        case kActSilu: return v * reciprocal_fast(1.0f + exp2_fast(v * -1.44269504f));
        case kActGelu: return gelu(v);
        case kActGeluTanh:   // 0.5 v (1 + tanh(u)) = v / (1 + e^-2u)
            return v * reciprocal_fast(1.0f + exp2_fast(v * fmaf(v * v, -2.0f * 0.79788456f * 0.044715f * 1.44269504f,
                                                                 -2.0f * 0.79788456f * 1.44269504f)));
        default: return v;
    }
}

__device__ __forceinline__ float value16(uint16_t v, bool bf16) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ float2 values16(uint32_t v, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// bias[n], in FP32 or the outputs' type
__device__ __forceinline__ float bias_at(const Epilogue& e, int64_t n, bool bf16) {
    if (e.bias == nullptr) return 0.0f;
    if (e.bias_f32) return __ldg(static_cast<const float*>(e.bias) + n);
    return value16(__ldg(static_cast<const uint16_t*>(e.bias) + n), bf16);
}

}  // namespace epi
}  // namespace fmpq
