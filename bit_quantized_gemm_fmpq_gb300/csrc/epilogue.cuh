// What a product does to its FP32 sums before it rounds them: bias, activation, residual.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.h"

namespace fmpq {
namespace epi {

// The activations in FP32. Exponentials and quotients good to 2 of their last places; gelu through erfc, whose
// relative error stays small where 1 + erf cancels. An argument of -inf gives NaN but for relu, as inf * 0 does.
__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case kActRelu: return v < 0.0f ? 0.0f : v;
        case kActSilu: return __fdividef(v, 1.0f + expf(-v));
        case kActGelu: return 0.5f * v * erfcf(v * -0.70710678f);
        case kActGeluTanh:   // 0.5 v (1 + tanh(u)) = v / (1 + e^-2u)
            return __fdividef(v, 1.0f + expf(v * fmaf(v * v, -2.0f * 0.79788456f * 0.044715f, -2.0f * 0.79788456f)));
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
