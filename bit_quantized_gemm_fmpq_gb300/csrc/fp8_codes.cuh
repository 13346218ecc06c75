// 16-bit values to floats, and floats to E4M3 codes: what the kernels that quantize share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fmpq_device.cuh"

namespace fmpq {
namespace {

constexpr float kQMax = 448.0f;   // the largest E4M3 value

__device__ __forceinline__ float load_as_float(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float load_as_float(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float2 unpack2(uint32_t v, const __half*) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ float2 unpack2(uint32_t v, const __nv_bfloat16*) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
// two values to two E4M3 bytes (lo in bits 0-7), to nearest, at most +-448
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// The largest of three magnitudes; NaN if one is.
__device__ __forceinline__ float most3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// The scale of a block of 128 channels from the eight values of each lane of a half warp (every lane calls it): NaN if one is.
__device__ __forceinline__ float scale_of(const float (&v)[8]) {
    const float mine = most3(most3(v[0], v[1], v[2]), most3(v[3], v[4], v[5]), most3(v[6], v[7], 0.0f));
    uint32_t amax = __float_as_uint(mine);   // as bits, NaN is above every number
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    return __fdiv_rn(__uint_as_float(amax), kQMax);
}
// The codes of eight values, e4m3(fl32(v / s)). Products with s's reciprocal, made 2^-21 smaller and larger,
// enclose the quotient (the reciprocal is good to 2^-23, each product rounds by 2^-24): where both round to the same
// code it is the quotient's, and elsewhere (one value in 2^17) the division decides.
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float s) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const float lo = inv * (1.0f - 4.76837158e-7f), hi = inv * (1.0f + 4.76837158e-7f);
    auto codes = [&](float f) {
        const float2 w = make_float2(f, f);
        const float2 a = dev::fmul2(make_float2(v[0], v[1]), w), b = dev::fmul2(make_float2(v[2], v[3]), w);
        const float2 c = dev::fmul2(make_float2(v[4], v[5]), w), d = dev::fmul2(make_float2(v[6], v[7]), w);
        return make_uint2(e4m3x2(a.x, a.y) | (e4m3x2(b.x, b.y) << 16), e4m3x2(c.x, c.y) | (e4m3x2(d.x, d.y) << 16));
    };
    const uint2 code = codes(lo), other = codes(hi);
    if (s >= 1.17549435e-38f && s <= 1e37f && code.x == other.x && code.y == other.y) return code;
    if (!(s > 0.0f)) return make_uint2(0u, 0u);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], s);
    return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16), e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}

}  // namespace
}  // namespace fmpq
