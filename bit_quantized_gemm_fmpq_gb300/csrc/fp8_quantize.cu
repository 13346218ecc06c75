// E4M3 activations and weights with a scale for each block of 128 (sm_103a).
//
//   s = fl32(max|x| / 448),  q = e4m3(fl32(x / s)),  x ~ q * s     (s = 0: every code is 0)
//
// over 128 channels of a token, or 128 x 128 of a weight matrix. Division and conversion round to
// nearest, so the codes do not depend on how the work is split.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fmpq_device.cuh"
#include "fp8_internal.h"

namespace fmpq {
namespace {

constexpr float kQMax = 448.0f;

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
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    // E4M3 -> fp16 is exact
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// The codes of eight values, e4m3(fl32(v / s)). Products with s's reciprocal, made 2^-21 smaller and larger,
// enclose the quotient (the reciprocal is good to 2^-23, each product rounds by 2^-24): where both round to the same
// code it is the quotient's, and elsewhere (one value in 2^17) the division decides.
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float s) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const float lo = inv * (1.0f - 4.76837158e-7f), hi = inv * (1.0f + 4.76837158e-7f);
    uint2 code, other;
    code.x = e4m3x2(v[0] * lo, v[1] * lo) | (e4m3x2(v[2] * lo, v[3] * lo) << 16);
    code.y = e4m3x2(v[4] * lo, v[5] * lo) | (e4m3x2(v[6] * lo, v[7] * lo) << 16);
    other.x = e4m3x2(v[0] * hi, v[1] * hi) | (e4m3x2(v[2] * hi, v[3] * hi) << 16);
    other.y = e4m3x2(v[4] * hi, v[5] * hi) | (e4m3x2(v[6] * hi, v[7] * hi) << 16);
    if (s >= 1.17549435e-38f && s <= 1e37f && code.x == other.x && code.y == other.y) return code;
    if (!(s > 0.0f)) return make_uint2(0u, 0u);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], s);
    return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16), e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}

// A warp takes 256 channels of a token, 16 lanes a block, 8 channels a lane (one 16-byte load, 8 bytes
// of codes); blockIdx.y chooses the channels, so that a CTA's stores of a block's codes (128 bytes a
// row) and scales are contiguous. kRows tokens a warp are in flight. 4096 x 8192 bf16: 29.4 us, 102 MB = 3.5 TB/s, 51%
// of the copy rate: its instructions bound it. With 8 rounded divisions a lane it took 32.6, with one token in
// flight or with four 31.3.
template <typename T, bool kVec, int kRows>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ X, int64_t ldx, int64_t M, int K, int nb,
                                                       const int32_t* __restrict__ positions, int slots, int64_t rows,
                                                       int64_t sstride, uint8_t* __restrict__ A,
                                                       float* __restrict__ scales) {
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    dev::pdl_wait();
    dev::pdl_launch_dependents();
    const int b = static_cast<int>(blockIdx.y) * 2 + half;
    const int k0 = b * 128 + l * 8;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * kRows;
    for (int64_t m0 = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kRows; m0 < M; m0 += step) {
        const T* x = X + m0 * ldx + k0;
        const bool whole = kVec && k0 + 8 <= K;
        uint4 raw[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (whole && m0 + i < M) raw[i] = __ldcs(reinterpret_cast<const uint4*>(x + i * ldx));
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t m = m0 + i;
            if (m >= M) break;
            float v[8];
            if (whole) {
                const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 f = unpack2(u[c], x);
                    v[2 * c] = f.x;
                    v[2 * c + 1] = f.y;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = k0 + c < K ? load_as_float(x + i * ldx + c) : 0.0f;
            }
            // as bits, NaN is above every number: a block with one gets the scale NaN
            uint32_t amax = 0u;
#pragma unroll
            for (int c = 0; c < 8; ++c) amax = max(amax, __float_as_uint(fabsf(v[c])));
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
            const float s = __fdiv_rn(__uint_as_float(amax), kQMax);
            const uint2 code = codes_of(v, s);
            if (b >= nb) continue;
            for (int j = 0; j < slots; ++j) {
                const int64_t r = positions != nullptr ? positions[m * slots + j] : m;
                if (r < 0) continue;
                uint8_t* row = A + (static_cast<int64_t>(b) * rows + r) * 128;
                *reinterpret_cast<uint2*>(row + (((l >> 1) ^ static_cast<int>(r & 7)) << 4) + (l & 1) * 8) = code;
                if (l == 0) scales[b * sstride + r] = s;
            }
        }
    }
}

// One CTA a 128 x 128 weight block: its absmax, then its codes into the packed tiles.
template <typename T>
__global__ void __launch_bounds__(256) pack_weights_kernel(const T* __restrict__ W, int64_t ldw, int K, int N, int gated,
                                                           int nb, uint8_t* __restrict__ Wp, float* __restrict__ scales) {
    __shared__ float red[8];
    const int b = blockIdx.x, sr = blockIdx.y;
    const int F = N / 2, fb = (F + 127) / 128;
    // the weight rows [n0, n1) of this scale row
    int n0 = sr * 128, n1 = min(n0 + 128, N);
    if (gated) {
        n0 = sr < fb ? sr * 128 : F + (sr - fb) * 128;
        n1 = min(n0 + 128, sr < fb ? F : N);
    }
    const int k = b * 128 + (threadIdx.x & 127);
    float amax = 0.0f;
    for (int n = n0 + (threadIdx.x >> 7); n < n1; n += 2)
        if (k < K) amax = fmaxf(amax, fabsf(load_as_float(W + static_cast<int64_t>(n) * ldw + k)));
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, red[i]);
    const float s = __fdiv_rn(amax, kQMax);
    if (threadIdx.x == 0) scales[static_cast<int64_t>(sr) * nb + b] = s;
    // the packed rows of the pair tile that hold these weight rows
    const int pair = gated ? (sr < fb ? sr : sr - fb) : sr >> 1;
    for (int p = threadIdx.x >> 7; p < 256; p += 2) {
        const int t = 2 * pair + (p >> 7), n = fp8_source_row(t, p & 127, N, gated);
        const bool mine = n >= n0 && n < n1;
        // rows past the last one belong to no scale row: the first block of the pair clears them
        const bool pad = n < 0 && (gated ? sr < fb : (sr & 1) == 0);
        if (!mine && !pad) continue;
        float q = 0.0f;
        if (mine && k < K) {
            const float w = load_as_float(W + static_cast<int64_t>(n) * ldw + k);
            if (s > 0.0f) q = __fdiv_rn(w, s);
            else if (isnan(w)) q = w;   // the block's other weights are 0, or NaN too
        }
        const int r = p & 127, kk = threadIdx.x & 127;
        Wp[(static_cast<int64_t>(t) * nb + b) * kTileBytes + r * 128 + (((kk >> 4) ^ (r & 7)) << 4) + (kk & 15)] =
            static_cast<uint8_t>(e4m3x2(q, 0.0f) & 0xFFu);
    }
}

// Codes [N][ldw] of an E4M3 checkpoint into the packed tiles, 16 bytes a thread.
__global__ void __launch_bounds__(256) pack_codes_kernel(const uint8_t* __restrict__ codes, int64_t ldw, int K, int N,
                                                         int gated, int nb, int tiles, uint8_t* __restrict__ Wp) {
    const int64_t chunks = static_cast<int64_t>(tiles) * nb * 1024;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < chunks;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int c = static_cast<int>(i & 7), r = static_cast<int>((i >> 3) & 127);
        const int64_t tb = i >> 10;
        const int b = static_cast<int>(tb % nb), t = static_cast<int>(tb / nb);
        const int n = fp8_source_row(t, r, N, gated);
        const int k = b * 128 + ((c ^ (r & 7)) << 4);
        uint4 out = make_uint4(0u, 0u, 0u, 0u);
        if (n >= 0) {
            const uint8_t* src = codes + static_cast<int64_t>(n) * ldw + k;
            if (k + 16 <= K && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
                out = *reinterpret_cast<const uint4*>(src);
            } else {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (k + j < K) w[j >> 2] |= static_cast<uint32_t>(src[j]) << (8 * (j & 3));
                out = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        reinterpret_cast<uint4*>(Wp)[i] = out;
    }
}

__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t* __restrict__ Wp, const float* __restrict__ scales,
                                                     int K, int N, int gated, int nb, int tiles, float* __restrict__ W) {
    const int64_t n_codes = static_cast<int64_t>(tiles) * nb * kTileBytes;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n_codes;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int byte = static_cast<int>(i & 15), c = static_cast<int>((i >> 4) & 7), r = static_cast<int>((i >> 7) & 127);
        const int64_t tb = i >> 14;
        const int b = static_cast<int>(tb % nb), t = static_cast<int>(tb / nb);
        const int n = fp8_source_row(t, r, N, gated), k = b * 128 + ((c ^ (r & 7)) << 4) + byte;
        if (n >= 0 && k < K)
            W[static_cast<int64_t>(n) * K + k] =
                e4m3_value(Wp[i]) * scales[static_cast<int64_t>(fp8_scale_row(n, N, gated)) * nb + b];
    }
}

template <typename T>
cudaError_t quantize_as(const void* X, int64_t ldx, int64_t M, int K, const int32_t* positions, int slots, int64_t rows,
                        void* A, float* scales, int num_sms, bool pdl, cudaStream_t stream) {
    const int nb = (K + 127) / 128;
    const int pairs = (nb + 1) / 2;
    const bool vec = ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(X) & 15u) == 0;
    // two tokens a warp once every warp has several: 2048 x 4096 9.1 against 9.7 us, 1024 x 4096 6.0 either way
    const bool deep = vec && M * pairs >= num_sms * 128LL;
    const int64_t per = deep ? 8 * 2 : 8, ctas = (M + per - 1) / per, most = (num_sms * 64LL + pairs - 1) / pairs;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most), static_cast<unsigned>(pairs));
    auto fn = !vec ? quantize_kernel<T, false, 1> : deep ? quantize_kernel<T, true, 2> : quantize_kernel<T, true, 1>;
    return launch_after(fn, grid, 256, 0, pdl, stream, static_cast<const T*>(X), ldx, M, K, nb,
                        positions, positions != nullptr ? slots : 1, rows, scale_stride(rows), static_cast<uint8_t*>(A), scales);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* X, int dtype, int64_t ldx, int64_t M, int K, const int32_t* positions,
                                int slots, int64_t rows, void* A, float* scales, int num_sms, bool pdl, cudaStream_t stream) {
    return dtype == kF16 ? quantize_as<__half>(X, ldx, M, K, positions, slots, rows, A, scales, num_sms, pdl, stream)
                         : quantize_as<__nv_bfloat16>(X, ldx, M, K, positions, slots, rows, A, scales, num_sms, pdl, stream);
}

cudaError_t launch_fp8_pack_weights(const fp8_layer& L, int expert, const void* W, int dtype, int64_t ldw, void* Wp,
                                    float* scales, cudaStream_t stream) {
    uint8_t* out = static_cast<uint8_t*>(Wp) + static_cast<int64_t>(expert) * L.pairs * 2 * L.nb * kTileBytes;
    float* s = scales + static_cast<int64_t>(expert) * L.scale_rows * L.nb;
    const dim3 grid(L.nb, L.scale_rows);
    if (dtype == kF16)
        pack_weights_kernel<<<grid, 256, 0, stream>>>(static_cast<const __half*>(W), ldw, L.K, L.N, L.gated, L.nb, out, s);
    else
        pack_weights_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(W), ldw, L.K, L.N, L.gated, L.nb,
                                                      out, s);
    return cudaGetLastError();
}

cudaError_t launch_fp8_pack_codes(const fp8_layer& L, int expert, const void* codes, int64_t ldw, void* Wp,
                                  cudaStream_t stream) {
    uint8_t* out = static_cast<uint8_t*>(Wp) + static_cast<int64_t>(expert) * L.pairs * 2 * L.nb * kTileBytes;
    const int64_t ctas = static_cast<int64_t>(L.pairs) * 2 * L.nb * 4;
    pack_codes_kernel<<<static_cast<int>(ctas < L.num_sms * 32LL ? ctas : L.num_sms * 32LL), 256, 0, stream>>>(
        static_cast<const uint8_t*>(codes), ldw, L.K, L.N, L.gated, L.nb, L.pairs * 2, out);
    return cudaGetLastError();
}

cudaError_t launch_fp8_unpack(const fp8_layer& L, int expert, const void* Wp, const float* scales, float* W,
                              cudaStream_t stream) {
    const uint8_t* in = static_cast<const uint8_t*>(Wp) + static_cast<int64_t>(expert) * L.pairs * 2 * L.nb * kTileBytes;
    unpack_kernel<<<L.num_sms * 16, 256, 0, stream>>>(in, scales + static_cast<int64_t>(expert) * L.scale_rows * L.nb, L.K,
                                                      L.N, L.gated, L.nb, L.pairs * 2, W);
    return cudaGetLastError();
}

}  // namespace fmpq
