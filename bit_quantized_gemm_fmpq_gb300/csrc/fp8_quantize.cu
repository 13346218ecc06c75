// E4M3 activations and weights with a scale for each block of 128 (sm_103a).
//
//   s = fl32(max|x| / 448),  q = e4m3(fl32(x / s)),  x ~ q * s     (s = 0: every code is 0)
//
// over 128 channels of a token, or 128 x 128 of a weight matrix. Division and conversion round to
// nearest, so the codes do not depend on how the work is split.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fmpq_device.cuh"
#include "fp8_codes.cuh"
#include "fp8_internal.h"

namespace fmpq {
namespace {

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    // E4M3 -> fp16 is exact
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// A warp takes 256 channels of a token, 16 lanes a block, 8 channels a lane (one 16-byte load, 8 bytes
// of codes); blockIdx.y chooses the channels, so that a CTA's stores of a block's codes (128 bytes a
// row) and scales are contiguous. kRows tokens a warp are in flight. 4096 x 8192 bf16: 27.4 us, 102 MB = 3.7 TB/s, 55%
// of the copy rate (4096 x 28672: 83 us, 63%): its instructions bound it. With one form for dense and routed tokens, and maxima of two values,
// it took 33 on the same day (100), with 8 rounded divisions a lane, one token in flight or four 2 to 3 us more still.
template <typename T, bool kVec, int kRows, bool kRouted>
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
            const float s = scale_of(v);
            const uint2 code = codes_of(v, s);
            if (b >= nb) continue;
            auto put = [&](int64_t r) {
                uint8_t* row = A + (static_cast<int64_t>(b) * rows + r) * 128;
                *reinterpret_cast<uint2*>(row + (((l >> 1) ^ static_cast<int>(r & 7)) << 4) + (l & 1) * 8) = code;
                if (l == 0) scales[b * sstride + r] = s;
            };
            if constexpr (!kRouted) {
                put(m);
            } else {
                for (int j = 0; j < slots; ++j) {
                    const int64_t r = positions[m * slots + j];
                    if (r >= 0) put(r);
                }
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
    auto fn = positions != nullptr ? (!vec ? quantize_kernel<T, false, 1, true> : deep ? quantize_kernel<T, true, 2, true> : quantize_kernel<T, true, 1, true>)
                                   : (!vec ? quantize_kernel<T, false, 1, false> : deep ? quantize_kernel<T, true, 2, false> : quantize_kernel<T, true, 1, false>);
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
