// The norms between two blocks of a transformer, fused with the gate, the residual sum and the E4M3 quantizer (sm_103a):
//
//   u = X, or norm(X; post_weight, post_bias)           the norm after a block
//   r = residual_scale * residual + gate * u            rounded once, where it is written
//   y = norm(r; weight, bias), of the unrounded r       the norm before the next block: 16 bits, or E4M3 codes with a
//                                                       scale for each token and 128 channels
//   norm(v; w, b) = v / sqrt(mean(v^2) + eps) * (offset + w) + b        (a layer norm: of v - mean(v))
//
// Everything between the reads of X and residual and the writes is FP32. A row is read once and kept in the
// registers of one CTA (8 channels a vector, kV vectors a thread); a layer norm's variance is the mean of the squared
// differences, a second reduction over those registers.
#include "fmpq_device.cuh"
#include "fp8_codes.cuh"
#include "fp8_internal.h"

namespace fmpq {
namespace {

// ---------------------------------------------------------------- eight values of a row or a vector

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float2 f = unpack2(w[c], static_cast<const T*>(nullptr));
        v[2 * c] = f.x;
        v[2 * c + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, const __half*) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, const __nv_bfloat16*) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store1(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Channels k .. k + 7 of a row, those past K as 0.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* row, int k, int K, float (&v)[8]) {
    if (kVec && k + 8 <= K) {
        unpack8<T>(*reinterpret_cast<const uint4*>(row + k), v);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = k + c < K ? load_as_float(row + k + c) : 0.0f;
    }
}
template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* row, int k, int K, const float (&v)[8]) {
    if (kVec && k + 8 <= K) {
        const T* t = nullptr;
        *reinterpret_cast<uint4*>(row + k) =
            make_uint4(pack2(v[0], v[1], t), pack2(v[2], v[3], t), pack2(v[4], v[5], t), pack2(v[6], v[7], t));
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (k + c < K) store1(row + k + c, v[c]);
    }
}
// The same of a weight, bias or gate: of X's type, or FP32.
template <typename T, bool kVec>
__device__ __forceinline__ void param8(const void* p, int fp32, int64_t first, int k, int K, float (&v)[8]) {
    if (!fp32) {
        load8<T, kVec>(static_cast<const T*>(p) + first, k, K, v);
        return;
    }
    const float* f = static_cast<const float*>(p) + first + k;
    if (kVec && k + 8 <= K) {
        const float4 a = *reinterpret_cast<const float4*>(f), b = *reinterpret_cast<const float4*>(f + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = k + c < K ? f[c] : 0.0f;
    }
}

// ---------------------------------------------------------------- sums over a row

struct Sums {
    float part[2][32];
};

// The sum over the CTA's threads, in each of them. Two buffers in turn: whoever writes one again has passed the
// barrier behind which the others had read it.
__device__ __forceinline__ float row_sum(float v, Sums& s, int& turn) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    const int warps = static_cast<int>(blockDim.x) >> 5;
    if (warps == 1) return v;
    float* part = s.part[turn];
    turn ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// ---------------------------------------------------------------- one step of a vector of eight

template <typename T, bool kVec>
__device__ __forceinline__ void scale8(const BlockNormArgs& p, float (&v)[8], float mean, float inv, const void* w,
                                       const void* b, int k) {
    float t[8];
    if (w != nullptr) {
        param8<T, kVec>(w, p.param_f32, 0, k, p.K, t);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = (v[c] - mean) * inv * (p.weight_offset + t[c]);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = (v[c] - mean) * inv;
    }
    if (b != nullptr) {
        param8<T, kVec>(b, p.param_f32, 0, k, p.K, t);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] += t[c];
    }
}

// u to r; residual already read.
template <typename T, bool kVec>
__device__ __forceinline__ void join8(const BlockNormArgs& p, float (&v)[8], const float (&res)[8], int64_t gate_row, int k) {
    if (p.gate != nullptr) {
        float t[8];
        param8<T, kVec>(p.gate, p.gate_f32, gate_row, k, p.K, t);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] *= t[c];
    }
    if (p.residual != nullptr)
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = fmaf(p.residual_scale, res[c], v[c]);
}

// y to memory: 16 bits, and codes (16 lanes of a half warp hold a block of 128; every lane calls it).
template <typename T, bool kVec>
__device__ __forceinline__ void put8(const BlockNormArgs& p, int64_t m, int k, const float (&v)[8]) {
    if (p.Y != nullptr && k < p.K) store8<T, kVec>(static_cast<T*>(p.Y) + m * p.ldy, k, p.K, v);
    if (p.A == nullptr) return;
    uint32_t amax = 0u;   // as bits, NaN is above every number
#pragma unroll
    for (int c = 0; c < 8; ++c) amax = max(amax, k + c < p.K ? __float_as_uint(fabsf(v[c])) : 0u);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    const int b = k >> 7;
    if (b >= p.nb) return;
    float q[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) q[c] = k + c < p.K ? v[c] : 0.0f;
    const float s = __fdiv_rn(__uint_as_float(amax), kQMax);
    const uint2 code = codes_of(q, s);
    const int l = (k >> 3) & 15;
    uint8_t* row = p.A + (static_cast<int64_t>(b) * p.M + m) * 128;
    *reinterpret_cast<uint2*>(row + (((l >> 1) ^ static_cast<int>(m & 7)) << 4) + (l & 1) * 8) = code;
    if (l == 0) p.a_scales[b * p.sstride + m] = s;
}

// mean and 1 / sqrt(mean square + eps) of the CTA's row from its registers.
template <int kV>
__device__ __forceinline__ void statistics(const BlockNormArgs& p, const float (&v)[kV][8], Sums& s, int& turn, float& mean,
                                           float& inv) {
    mean = 0.0f;
    const float count = static_cast<float>(p.K);
    if (p.layer_norm) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int c = 0; c < 8; ++c) sum += v[i][c];
        mean = row_sum(sum, s, turn) / count;
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int k = (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float d = v[i][c] - mean;   // (values past K are 0, and do not count)
            if (!p.layer_norm || k + c < p.K) sq = fmaf(d, d, sq);
        }
    }
    inv = __frsqrt_rn(row_sum(sq, s, turn) / count + p.eps);
}

// One CTA a row, kV vectors of 8 channels a thread: blockDim.x * 8 * kV >= nb * 128.
template <typename T, bool kVec, int kV>
__global__ void __launch_bounds__(kV == 1 ? 1024 : 512) block_norm_kernel(const BlockNormArgs p) {
    __shared__ Sums sums;
    int turn = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + m * p.ldx;
        const T* res = static_cast<const T*>(p.residual) + m * p.ldr;
        const int64_t gate_row = p.gate != nullptr ? m / p.gate_tokens * p.ldg : 0;
        float v[kV][8], add[kV][8];
        auto channel = [&](int i) { return (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8; };
#pragma unroll
        for (int i = 0; i < kV; ++i) load8<T, kVec>(x, channel(i), p.K, v[i]);
        if (p.residual != nullptr)
#pragma unroll
            for (int i = 0; i < kV; ++i) load8<T, kVec>(res, channel(i), p.K, add[i]);
        float mean, inv;
        if (p.post_norm) {
            statistics(p, v, sums, turn, mean, inv);
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (channel(i) < p.K) scale8<T, kVec>(p, v[i], mean, inv, p.post_weight, p.post_bias, channel(i));
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (channel(i) >= p.K) continue;
            join8<T, kVec>(p, v[i], add[i], gate_row, channel(i));
            // (past K: a post norm's value of 0 is not 0)
            if (channel(i) + 8 > p.K)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (channel(i) + c >= p.K) v[i][c] = 0.0f;
            if (p.R != nullptr) store8<T, kVec>(static_cast<T*>(p.R) + m * p.ldo, channel(i), p.K, v[i]);
        }
        if (!p.pre_norm) continue;
        statistics(p, v, sums, turn, mean, inv);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (channel(i) < p.K) scale8<T, kVec>(p, v[i], mean, inv, p.weight, p.bias, channel(i));
            put8<T, kVec>(p, m, channel(i), v[i]);
        }
    }
}

// Rows that do not fit the registers: X and residual are read again (from the L2) for each sum and for the outputs. A thread
// reads a position of X and residual last before it writes there, so that R and Y may be their buffers.
template <typename T, bool kVec>
__global__ void __launch_bounds__(1024) block_norm_long_kernel(const BlockNormArgs p) {
    __shared__ Sums sums;
    int turn = 0;
    const float count = static_cast<float>(p.K);
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + m * p.ldx;
        const T* res = static_cast<const T*>(p.residual) + m * p.ldr;
        const int64_t gate_row = p.gate != nullptr ? m / p.gate_tokens * p.ldg : 0;
        float mean[2] = {0.0f, 0.0f}, inv[2] = {1.0f, 1.0f};   // of X, of r
        auto value = [&](int which, int k, float (&v)[8]) {   // X (0) or r (1) at channels k .. k + 7, 0 past K
            load8<T, kVec>(x, k, p.K, v);
            if (which == 0) return;
            float add[8];
            if (p.residual != nullptr) load8<T, kVec>(res, k, p.K, add);
            if (p.post_norm) scale8<T, kVec>(p, v, mean[0], inv[0], p.post_weight, p.post_bias, k);
            join8<T, kVec>(p, v, add, gate_row, k);
            if (k + 8 > p.K)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (k + c >= p.K) v[c] = 0.0f;
        };
        for (int which = 0; which < 2; ++which) {
            if (which == 0 ? !p.post_norm : !p.pre_norm) continue;
            if (p.layer_norm) {
                float sum = 0.0f;
                for (int k = static_cast<int>(threadIdx.x) * 8; k < p.K; k += static_cast<int>(blockDim.x) * 8) {
                    float v[8];
                    value(which, k, v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) sum += v[c];
                }
                mean[which] = row_sum(sum, sums, turn) / count;
            }
            float sq = 0.0f;
            for (int k = static_cast<int>(threadIdx.x) * 8; k < p.K; k += static_cast<int>(blockDim.x) * 8) {
                float v[8];
                value(which, k, v);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float d = v[c] - mean[which];
                    if (!p.layer_norm || k + c < p.K) sq = fmaf(d, d, sq);
                }
            }
            inv[which] = __frsqrt_rn(row_sum(sq, sums, turn) / count + p.eps);
        }
        const int end = p.nb * 128;   // (whole half warps: K is rounded up to a block)
        for (int k0 = 0; k0 < end; k0 += static_cast<int>(blockDim.x) * 8) {
            const int k = k0 + static_cast<int>(threadIdx.x) * 8;
            float v[8] = {};
            if (k < p.K) {
                value(1, k, v);
                if (p.R != nullptr) store8<T, kVec>(static_cast<T*>(p.R) + m * p.ldo, k, p.K, v);
            }
            if (!p.pre_norm) continue;
            if (k < p.K) scale8<T, kVec>(p, v, mean[1], inv[1], p.weight, p.bias, k);
            put8<T, kVec>(p, m, k, v);
        }
    }
}

template <typename T, bool kVec>
cudaError_t block_norm_as(const BlockNormArgs& p, int num_sms, cudaStream_t stream) {
    const int vectors = p.nb * 16;   // of 8 channels
    const int64_t most = static_cast<int64_t>(num_sms) * 64;
    const unsigned grid = static_cast<unsigned>(p.M < most ? p.M : most);
    auto threads_for = [&](int per) { return ((vectors + per - 1) / per + 31) / 32 * 32; };
    // few rows: as many threads a row as there are vectors, for the shortest chain; else 4 vectors a thread
    const bool few = p.M < 2 * num_sms;
    if (few && threads_for(1) <= 1024) {
        block_norm_kernel<T, kVec, 1><<<grid, threads_for(1), 0, stream>>>(p);
    } else if (threads_for(4) <= 512) {
        if (threads_for(4) >= 128) block_norm_kernel<T, kVec, 4><<<grid, threads_for(4), 0, stream>>>(p);
        else if (threads_for(2) >= 64) block_norm_kernel<T, kVec, 2><<<grid, threads_for(2), 0, stream>>>(p);
        else block_norm_kernel<T, kVec, 1><<<grid, threads_for(1), 0, stream>>>(p);
    } else {
        block_norm_long_kernel<T, kVec><<<grid, 1024, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& p, int num_sms, cudaStream_t stream) {
    auto aligned = [](const void* v) { return (reinterpret_cast<uintptr_t>(v) & 15u) == 0; };
    const bool vec = aligned(p.X) && p.ldx % 8 == 0 && aligned(p.residual) && p.ldr % 8 == 0 && aligned(p.R) && p.ldo % 8 == 0 &&
                     aligned(p.Y) && p.ldy % 8 == 0 && aligned(p.gate) && p.ldg % 8 == 0 && aligned(p.weight) && aligned(p.bias) &&
                     aligned(p.post_weight) && aligned(p.post_bias);
    if (p.dtype == kF16)
        return vec ? block_norm_as<__half, true>(p, num_sms, stream) : block_norm_as<__half, false>(p, num_sms, stream);
    return vec ? block_norm_as<__nv_bfloat16, true>(p, num_sms, stream) : block_norm_as<__nv_bfloat16, false>(p, num_sms, stream);
}

}  // namespace fmpq
