// E4M3 product with a scale for each block of 128 (sm_103a), plain and routed to experts:
//
//   Y[m][n] = sum_b a_scale[b][m] * w_scale[n / 128][b] * P[m][n][b],
//   P[m][n][b] = sum over the 128 channels of block b of a_code * w_code, in FP32.
//
// First form: one thread a weight row, 16 tokens a CTA, FP32 arithmetic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_internal.h"

namespace fmpq {
namespace {

constexpr int kTok = 16;

__device__ __forceinline__ void e4m3x4(uint32_t v, float* f) {
    uint32_t a, b;
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}" : "=r"(a), "=r"(b) : "r"(v));
    const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a)), y = __half22float2(*reinterpret_cast<__half2*>(&b));
    f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
}
__device__ __forceinline__ uint8_t to_e4m3(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return static_cast<uint8_t>(r);
}

struct SimpleParams {
    Fp8GemmArgs a;
    int K, N, nb, pairs, scale_rows, gated, experts;
};

__global__ void __launch_bounds__(256) simple_kernel(const SimpleParams p) {
    __shared__ float xs[kTok][128];
    __shared__ float sx[kTok];
    __shared__ float h[256][kTok + 1];
    __shared__ float hmax[kTok];
    const int e = blockIdx.z, pair = blockIdx.x;
    const int64_t first = p.a.start ? p.a.start[e] : 0;
    const int64_t count = p.a.count ? p.a.count[e] : p.a.rows;
    const int64_t sstride = scale_stride(p.a.rows);
    const int t = 2 * pair + (threadIdx.x >> 7), r = threadIdx.x & 127;
    const int n = fp8_source_row(t, r, p.N, p.gated);
    const uint8_t* w = static_cast<const uint8_t*>(p.a.W) +
                       ((static_cast<int64_t>(e) * p.pairs * 2 + t) * p.nb) * kTileBytes + r * 128;
    const float* ws = p.a.w_scales + (static_cast<int64_t>(e) * p.scale_rows + (n >= 0 ? fp8_scale_row(n, p.N, p.gated) : 0)) * p.nb;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTok; m0 < count; m0 += static_cast<int64_t>(gridDim.y) * kTok) {
        float acc[kTok];
        for (int i = 0; i < kTok; ++i) acc[i] = 0.0f;
        for (int b = 0; b < p.nb; ++b) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTok * 32; i += 256) {
                const int m = i >> 5, c4 = i & 31;
                const int64_t row = first + m0 + m;
                float f[4] = {0.f, 0.f, 0.f, 0.f};
                if (m0 + m < count)
                    e4m3x4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.a.A) + (b * p.a.rows + row) * 128 +
                                                              (((c4 >> 2) ^ static_cast<int>(row & 7)) << 4) + (c4 & 3) * 4), f);
                for (int j = 0; j < 4; ++j) xs[m][c4 * 4 + j] = f[j];
            }
            if (threadIdx.x < kTok) sx[threadIdx.x] = m0 + threadIdx.x < count ? p.a.a_scales[b * sstride + first + m0 + threadIdx.x] : 0.0f;
            __syncthreads();
            float P[kTok];
            for (int i = 0; i < kTok; ++i) P[i] = 0.0f;
            for (int c = 0; c < 8; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(w + static_cast<int64_t>(b) * kTileBytes + ((c ^ (r & 7)) << 4));
                float f[16];
                e4m3x4(v.x, f); e4m3x4(v.y, f + 4); e4m3x4(v.z, f + 8); e4m3x4(v.w, f + 12);
                for (int j = 0; j < 16; ++j)
#pragma unroll
                    for (int i = 0; i < kTok; ++i) P[i] = fmaf(f[j], xs[i][c * 16 + j], P[i]);
            }
            const float s = ws[b];
#pragma unroll
            for (int i = 0; i < kTok; ++i) acc[i] = fmaf(P[i], s * sx[i], acc[i]);
        }
        if (!p.gated) {
            for (int i = 0; i < kTok; ++i) {
                if (m0 + i >= count || n < 0) continue;
                const int64_t row = first + m0 + i;
                float y = acc[i];
                if (p.a.pair_weight) y *= p.a.pair_weight[p.a.pair_of[row]];
                if (p.a.dtype == kF16) static_cast<__half*>(p.a.Y)[row * p.a.ldy + n] = __float2half(y);
                else static_cast<__nv_bfloat16*>(p.a.Y)[row * p.a.ldy + n] = __float2bfloat16(y);
            }
            continue;
        }
        __syncthreads();
        for (int i = 0; i < kTok; ++i) h[threadIdx.x][i] = acc[i];
        __syncthreads();
        if ((r & 31) < 16)
            for (int i = 0; i < kTok; ++i) {
                const float g = h[threadIdx.x][i];
                h[threadIdx.x][i] = g / (1.0f + expf(-g)) * h[threadIdx.x + 16][i];
            }
        __syncthreads();
        if (threadIdx.x < kTok) {
            float m = 0.0f;
            for (int i = 0; i < 256; ++i) if ((i & 31) < 16) m = fmaxf(m, fabsf(h[i][threadIdx.x]));
            hmax[threadIdx.x] = __fdiv_rn(m, 448.0f);
        }
        __syncthreads();
        if ((r & 31) < 16) {
            const int l = r & 15;
            const int ch = 64 * (t & 1) + 16 * (r >> 5) + 4 * ((l & 7) >> 1) + 2 * (l >> 3) + (l & 1);
            for (int i = 0; i < kTok; ++i) {
                if (m0 + i >= count) continue;
                const int64_t row = first + m0 + i;
                const float s = hmax[i];
                static_cast<uint8_t*>(p.a.H)[(static_cast<int64_t>(pair) * p.a.rows + row) * 128 + (((ch >> 4) ^ static_cast<int>(row & 7)) << 4) + (ch & 15)] =
                    to_e4m3(s > 0.0f ? __fdiv_rn(h[threadIdx.x][i], s) : 0.0f);
            }
        }
        if (threadIdx.x < kTok && m0 + threadIdx.x < count) p.a.h_scales[pair * sstride + first + m0 + threadIdx.x] = hmax[threadIdx.x];
        __syncthreads();
    }
}

}  // namespace

size_t fp8_gemm_workspace(const fp8_layer&, int64_t) { return 0; }

cudaError_t launch_fp8_gemm(const fp8_layer& L, const Fp8GemmArgs& a, cudaStream_t stream) {
    SimpleParams p{a, L.K, L.N, L.nb, L.pairs, L.scale_rows, L.gated, L.experts};
    const int64_t tiles = (a.pairs_routed + kTok - 1) / kTok;
    const dim3 grid(L.pairs, static_cast<unsigned>(tiles < 256 ? tiles : 256), L.experts);
    simple_kernel<<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fmpq
