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
#include <climits>
#include <initializer_list>
#include <type_traits>

#include "fmpq_device.cuh"
#include "fmpq_internal.h"
#include "fp8_codes.cuh"
#include "fp8_internal.h"
#include "pieces.cuh"

namespace fmpq {
namespace {

// Arithmetic runs on pairs (packed FP32 instructions): a vector of 8 channels is four of them.
using V8 = float2[4];

// How the vectors of a kernel lie: kWhole: K is a multiple of 8 and weights and outputs are on 16-byte boundaries, so every vector
// below K is a 16-byte access; kMixed: a row's last vector may be partial; kAny: any alignment of the elements (one CTA a row, 4481 x 4291, X 2
// bytes off: 90 us, by single elements 119; 777 x 2868, rows on 8-byte boundaries: 10.2, 17).
enum { kWhole = 0, kMixed = 1, kAny = 2 };
// Which norm: known to the compiler, or a branch.
enum { kRms = 0, kLayer = 1, kEither = 2 };

template <int kNorm>
__device__ __forceinline__ bool is_layer(const BlockNormArgs& p) { return kNorm == kEither ? p.layer_norm != 0 : kNorm == kLayer; }

// ---------------------------------------------------------------- eight values of a row or a vector

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, V8& v) {
    const T* t = nullptr;
    v[0] = unpack2(u.x, t);
    v[1] = unpack2(u.y, t);
    v[2] = unpack2(u.z, t);
    v[3] = unpack2(u.w, t);
}
__device__ __forceinline__ uint32_t pack2(float2 f, const __half*) {
    const __half2 v = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float2 f, const __nv_bfloat16*) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store1(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float& at(V8& v, int c) { return (c & 1) ? v[c >> 1].y : v[c >> 1].x; }
__device__ __forceinline__ float at(const V8& v, int c) { return (c & 1) ? v[c >> 1].y : v[c >> 1].x; }

// Channels k .. k + 7 of a row, those past K as 0 (kWhole: k < K).
template <typename T, int kLie>
__device__ __forceinline__ void load8(const T* row, int k, int K, V8& v) {
    if (kLie == kWhole || (kLie == kMixed && k + 8 <= K)) {
        unpack8<T>(*reinterpret_cast<const uint4*>(row + k), v);
    } else if (kLie == kAny && k + 8 <= K) {
        unpack8<T>(eight_at(row, k), v);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) at(v, c) = k + c < K ? load_as_float(row + k + c) : 0.0f;
    }
}
template <typename T, int kLie>
__device__ __forceinline__ void store8(T* row, int k, int K, const V8& v) {
    if (kLie == kWhole || (kLie == kMixed && k + 8 <= K)) {
        const T* t = nullptr;
        *reinterpret_cast<uint4*>(row + k) = make_uint4(pack2(v[0], t), pack2(v[1], t), pack2(v[2], t), pack2(v[3], t));
    } else if (kLie == kAny && k + 8 <= K) {   // in the widest accesses that the row's start allows
        const T* t = nullptr;
        T* to = row + k;
        const uint32_t o[4] = {pack2(v[0], t), pack2(v[1], t), pack2(v[2], t), pack2(v[3], t)};
        const uint32_t past = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 7u);
        if (past == 0) {
            reinterpret_cast<uint2*>(to)[0] = make_uint2(o[0], o[1]);
            reinterpret_cast<uint2*>(to)[1] = make_uint2(o[2], o[3]);
        } else if (past == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(to)[i] = o[i];
        } else {
            *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(o[0]);
#pragma unroll
            for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t*>(to + 1)[i] = __funnelshift_r(o[i], o[i + 1], 16);
            *reinterpret_cast<uint16_t*>(to + 7) = static_cast<uint16_t>(o[3] >> 16);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (k + c < K) store1(row + k + c, at(v, c));
    }
}
// The same of a weight, bias or gate: of X's type, or FP32.
template <typename T, int kLie>
__device__ __forceinline__ void param8(const void* p, int fp32, int64_t first, int k, int K, V8& v) {
    if (!fp32) {
        load8<T, kLie>(static_cast<const T*>(p) + first, k, K, v);
        return;
    }
    const float* f = static_cast<const float*>(p) + first + k;
    if (kLie == kWhole || (kLie == kMixed && k + 8 <= K)) {
        const float4 a = *reinterpret_cast<const float4*>(f), b = *reinterpret_cast<const float4*>(f + 4);
        v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) at(v, c) = k + c < K ? f[c] : 0.0f;
    }
}

// ---------------------------------------------------------------- sums over a row

constexpr int kMostStages = 4;   // rows in flight a CTA

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

__device__ __forceinline__ void add8(float& sum, const V8& v) {
    const float2 a = fadd2(fadd2(v[0], v[1]), fadd2(v[2], v[3]));
    sum += a.x + a.y;
}
// sum += (v - mean)^2; a layer norm's values past K do not count (the others are 0 there)
template <int kLie, int kNorm>
__device__ __forceinline__ void square8(const BlockNormArgs& p, float2& sum, const V8& v, float mean, int k) {
    if (!is_layer<kNorm>(p)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = dev::ffma2(v[i], v[i], sum);
        return;
    }
    if (kLie == kWhole && k >= p.K) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 d = fadd2(v[i], both(-mean));
        if (kLie != kWhole) {
            if (k + 2 * i >= p.K) d.x = 0.0f;
            if (k + 2 * i + 1 >= p.K) d.y = 0.0f;
        }
        sum = dev::ffma2(d, d, sum);
    }
}
// 1 / sqrt(mean square + eps), rounded once: all of a row's values carry its error. (rsqrtf, off by up to two steps: 45 of 33 million E4M3 codes and 686 of as many
// bf16 values of r are not those of 64 bits, in the mean of six inputs; this: 39 and 621, as FP32's correctly rounded root and quotient, 42 and 630.) One step of Newton's iteration from rsqrtf's y, y + y / 2 (1 - d y^2), d y in two parts so that the residual is
// good to 2^-46: the result is within 2^-20 of a step of the nearest value's half step (of all 2^31 positive d, 257 next to a tie go to its other side). Both norms
// at 4096 x 8192: 66.4 us; with __frsqrt_rn, which has no such exceptions and three times the instructions, 67.4; with rsqrtf alone 65.6.
__device__ __forceinline__ float inverse(const BlockNormArgs& p, float mean_square) {
    const float d = mean_square + p.eps, y = rsqrtf(d);
    const float h = d * y, l = fmaf(d, y, -h);
    const float rest = fmaf(-l, y, fmaf(-h, y, 1.0f));
    return d < INFINITY ? fmaf(0.5f * y, rest, y) : y;   // (of infinity 0, of NaN NaN)
}

template <typename T, int kLie, int kNorm>
__device__ __forceinline__ void scale8(const BlockNormArgs& p, V8& v, float mean, float inv, const void* w, const void* b, int k) {
    V8 t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (is_layer<kNorm>(p)) v[i] = fadd2(v[i], both(-mean));
        v[i] = dev::fmul2(v[i], both(inv));
    }
    if (w != nullptr) {
        param8<T, kLie>(w, p.param_f32, 0, k, p.K, t);
        if (p.weight_offset != 0.0f)
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = fadd2(t[i], both(p.weight_offset));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = dev::fmul2(v[i], t[i]);
    }
    if (b != nullptr) {
        param8<T, kLie>(b, p.param_f32, 0, k, p.K, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fadd2(v[i], t[i]);
    }
}

// u to r; residual already read.
template <typename T, int kLie>
__device__ __forceinline__ void join8(const BlockNormArgs& p, V8& v, const V8& res, int64_t gate_row, int k) {
    if (p.gate != nullptr) {
        V8 t;
        param8<T, kLie>(p.gate, p.gate_f32, gate_row, k, p.K, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = dev::fmul2(v[i], t[i]);
    }
    if (p.residual != nullptr)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = dev::ffma2(both(p.residual_scale), res[i], v[i]);
}
// First element of the gate's row for row m. (M is at most 2^24: 32 bits do.)
__device__ __forceinline__ int64_t gate_row_of(const BlockNormArgs& p, int64_t m) {
    if (p.gate == nullptr || p.gate_tokens >= p.M) return 0;
    return static_cast<int64_t>(static_cast<uint32_t>(m) / static_cast<uint32_t>(p.gate_tokens)) * p.ldg;
}

// y to memory: 16 bits, and codes (16 lanes of a half warp hold a block of 128; every lane calls it, with 0 past K).
template <typename T, int kLie>
__device__ __forceinline__ void put8(const BlockNormArgs& p, int64_t m, int k, V8& v) {
    if (p.Y != nullptr && k < p.K) store8<T, kLie>(static_cast<T*>(p.Y) + m * p.ldy, k, p.K, v);
    if (p.A == nullptr) return;
    if (kLie != kWhole && k < p.K && k + 8 > p.K)
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (k + c >= p.K) at(v, c) = 0.0f;
    const float q[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    const float s = scale_of(q);
    const int b = k >> 7;
    if (b >= p.nb) return;
    const uint2 code = codes_of(q, s);
    const int l = (k >> 3) & 15;
    uint8_t* row = p.A + (static_cast<int64_t>(b) * p.M + m) * 128;
    *reinterpret_cast<uint2*>(row + (((l >> 1) ^ static_cast<int>(m & 7)) << 4) + (l & 1) * 8) = code;
    if (l == 0) p.a_scales[b * p.sstride + m] = s;
}

// mean and 1 / sqrt(mean square + eps) of the CTA's row from its registers (0 past K).
template <int kLie, int kNorm, int kV>
__device__ __forceinline__ void statistics(const BlockNormArgs& p, const V8 (&v)[kV], Sums& s, int& turn, float& mean, float& inv) {
    mean = 0.0f;
    if (is_layer<kNorm>(p)) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) add8(sum, v[i]);
        mean = row_sum(sum, s, turn) * p.inv_count;
    }
    float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kV; ++i) square8<kLie, kNorm>(p, sq, v[i], mean, (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8);
    inv = inverse(p, row_sum(sq.x + sq.y, s, turn) * p.inv_count);
}

// ---------------------------------------------------------------- kernels

// One CTA a row, kV vectors of 8 channels a thread: blockDim.x * 8 * kV >= nb * 128.
template <typename T, int kLie, int kV>
__global__ void __launch_bounds__(kV <= 2 ? 1024 : 512) block_norm_kernel(const BlockNormArgs p) {
    __shared__ Sums sums;
    int turn = 0;
    dev::pdl_wait();
    dev::pdl_launch_dependents();
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + m * p.ldx;
        const T* res = static_cast<const T*>(p.residual) + m * p.ldr;
        const int64_t gate_row = gate_row_of(p, m);
        V8 v[kV], add[kV];
        auto channel = [&](int i) { return (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8; };
#pragma unroll
        for (int i = 0; i < kV; ++i) load8<T, kLie>(x, channel(i), p.K, v[i]);
        if (p.residual != nullptr)
#pragma unroll
            for (int i = 0; i < kV; ++i) load8<T, kLie>(res, channel(i), p.K, add[i]);
        float mean, inv;
        if (p.post_norm) statistics<kLie, kEither>(p, v, sums, turn, mean, inv);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (channel(i) >= p.K) continue;
            if (p.post_norm) scale8<T, kLie, kEither>(p, v[i], mean, inv, p.post_weight, p.post_bias, channel(i));
            join8<T, kLie>(p, v[i], add[i], gate_row, channel(i));
            if (channel(i) + 8 > p.K)   // (a post norm's value of 0 is not 0)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (channel(i) + c >= p.K) at(v[i], c) = 0.0f;
            if (p.R != nullptr) store8<T, kLie>(static_cast<T*>(p.R) + m * p.ldo, channel(i), p.K, v[i]);
        }
        if (!p.pre_norm) continue;
        statistics<kLie, kEither>(p, v, sums, turn, mean, inv);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (channel(i) < p.K) scale8<T, kLie, kEither>(p, v[i], mean, inv, p.weight, p.bias, channel(i));
            put8<T, kLie>(p, m, channel(i), v[i]);
        }
    }
}

// Rows that do not fit the registers: X and residual are read again (from the L2) for each sum and for the outputs. A thread
// reads a position of X and residual last before it writes there, so that R and Y may be their buffers.
template <typename T, int kLie>
__global__ void __launch_bounds__(1024) block_norm_long_kernel(const BlockNormArgs p) {
    __shared__ Sums sums;
    int turn = 0;
    dev::pdl_wait();
    dev::pdl_launch_dependents();
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + m * p.ldx;
        const T* res = static_cast<const T*>(p.residual) + m * p.ldr;
        const int64_t gate_row = gate_row_of(p, m);
        float mean[2] = {0.0f, 0.0f}, inv[2] = {1.0f, 1.0f};   // of X, of r
        auto value = [&](int which, int k, V8& v) {   // X (0) or r (1) at channels k .. k + 7, 0 past K
            load8<T, kLie>(x, k, p.K, v);
            if (which == 0) return;
            V8 add;
            if (p.residual != nullptr) load8<T, kLie>(res, k, p.K, add);
            if (p.post_norm) scale8<T, kLie, kEither>(p, v, mean[0], inv[0], p.post_weight, p.post_bias, k);
            join8<T, kLie>(p, v, add, gate_row, k);
            if (k + 8 > p.K)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (k + c >= p.K) at(v, c) = 0.0f;
        };
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (which == 0 ? !p.post_norm : !p.pre_norm) continue;
            if (p.layer_norm) {
                float sum = 0.0f;
                for (int k = static_cast<int>(threadIdx.x) * 8; k < p.K; k += static_cast<int>(blockDim.x) * 8) {
                    V8 v;
                    value(which, k, v);
                    add8(sum, v);
                }
                mean[which] = row_sum(sum, sums, turn) * p.inv_count;
            }
            float2 sq = make_float2(0.0f, 0.0f);
            for (int k = static_cast<int>(threadIdx.x) * 8; k < p.K; k += static_cast<int>(blockDim.x) * 8) {
                V8 v;
                value(which, k, v);
                square8<kLie, kEither>(p, sq, v, mean[which], k);
            }
            inv[which] = inverse(p, row_sum(sq.x + sq.y, sums, turn) * p.inv_count);
        }
        const int end = p.nb * 128;   // (whole half warps: K is rounded up to a block)
        for (int k0 = 0; k0 < end; k0 += static_cast<int>(blockDim.x) * 8) {
            const int k = k0 + static_cast<int>(threadIdx.x) * 8;
            V8 v = {};
            if (k < p.K) {
                value(1, k, v);
                if (p.R != nullptr) store8<T, kLie>(static_cast<T*>(p.R) + m * p.ldo, k, p.K, v);
            }
            if (!p.pre_norm) continue;
            if (k < p.K) scale8<T, kLie, kEither>(p, v, mean[1], inv[1], p.weight, p.bias, k);
            put8<T, kLie>(p, m, k, v);
        }
    }
}

// Bytes that a row of K channels takes in the ring, wherever it starts.
__host__ __device__ inline uint32_t ring_row_bytes(int K) { return ((static_cast<uint32_t>(K) + 7) / 8 * 8 + 8) * 2; }

// Many rows: the CTAs stay, and the next rows are on their way into a ring in shared memory (bulk copies) while one is worked on. Two vectors
// a thread (three, or four, where 1024 threads would not do: 2048 x 24576 85 us with three, 102 with four). Its instructions and the chain of a row through its barriers bound it (4096 x 8192 bf16,
// both norms, a gate, codes: 66.6 us, 236 MB = 3.5 TB/s, an issue slot used in 64 of 100; one norm and the residual 46; the sum alone 32.5,
// 6.2 TB/s), so what can be is uniform or made once: a row's addresses are a base for the CTA and 32-bit offsets of a thread, arithmetic is
// on pairs, P (the weights' type) and the norm are the compiler's. One CTA a row without the ring took 138. No faster: four vectors a thread
// (70), three CTAs of 40 registers in place of two, the weights in shared memory (which leave the ring two rows) or asked for before the sums,
// all within 1 us; without the codes' stores, the scales' or the reduction of a block's maximum it would still take within 1 us of this.
// X and residual lie anywhere: the copies begin on the boundary before a row, and vectors are shifted out of the ring (2325 x 2816 fp16, rows
// 2 bytes off, both norms: 13.6 us, 36 as one CTA a row by single elements). Weights and outputs lie on 16-byte boundaries (kWhole) or K and
// they are anything (kAny: 7572 x 5913 bf16, rows 2 bytes off, both norms, codes: 117 us, 250 as one CTA a row; its shifts and narrow stores
// are instructions more; a warp that shuffles its lanes' values into whole pieces for the stores takes 127).
template <typename P>
__device__ __forceinline__ void param_at(const void* p, uint32_t k, V8& v) {
    if constexpr (sizeof(P) == 2) {
        unpack8<P>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + k * 2u)), v);
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const uint8_t*>(p) + k * 4u);
        const float4 a = __ldg(f), b = __ldg(f + 1);
        v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
    }
}

// The end of a CTA of the kernel below that gave up a row: its rows from there on become NaN, and the copies under way land (a short bound, far longer
// than a copy). Not inlined: the kernel would take registers for it (777 x 2868, a layer norm: 7.5 us in place of 5.9).
template <typename T>
__device__ __noinline__ void give_up(const BlockNormArgs& p, int from, uint64_t* landed, int stages) {
    const int rows = static_cast<int>(p.M), step = static_cast<int>(gridDim.x);
    const float nan = __int_as_float(0x7FFFFFFF);
    for (int64_t m = from; m < rows; m += step) {
        for (int c = threadIdx.x; c < p.K; c += blockDim.x) {
            if (p.R != nullptr) store1(static_cast<T*>(p.R) + m * p.ldo + c, nan);
            if (p.Y != nullptr) store1(static_cast<T*>(p.Y) + m * p.ldy + c, nan);
            if (p.A != nullptr && c < p.nb) p.a_scales[c * p.sstride + m] = nan;
        }
    }
    if (threadIdx.x != 0) return;
    int n = (from - static_cast<int>(blockIdx.x)) / step;   // the row's number among the CTA's: its slot, and those behind it
    for (int i = 0; i < stages && blockIdx.x + static_cast<int64_t>(n) * step < rows; ++i, ++n)
        dev::mbar_wait(&landed[n % stages], (n / stages) & 1, nullptr, 1u << 16);
}

// A copy lands, or its wait gives up after seconds, a thread's last wait then. Threads may disagree, so the first row that any of them gave up counts: no
// slot is filled again from its barrier on, and at the end the CTA's rows from there on are made NaN and the copies under way land.
// kTest: the row `withheld` gets no copy, and waits end after `polls`.
template <typename T, typename P, int kNorm, int kV, int kLie, bool kTest = false>
__global__ void __launch_bounds__(1024) block_norm_stream_kernel(const __grid_constant__ BlockNormArgs p, int stages) {
    extern __shared__ __align__(128) uint8_t ring[];   // [stage][X's row, then the residual's]
    __shared__ Sums sums;
    __shared__ uint64_t landed[kMostStages];
    __shared__ int given_up;   // the first such row
    const uint32_t polls = kTest ? p.polls : dev::kMaxPolls;
    // (a row of a slot has room for a row at any place in its pieces, and for the piece behind its last vector's)
    const uint32_t row_bytes = ring_row_bytes(p.K), slot_bytes = p.residual != nullptr ? 2 * row_bytes : row_bytes;
    const int rows = static_cast<int>(p.M), step = static_cast<int>(gridDim.x);
    auto load = [&](int m, int stage) {
        const T* x = static_cast<const T*>(p.X) + m * p.ldx;
        const T* r = static_cast<const T*>(p.residual) + m * p.ldr;
        const uint32_t x_off = elements_past(x), r_off = elements_past(r);
        auto pieces = [&](uint32_t off) { return ((off + static_cast<uint32_t>(p.K)) * 2 + 15u) & ~15u; };
        const uint32_t x_bytes = pieces(x_off), r_bytes = p.residual != nullptr ? pieces(r_off) : 0u;
        dev::mbar_arrive_expect_tx(&landed[stage], x_bytes + r_bytes);
        if (!kTest || m != p.withheld) dev::bulk_g2s(ring + stage * slot_bytes, x - x_off, x_bytes, &landed[stage]);
        if (p.residual != nullptr) dev::bulk_g2s(ring + stage * slot_bytes + row_bytes, r - r_off, r_bytes, &landed[stage]);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) dev::mbar_init(&landed[i], 1);
        given_up = INT_MAX;
        dev::fence_barrier_init();
    }
    dev::pdl_wait();
    dev::pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + static_cast<int64_t>(i) * step < rows) load(static_cast<int>(blockIdx.x) + i * step, i);
    }
    __syncthreads();

    // this thread's vectors: first channel, whether there is one, places of codes and scale
    uint32_t k[kV], code_at[kV], scale_at[kV];
    bool in[kV];
    const uint32_t l = threadIdx.x & 15u, piece = (l >> 1) << 4;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        k[i] = (i * blockDim.x + threadIdx.x) * 8u;
        in[i] = k[i] < static_cast<uint32_t>(p.K);
        code_at[i] = (k[i] >> 7) * static_cast<uint32_t>(p.M) * 128u + (l & 1u) * 8u;
        scale_at[i] = (k[i] >> 7) * static_cast<uint32_t>(p.sstride) * 4u;
    }
    const bool single = blockDim.x == 32;
    int turn = 0, stage = 0;
    uint32_t phase = 0;
    bool lost = false;   // this thread gave up a row
    for (int m = static_cast<int>(blockIdx.x); m < rows; m += step) {
        if (!lost && !dev::mbar_wait(&landed[stage], phase, nullptr, polls)) {
            lost = true;
            atomicMin(&given_up, m);
        }
        const uint8_t* x = ring + stage * slot_bytes;
        // what a row's last vector has past K (kAny) is 0
        auto cut = [&](uint32_t k, V8& v) {
            if (kLie == kAny && k + 8 > static_cast<uint32_t>(p.K))
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (k + c >= static_cast<uint32_t>(p.K)) at(v, c) = 0.0f;
        };
        // a vector of a row in the ring, which begins `off` elements into it
        auto from_ring = [&](const uint8_t* row, uint32_t off, uint32_t k, V8& v) {
            const uint4* at = reinterpret_cast<const uint4*>(row + k * 2u);
            unpack8<T>(off == 0 ? at[0] : shifted(at[0], at[1], off), v);
            cut(k, v);
        };
        auto param = [&](const void* w, uint32_t k, V8& t) {
            if constexpr (kLie == kAny) param8<T, kAny>(w, p.param_f32, 0, static_cast<int>(k), p.K, t);
            else param_at<P>(w, k, t);
        };
        V8 v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = both(lost ? __int_as_float(0x7FFFFFFF) : 0.0f);
            if (in[i] && !lost) from_ring(x, elements_past(static_cast<const T*>(p.X) + m * p.ldx), k[i], v[i]);
        }
        float mean = 0.0f, inv;
        // v = (v - mean) * inv * w + b
        auto scale = [&](const void* w, const void* b) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                V8 t;
                if (kNorm == kLayer)
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = fadd2(v[i][c], both(-mean));
                if (w != nullptr && in[i]) {
                    param(w, k[i], t);
                    if (p.weight_offset != 0.0f)
#pragma unroll
                        for (int c = 0; c < 4; ++c) t[c] = fadd2(t[c], both(p.weight_offset));
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = dev::fmul2(dev::fmul2(v[i][c], both(inv)), t[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = dev::fmul2(v[i][c], both(inv));
                }
                if (b != nullptr && in[i]) {
                    param(b, k[i], t);
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = fadd2(v[i][c], t[c]);
                }
                if (kNorm == kLayer && !in[i])
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = both(0.0f);
                if (in[i]) cut(k[i], v[i]);   // (its value of 0 is not 0)
            }
        };
        if (p.post_norm) {
            statistics<kLie, kNorm>(p, v, sums, turn, mean, inv);
            scale(p.post_weight, p.post_bias);
        }
        if (p.gate != nullptr) {
            const int64_t gate_row = gate_row_of(p, m);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (!in[i]) continue;
                V8 t;
                if constexpr (kLie == kAny) param8<T, kAny>(p.gate, p.gate_f32, gate_row, static_cast<int>(k[i]), p.K, t);
                else if (p.gate_f32) param_at<float>(static_cast<const float*>(p.gate) + gate_row, k[i], t);
                else param_at<T>(static_cast<const T*>(p.gate) + gate_row, k[i], t);
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] = dev::fmul2(v[i][c], t[c]);
            }
        }
        if (p.residual != nullptr) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (!in[i]) continue;
                V8 t;
                from_ring(x + row_bytes, elements_past(static_cast<const T*>(p.residual) + m * p.ldr), k[i], t);
#pragma unroll
                for (int c = 0; c < 4; ++c) v[i][c] = dev::ffma2(both(p.residual_scale), t[c], v[i][c]);
            }
        }
        if (p.R != nullptr) {
            uint8_t* row = static_cast<uint8_t*>(p.R) + m * p.ldo * 2;
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (in[i]) store8<T, kLie>(reinterpret_cast<T*>(row), static_cast<int>(k[i]), p.K, v[i]);
        }
        if (p.pre_norm) statistics<kLie, kNorm>(p, v, sums, turn, mean, inv);
        if (!p.pre_norm || single) __syncthreads();   // (else the statistics' own barrier)
        // every thread has read the row (or given it up)
        if (threadIdx.x == 0 && m + static_cast<int64_t>(stages) * step < rows && *static_cast<volatile int*>(&given_up) > m)
            load(m + stages * step, stage);
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
        if (!p.pre_norm) continue;
        scale(p.weight, p.bias);
        if (p.Y != nullptr) {
            uint8_t* row = static_cast<uint8_t*>(p.Y) + m * p.ldy * 2;
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (in[i]) store8<T, kLie>(reinterpret_cast<T*>(row), static_cast<int>(k[i]), p.K, v[i]);
        }
        if (p.A != nullptr) {
            uint8_t* codes = p.A + static_cast<int64_t>(m) * 128;
            uint8_t* scales = reinterpret_cast<uint8_t*>(p.a_scales + m);
            const uint32_t swizzled = piece ^ ((m & 7) << 4);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float q[8] = {v[i][0].x, v[i][0].y, v[i][1].x, v[i][1].y, v[i][2].x, v[i][2].y, v[i][3].x, v[i][3].y};
                const float s = scale_of(q);
                if (k[i] >= static_cast<uint32_t>(p.nb) * 128u) continue;
                *reinterpret_cast<uint2*>(codes + (code_at[i] + swizzled)) = codes_of(q, s);
                if (l == 0) *reinterpret_cast<float*>(scales + scale_at[i]) = s;
            }
        }
    }
    __syncthreads();
    if (given_up != INT_MAX) give_up<T>(p, given_up, landed, stages);
}

// Threads that a row of nb blocks takes at `per` vectors each.
int threads_for(int nb, int per) { return ((nb * 16 + per - 1) / per + 31) / 32 * 32; }

constexpr int kRingBytes = 225 * 1024;

// Whether the rows are long enough and a CTA's ring holds two; and the kernel over it. (not `whole`, against one CTA a row: 4096 x 1501 bf16 21.0
// us to 19.6, 4096 x 2001 23.1 to 25.2, 4481 x 4291 49 to 100)
bool fits_stream(const BlockNormArgs& p, bool whole) {
    const int slot = static_cast<int>(ring_row_bytes(p.K)) * (p.residual != nullptr ? 2 : 1);
    return p.K >= (whole ? 512 : 1792) && threads_for(p.nb, 4) <= 1024 && 2 * slot <= kRingBytes && p.M * p.nb * 128 < INT64_C(1) << 32;   // (32-bit offsets of the codes)
}
template <typename T>
cudaError_t block_norm_stream(const BlockNormArgs& p, bool whole, int num_sms, cudaStream_t stream) {
    using std::integral_constant;
    const int per = threads_for(p.nb, 2) <= 1024 ? 2 : threads_for(p.nb, 3) <= 1024 ? 3 : 4, threads = threads_for(p.nb, per);
    auto of = [&](auto norm, auto v) {
        if (!whole) return block_norm_stream_kernel<T, T, norm.value, v.value, kAny>;
        return p.param_f32 ? block_norm_stream_kernel<T, float, norm.value, v.value, kWhole> : block_norm_stream_kernel<T, T, norm.value, v.value, kWhole>;
    };
    auto at = [&](auto norm) {
        return per == 2 ? of(norm, integral_constant<int, 2>{}) : per == 3 ? of(norm, integral_constant<int, 3>{}) : of(norm, integral_constant<int, 4>{});
    };
    auto fn = p.layer_norm ? at(integral_constant<int, kLayer>{}) : at(integral_constant<int, kRms>{});
    if (p.polls != 0) {
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            if (!whole || p.param_f32 || per != 2) return cudaErrorNotSupported;
            fn = p.layer_norm ? block_norm_stream_kernel<T, T, kLayer, 2, kWhole, true> : block_norm_stream_kernel<T, T, kRms, 2, kWhole, true>;
        } else {
            return cudaErrorNotSupported;
        }
    }
    const int slot = static_cast<int>(ring_row_bytes(p.K)) * (p.residual != nullptr ? 2 : 1);
    // CTAs an SM by its registers (4096 x 8960: 55 us, at 64 registers a thread for every kernel 78; 4481 x 4291: 49, 66)
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(fn));
    if (e != cudaSuccess) return e;
    int resident = 65536 / (((a.numRegs + 7) & ~7) * threads);
    if (resident > 16) resident = 16;
    int stages = 200 * 1024 / resident / slot;
    stages = stages > kMostStages ? kMostStages : stages < 2 ? 2 : stages;
    e = ensure_smem_limit(reinterpret_cast<const void*>(fn), kRingBytes);
    if (e != cudaSuccess) return e;
    const int64_t ctas = static_cast<int64_t>(num_sms) * resident;
    return launch_after(fn, dim3(static_cast<unsigned>(p.M < ctas ? p.M : ctas)), threads, stages * slot, true, stream, p, stages);
}

// One CTA a row. Few rows: as many threads a row as there are vectors, for the shortest chain; else up to 4 vectors a thread.
template <typename T, int kLie>
cudaError_t block_norm_rows(const BlockNormArgs& p, bool few, int num_sms, cudaStream_t stream) {
    const int64_t most = static_cast<int64_t>(num_sms) * 64;
    const dim3 grid(static_cast<unsigned>(p.M < most ? p.M : most));
    auto launch = [&](auto kernel, int per) { return launch_after(kernel, grid, threads_for(p.nb, per), 0, true, stream, p); };
    if (few && threads_for(p.nb, 1) <= 1024) return launch(block_norm_kernel<T, kLie, 1>, 1);
    if (few && threads_for(p.nb, 2) <= 1024) return launch(block_norm_kernel<T, kLie, 2>, 2);
    if (threads_for(p.nb, 4) > 512) return launch_after(block_norm_long_kernel<T, kLie>, grid, 1024, 0, true, stream, p);
    if (threads_for(p.nb, 4) >= 128) return launch(block_norm_kernel<T, kLie, 4>, 4);
    if (threads_for(p.nb, 2) >= 64) return launch(block_norm_kernel<T, kLie, 2>, 2);
    return launch(block_norm_kernel<T, kLie, 1>, 1);
}

template <typename T>
cudaError_t block_norm_of(const BlockNormArgs& p, int num_sms, cudaStream_t stream) {
    // bits of the addresses where rows and vectors start
    uintptr_t in = 0, out = 0;
    for (const void* v : {p.X, p.residual}) in |= reinterpret_cast<uintptr_t>(v);
    for (int64_t ld : {p.ldx, p.ldr}) in |= static_cast<uintptr_t>(ld) * 2;
    for (const void* v : {static_cast<const void*>(p.R), static_cast<const void*>(p.Y), p.gate, p.weight, p.bias, p.post_weight, p.post_bias})
        out |= reinterpret_cast<uintptr_t>(v);
    for (int64_t ld : {p.ldo, p.ldy}) out |= static_cast<uintptr_t>(ld) * 2;
    out |= static_cast<uintptr_t>(p.ldg) * (p.gate_f32 ? 4 : 2);
    const bool few = p.M < 2 * num_sms;
    const bool whole = p.K % 8 == 0 && (out & 15u) == 0;
    if (!few && fits_stream(p, whole)) return block_norm_stream<T>(p, whole, num_sms, stream);
    if (p.polls != 0) return cudaErrorNotSupported;
    return ((in | out) & 15u) == 0 ? block_norm_rows<T, kMixed>(p, few, num_sms, stream) : block_norm_rows<T, kAny>(p, few, num_sms, stream);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& p, int num_sms, cudaStream_t stream) {
    return p.dtype == kF16 ? block_norm_of<__half>(p, num_sms, stream) : block_norm_of<__nv_bfloat16>(p, num_sms, stream);
}

}  // namespace fmpq
