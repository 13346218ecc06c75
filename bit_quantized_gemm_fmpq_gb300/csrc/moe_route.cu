// Routing to experts (sm_103a): the top-k experts of each token from the router's logits, the
// plan that sorts the chosen (token, slot) pairs by expert, and the sum of the experts' outputs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_internal.h"

namespace fmpq {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kNone = -INFINITY;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Unsigned integers in the order of the values (-0 counts as 0).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(kAll, ordered(v))); }
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const double o = __shfl_xor_sync(kAll, v, d);
        if (o > v) v = o;
    }
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

struct Rules {
    int E, k, groups, top_groups, group_top;
};

// Two keys computed in FP32 may be closer than their errors: each is within 8 half steps of its
// value (an exponential, a sum, a quotient and the bias), a group's sum of two within 16.
__device__ __forceinline__ bool close_call(float hi, float lo) {
    return hi - lo <= 1.9073486e-6f * fmaxf(1.0f, fmaxf(fabsf(hi), fabsf(lo)));   // 2^-19
}
__device__ __forceinline__ bool close_call(double, double) { return false; }

// Drop the experts outside the best groups: keys of the others become -inf. Lane L holds the
// experts L * NI .. L * NI + NI - 1. Returns whether a close call decided.
template <int NI, typename V>
__device__ __forceinline__ bool keep_best_groups(V (&key)[NI], const Rules& r, int lane, bool check) {
    const int per = r.E / r.groups;
    V mine = V(kNone);   // lane g: the value of group g
    for (int g = 0; g < r.groups; ++g) {
        const int lo = g * per - lane * NI, hi = lo + per;
        V b1 = V(kNone), b2 = V(kNone);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (i >= lo && i < hi) {
                const V v = key[i];
                if (v > b1) { b2 = b1; b1 = v; }
                else if (v > b2) b2 = v;
            }
        const V m1 = warp_max(b1);
        V value = m1;
        if (r.group_top == 2) {
            const unsigned who = __ballot_sync(kAll, b1 == m1);
            if (lane == __ffs(who) - 1) b1 = b2;
            const V m2 = warp_max(b1);
            if (m2 > V(kNone)) value += m2;
        }
        if (lane == g) mine = value;
    }
    unsigned chosen = 0;
    V last = V(kNone);
    for (int i = 0; i < r.top_groups; ++i) {
        const V m = warp_max(mine);
        if (!(m > V(kNone))) break;
        const int g = __ffs(__ballot_sync(kAll, mine == m)) - 1;
        chosen |= 1u << g;
        if (lane == g) mine = V(kNone);
        last = m;
    }
    bool close = false;
    if (check) {
        const V next = warp_max(mine);
        close = next > V(kNone) && close_call(last, next);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane * NI + i;
        if (e < r.E && !((chosen >> (e / per)) & 1u)) key[i] = V(kNone);
    }
    return close;
}

// The k largest keys, the lowest index first among equals: lane j receives the j-th expert and its
// item's score. `logit` and `bias` tell a true tie (both equal) from a close call.
template <int NI, typename V>
__device__ __forceinline__ bool take_top(V (&key)[NI], const float (&score)[NI], const float (&logit)[NI],
                                         const float* bias, const Rules& r, int lane, bool check, int& my_id,
                                         float& my_score) {
    bool close = false;
    V last = V(kNone);
    float last_logit = 0.0f, last_bias = 0.0f;
    const int rounds = check && r.k < r.E ? r.k + 1 : r.k;
    for (int j = 0; j < rounds; ++j) {
        V best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NI; ++i)
            if (key[i] > best) { best = key[i]; at = i; }
        const V m = warp_max(best);
        if (!(m > V(kNone))) break;
        const int w = __ffs(__ballot_sync(kAll, best == m)) - 1;
        at = __shfl_sync(kAll, at, w);
        float sc = 0.0f, lg = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (i == at) {
                sc = score[i];
                lg = logit[i];
                if (lane == w) key[i] = V(kNone);
            }
        const int id = w * NI + at;
        if (check) {
            lg = __shfl_sync(kAll, lg, w);
            const float bs = bias != nullptr ? bias[id] : 0.0f;
            if (j > 0 && close_call(last, m) && !(lg == last_logit && bs == last_bias)) close = true;
            last = m;
            last_logit = lg;
            last_bias = bs;
        }
        sc = __shfl_sync(kAll, sc, w);
        if (lane == j && j < r.k) {
            my_id = id;
            my_score = sc;
        }
    }
    return close;
}

// The same choice with keys in 64 bits, for the tokens where FP32 cannot tell.
template <int NI>
__device__ __noinline__ void choose_in_64(const float* logit, const float* score, const float* bias, int sigmoid, float top,
                                          const Rules r, int lane, int* id_out, float* score_out) {
    double key[NI];
    float lg[NI], sc[NI];
    double total = 0.0;
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
        lg[i] = logit[i];
        sc[i] = score[i];
        const double x = static_cast<double>(lg[i]);
        double v = 0.0;
        if (lg[i] > kNone) v = sigmoid ? 1.0 / (1.0 + exp(-x)) : (lg[i] == top ? 1.0 : exp(x - static_cast<double>(top)));
        key[i] = v;
        total += v;
    }
    if (!sigmoid) {
        total = warp_sum(total);
        if (!(total > 0.0)) total = 1.0;
    } else {
        total = 1.0;
    }
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
        const int e = lane * NI + i;
        double v = key[i] / total;
        if (e < r.E && bias != nullptr) v += static_cast<double>(bias[e]);
        key[i] = (lg[i] > kNone && v > kNone) ? v : static_cast<double>(kNone);
    }
    if (r.groups > 1) keep_best_groups<NI, double>(key, r, lane, false);
    take_top<NI, double>(key, sc, lg, bias, r, lane, false, *id_out, *score_out);
}

// A warp a token. NI experts a lane (E <= 32 * NI), in order, so that the lowest lane holds the
// lowest index.
template <typename T, int NI>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs p) {
    const int lane = threadIdx.x & 31;
    const Rules r{p.E, p.k, p.groups, p.top_groups, p.group_top};
    const bool by_logit = p.bias == nullptr && (p.groups == 1 || p.group_top == 1);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); t < p.T;
         t += static_cast<int64_t>(gridDim.x) * 4) {
        const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
        float logit[NI], score[NI], key[NI];
        float top = kNone;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane * NI + i;
            float v = e < p.E ? as_float(row[e]) : kNone;
            if (!(v > kNone)) v = kNone;   // NaN counts as masked
            logit[i] = v;
            top = fmaxf(top, v);
        }
        top = warp_max(top);
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < NI; ++i) score[i] = logit[i] > kNone ? 1.0f / (1.0f + expf(-logit[i])) : 0.0f;
        } else {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                // (an infinite top: it takes all)
                score[i] = logit[i] > kNone ? (logit[i] == top ? 1.0f : expf(logit[i] - top)) : 0.0f;
                total += score[i];
            }
            total = warp_sum(total);
            const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) score[i] *= inv;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane * NI + i;
            float v = logit[i];
            if (!by_logit && v > kNone) {
                v = score[i];
                if (p.bias != nullptr) v += p.bias[e];
                if (!(v > kNone)) v = kNone;
            }
            key[i] = v;
        }
        int id = -1;
        float sc = 0.0f;
        bool close = false;
        if (p.groups > 1) close = keep_best_groups<NI, float>(key, r, lane, !by_logit);
        close |= take_top<NI, float>(key, score, logit, p.bias, r, lane, !by_logit, id, sc);
        if (close) {
            id = -1;
            sc = 0.0f;
            choose_in_64<NI>(logit, score, p.bias, p.sigmoid, top, r, lane, &id, &sc);
        }
        if (p.renormalize) {
            const float total = warp_sum(sc);
            sc = total > 0.0f ? sc / total : 0.0f;
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = sc * p.scale;
        }
    }
}

template <typename T>
cudaError_t route_as(const RouteArgs& a, cudaStream_t stream) {
    const int64_t ctas = (a.T + 3) / 4;
    const int grid = static_cast<int>(ctas < 65535 ? ctas : 65535);
    if (a.E <= 32) route_kernel<T, 1><<<grid, 128, 0, stream>>>(a);
    else if (a.E <= 64) route_kernel<T, 2><<<grid, 128, 0, stream>>>(a);
    else if (a.E <= 128) route_kernel<T, 4><<<grid, 128, 0, stream>>>(a);
    else if (a.E <= 256) route_kernel<T, 8><<<grid, 128, 0, stream>>>(a);
    else route_kernel<T, 16><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- the plan
// A stable counting sort of the pairs by expert, without atomics on positions: chunks of 1024
// pairs, a CTA each. With several chunks a first launch counts every chunk's pairs per expert; the
// CTA of chunk c then adds up the counts before it.
constexpr int kChunk = 1024;

__global__ void __launch_bounds__(kChunk) plan_count_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                            int32_t* __restrict__ counts) {
    extern __shared__ int32_t hist[];
    for (int e = threadIdx.x; e < E; e += kChunk) hist[e] = 0;
    __syncthreads();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x;
    const int id = i < P ? ids[i] : -1;
    if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kChunk) counts[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
}

// dynamic shared memory: [E] totals then starts, [E] next row of this chunk, [32][E] 16-bit counts
// of each warp
__global__ void __launch_bounds__(kChunk) plan_place_kernel(const int32_t* __restrict__ ids, int64_t P, int E, int chunks,
                                                            const int32_t* __restrict__ counts, int32_t* __restrict__ plan,
                                                            int64_t pairs_cap) {
    extern __shared__ int32_t sm[];
    int32_t* total = sm;
    int32_t* base = sm + E;
    uint16_t* per_warp = reinterpret_cast<uint16_t*>(sm + 2 * E);
    __shared__ int32_t carry[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < 32 * E; i += kChunk) per_warp[i] = 0;
    __syncthreads();
    // ranks inside the warp, counts of the warp
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x;
    int id = i < P ? ids[i] : -1;
    if (id >= E) id = -1;
    const unsigned same = __match_any_sync(kAll, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (id >= 0 && rank == 0) per_warp[warp * E + id] = static_cast<uint16_t>(__popc(same));
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kChunk) {
        int here = 0;
        for (int w = 0; w < 32; ++w) {   // exclusive over the warps
            const int c = per_warp[w * E + e];
            per_warp[w * E + e] = static_cast<uint16_t>(here);
            here += c;
        }
        int before = 0, all = here;
        if (chunks > 1) {
            all = 0;
            for (int c = 0; c < chunks; ++c) {
                const int v = counts[static_cast<int64_t>(c) * E + e];
                if (c < static_cast<int>(blockIdx.x)) before += v;
                all += v;
            }
        }
        total[e] = all;
        base[e] = before;
    }
    __syncthreads();
    // first rows: an exclusive sum of the totals, each rounded up to 8 (E <= 1024: one a thread)
    const int mine = static_cast<int>(threadIdx.x) < E ? (total[threadIdx.x] + 7) & ~7 : 0;
    int sum = mine;
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 31) carry[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        int c = carry[lane];
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kAll, c, d);
            if (lane >= d) c += o;
        }
        carry[lane] = c;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < E) {
        const int start = sum - mine + (warp > 0 ? carry[warp - 1] : 0);
        if (blockIdx.x == 0) {
            plan[threadIdx.x] = start;
            plan[E + threadIdx.x] = total[threadIdx.x];
        }
        base[threadIdx.x] += start;
    }
    __syncthreads();
    if (i < P) {
        int32_t row = -1;
        if (id >= 0) {
            row = base[id] + per_warp[warp * E + id] + rank;
            plan[2 * E + P + row] = static_cast<int32_t>(i);
        }
        plan[2 * E + i] = row;
    }
}

// ---------------------------------------------------------------- the sum over a token's experts
// Eight columns a thread, the slots in order, FP32 sums.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) combine_kernel(const T* __restrict__ D, int64_t ldd, const int32_t* __restrict__ row_of,
                                                      int64_t tokens, int k, int N, T* __restrict__ Y, int64_t ldy) {
    const int per_row = (N + 7) / 8;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < tokens * per_row;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = i / per_row;
        const int n = static_cast<int>(i % per_row) * 8;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const bool whole = kVec && n + 8 <= N;
        for (int j = 0; j < k; ++j) {
            const int32_t r = row_of[t * k + j];
            if (r < 0) continue;
            const T* d = D + r * ldd + n;
            if (whole) {
                T v[8];
                *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(d);
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[c] += as_float(v[c]);
            } else {
                for (int c = 0; c < 8; ++c)
                    if (n + c < N) acc[c] += as_float(d[c]);
            }
        }
        T o[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = T(acc[c]);
        T* y = Y + t * ldy + n;
        if (whole) {
            *reinterpret_cast<uint4*>(y) = *reinterpret_cast<uint4*>(o);
        } else {
            for (int c = 0; c < 8; ++c)
                if (n + c < N) y[c] = o[c];
        }
    }
}

template <typename T>
cudaError_t combine_as(const void* D, int64_t ldd, const int32_t* row_of, int64_t tokens, int k, int N, void* Y, int64_t ldy,
                       cudaStream_t stream) {
    const int64_t ctas = (tokens * ((N + 7) / 8) + 255) / 256;
    const int grid = static_cast<int>(ctas < 1 << 20 ? ctas : 1 << 20);
    const bool vec = ldd % 8 == 0 && ldy % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(D) | reinterpret_cast<uintptr_t>(Y)) & 15u) == 0;
    auto fn = vec ? combine_kernel<T, true> : combine_kernel<T, false>;
    fn<<<grid, 256, 0, stream>>>(static_cast<const T*>(D), ldd, row_of, tokens, k, N, static_cast<T*>(Y), ldy);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t stream) {
    if (a.dtype == kF32) return route_as<float>(a, stream);
    return a.dtype == kF16 ? route_as<__half>(a, stream) : route_as<__nv_bfloat16>(a, stream);
}

cudaError_t launch_moe_plan(const int32_t* ids, int64_t T, int k, int E, int32_t* plan, int32_t* counts,
                            cudaStream_t stream) {
    const int64_t P = T * k;
    const int chunks = static_cast<int>((P + kChunk - 1) / kChunk);
    if (chunks > 1) plan_count_kernel<<<chunks, kChunk, E * sizeof(int32_t), stream>>>(ids, P, E, counts);
    const int smem = E * 8 + 32 * E * 2;
    const cudaError_t e = cudaFuncSetAttribute(plan_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 * 72);
    if (e != cudaSuccess) return e;
    plan_place_kernel<<<chunks, kChunk, smem, stream>>>(ids, P, E, chunks, counts, plan, moe_rows_of(T, k, E));
    return cudaGetLastError();
}

cudaError_t launch_moe_combine(const void* D, int dtype, int64_t ldd, const int32_t* row_of, int64_t T, int k, int N,
                               void* Y, int64_t ldy, cudaStream_t stream) {
    return dtype == kF16 ? combine_as<__half>(D, ldd, row_of, T, k, N, Y, ldy, stream)
                         : combine_as<__nv_bfloat16>(D, ldd, row_of, T, k, N, Y, ldy, stream);
}

}  // namespace fmpq
