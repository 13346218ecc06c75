// Routing to experts (sm_103a): the top-k experts of each token from the router's logits, the
// plan that sorts the chosen (token, slot) pairs by expert, and the sum of the experts' outputs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fmpq_device.cuh"
#include "fmpq_internal.h"
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
    bool lanes;   // every group is a power of two of whole lanes
};

// Two keys computed in FP32 may be closer than their errors. A key's is at most 8e-7 max(1, |key|): the
// fast exponential and quotient leave 5e-7 of a score (at most 1), adding the bias rounds once. Packing
// (pack_items) takes the last 4 bits, 1.8e-6 of a key at most. Sums of two keys err by the keys' size, which may be far
// above the sum's: `size` is the largest key's. (Sums past FP32's range, whose difference is not a number, are close.)
__device__ __forceinline__ bool close_call(float hi, float lo, float step, float size = 1.0f) {
    return !(hi - lo > step * fmaxf(fmaxf(1.0f, size), fmaxf(fabsf(hi), fabsf(lo))));
}
__device__ __forceinline__ float size_of(float key) { return key > kNone ? fabsf(key) : 0.0f; }
__device__ __forceinline__ float size_of(double) { return 0.0f; }
constexpr float kStep = 3.8146973e-6f;   // 2^-18: two packed keys, or two sums of two keys
__device__ __forceinline__ bool close_call(double, double, float, float = 1.0f) { return false; }

// Whether this lane's group is among the best, from the two best keys of each lane; b2 becomes the
// group's second best. Groups are runs of `width` lanes.
template <typename V>
__device__ __forceinline__ bool keep_group(V b1, V& b2, const Rules& r, int width, int lane, bool check, bool& close) {
    for (int d = 1; d < width; d <<= 1) {
        const V o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
        const V low = b1 > o1 ? o1 : b1, second = b2 > o2 ? b2 : o2;
        b2 = low > second ? low : second;
        b1 = b1 > o1 ? b1 : o1;
    }
    const V value = r.group_top == 2 && b2 > V(kNone) ? b1 + b2 : b1;
    // its place among the groups: the number of better ones, the lower index first among equals
    const int mine = lane / width;
    int place = 0;
    for (int g = 0; g < r.groups; ++g) {
        const V o = __shfl_sync(kAll, value, g * width);
        place += (o > value || (o == value && g < mine)) ? 1 : 0;
    }
    const bool keep = place < r.top_groups && value > V(kNone);
    if (check && r.top_groups < r.groups) {
        const V worst = -warp_max(keep ? -value : V(kNone)), next = warp_max(keep ? V(kNone) : value);
        const float size = warp_max(fmaxf(size_of(b1), r.group_top == 2 ? size_of(b2) : 0.0f));
        close = next > V(kNone) && close_call(worst, next, kStep, size);
    }
    return keep;
}

// Drop the experts outside the best groups: keys of the others become -inf. Lane L holds the
// experts L * NI .. L * NI + NI - 1. Returns whether a close call decided (check only).
template <int NI, typename V>
__device__ __forceinline__ bool keep_best_groups(V (&key)[NI], const Rules& r, int lane, bool check) {
    const int per = r.E / r.groups;
    if (r.lanes) {
        // the two best keys of a lane, then of the lanes of its group
        V b1 = V(kNone), b2 = V(kNone);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const V v = key[i];
            b2 = v > b1 ? b1 : (v > b2 ? v : b2);
            b1 = v > b1 ? v : b1;
        }
        bool close = false;
        const bool keep = keep_group<V>(b1, b2, r, per / NI, lane, check, close);
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = keep ? key[i] : V(kNone);
        return close;
    }
    V mine = V(kNone);   // lane g: the value of group g
    float size = 0.0f;
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
        size = fmaxf(size, size_of(m1));
        if (r.group_top == 2) {
            const unsigned who = __ballot_sync(kAll, b1 == m1);
            if (lane == __ffs(who) - 1) b1 = b2;
            const V m2 = warp_max(b1);
            if (m2 > V(kNone)) value += m2;
            size = fmaxf(size, size_of(m2));
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
        close = next > V(kNone) && close_call(last, next, kStep, size);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane * NI + i;
        if (e < r.E && !((chosen >> (e / per)) & 1u)) key[i] = V(kNone);
    }
    return close;
}

// A lane's keys as sorted integers, largest first: the ordered key with its last bits replaced by the
// item's number counted from the end (the lowest index first among keys that agree in the rest; a
// masked key is 0). Odd-even merge sort: a comparison is one minimum and one maximum.
template <int NI>
__device__ __forceinline__ void pack_items(const float (&key)[NI], uint32_t (&item)[NI]) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
        item[i] = key[i] > kNone ? (ordered(key[i]) & ~static_cast<uint32_t>(NI - 1)) | static_cast<uint32_t>(NI - 1 - i) : 0u;
#pragma unroll
    for (int p = 1; p < NI; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < NI; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < NI && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t x = item[i + j], y = item[i + j + q];
                        item[i + j] = max(x, y);
                        item[i + j + q] = min(x, y);
                    }
}

// The k largest keys, the lowest index first among equals: lane j receives the j-th expert.
template <int NI>
__device__ __forceinline__ void take_top(const double (&key)[NI], const Rules& r, int lane, int& my_id) {
    unsigned left = (1u << NI) - 1u;   // this lane's items not taken
    for (int j = 0; j < r.k; ++j) {
        double best = static_cast<double>(kNone);
        int at = 0;
#pragma unroll 1
        for (int i = 0; i < NI; ++i)
            if (((left >> i) & 1u) && key[i] > best) { best = key[i]; at = i; }
        const double m = warp_max(best);
        if (!(m > static_cast<double>(kNone))) break;
        const int w = __ffs(__ballot_sync(kAll, best == m)) - 1;
        at = __shfl_sync(kAll, at, w);
        if (lane == w) left &= ~(1u << at);
        if (lane == j) my_id = w * NI + at;
    }
}

// The choice with keys in 64 bits, for the tokens where FP32 cannot tell.
template <typename T, int NI>
__device__ __noinline__ int choose_in_64(const T* row, const float* bias, int sigmoid, bool by_logit, float top,
                                         const Rules r, int lane) {
    double key[NI];
    double total = 0.0;
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
        const int e = lane * NI + i;
        const float x = e < r.E ? as_float(row[e]) : kNone;
        double v = static_cast<double>(kNone);
        if (x > kNone && by_logit) {
            v = static_cast<double>(x);
        } else if (x > kNone) {
            v = sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x)))
                        : (x == top ? 1.0 : exp(static_cast<double>(x) - static_cast<double>(top)));
            total += v;
        }
        key[i] = v;
    }
    total = sigmoid || by_logit ? 1.0 : warp_sum(total);
#pragma unroll 1
    for (int i = 0; i < NI; ++i)
        if (key[i] > static_cast<double>(kNone)) {
            double v = key[i] / total;
            if (bias != nullptr) v += static_cast<double>(bias[lane * NI + i]);
            key[i] = v > static_cast<double>(kNone) ? v : static_cast<double>(kNone);
        }
    if (r.groups > 1) keep_best_groups<NI, double>(key, r, lane, false);
    int id = -1;
    take_top<NI>(key, r, lane, id);
    return id;
}

// keep_group with sigmoid keys in 64 bits of the lane's items in `need` (those that may be among a
// group's two best).
template <typename T, int NI>
__device__ __noinline__ bool keep_group_in_64(const T* row, const float* bias, unsigned need, const Rules r, int lane) {
    double b1 = static_cast<double>(kNone), b2 = b1;
    while (__any_sync(kAll, need != 0u)) {
        if (need != 0u) {
            const int e = lane * NI + __ffs(need) - 1;
            double v = 1.0 / (1.0 + exp(-static_cast<double>(as_float(row[e]))));
            if (bias != nullptr) v += static_cast<double>(bias[e]);
            b2 = v > b1 ? b1 : (v > b2 ? v : b2);
            b1 = v > b1 ? v : b1;
            need &= need - 1u;
        }
        __syncwarp();
    }
    bool close = false;
    return keep_group<double>(b1, b2, r, r.E / r.groups / NI, lane, false, close);
}

// Lanes 0 .. n - 1 hold experts, their logits x and biases: sort them by the logits, or by the sigmoid keys
// in 64 bits, the lowest index first among equals.
__device__ __noinline__ void order_in_64(float x, float b, bool by_logit, int n, int lane, int& id) {
    double key = static_cast<double>(x);
    if (!by_logit) key = 1.0 / (1.0 + exp(-key)) + static_cast<double>(b);
    if (lane >= n) key = static_cast<double>(kNone);
    int place = 0, from = lane;
    for (int i = 0; i < n; ++i) {
        const double o = __shfl_sync(kAll, key, i);
        const int other = __shfl_sync(kAll, id, i);
        place += (o > key || (o == key && other < id)) ? 1 : 0;
    }
    for (int i = 0; i < n; ++i) {
        const unsigned who = __ballot_sync(kAll, lane < n && place == i);
        if (lane == i) from = __ffs(who) - 1;
    }
    id = __shfl_sync(kAll, id, from);
}

// Within 5e-7 of the sigmoid (results below the smallest normal number become 0).
__device__ __forceinline__ float fast_sigmoid(float x) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}

// A lane's NI consecutive logits.
template <typename T, int NI, bool kVec>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, float (&logit)[NI]) {
    if constexpr (kVec) {
        constexpr int kBytes = NI * static_cast<int>(sizeof(T));
        constexpr int kWidth = kBytes < 16 ? kBytes : 16;
        struct alignas(kWidth) Piece {
            T v[kWidth / sizeof(T)];
        };
#pragma unroll
        for (int i = 0; i < kBytes / kWidth; ++i) {
            const Piece w = reinterpret_cast<const Piece*>(row + lane * NI)[i];
#pragma unroll
            for (int j = 0; j < kWidth / static_cast<int>(sizeof(T)); ++j) logit[i * (kWidth / sizeof(T)) + j] = as_float(w.v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) logit[i] = lane * NI + i < E ? as_float(row[lane * NI + i]) : kNone;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) logit[i] = logit[i] > kNone ? logit[i] : kNone;   // NaN counts as masked
}

// A warp a token. NI experts a lane (E <= 32 * NI), in order, so that the lowest lane holds the
// lowest index. Each lane sorts its items once; a round then takes the largest head (one integer
// reduction and one ballot). Keys use the fast exponential; a chosen expert's weight is computed
// again, accurately, by the lane that keeps it.
// Its instructions bound it, not its bytes (16384 x 256 FP32 logits: 16.8 MB are 2.5 us at the copy rate). Measured
// there with sigmoid keys, biases, the best 4 of 8 groups and k = 8: 25 us, about 1020 warp instructions a token;
// 4099 x 60 of bf16, softmax, k = 4: 6.2 us; one token: 4.2 us, most of it the launch.
template <typename T, int NI, bool kVec>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs p, const Rules r) {
    const int lane = threadIdx.x & 31;
    const bool by_logit = p.bias == nullptr && (p.groups == 1 || p.group_top == 1);
    // 16-bit logits keep their order when packed: their last bits are the same for all
    const bool exact = by_logit && sizeof(T) == 2;
    float bias[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) bias[i] = p.bias != nullptr && lane * NI + i < p.E ? p.bias[lane * NI + i] : 0.0f;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); t < p.T;
         t += static_cast<int64_t>(gridDim.x) * 4) {
        const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
        float key[NI];
        load_logits<T, NI, kVec>(row, p.E, lane, key);
        float top = kNone, total = 1.0f;
        if (!p.sigmoid) {
#pragma unroll
            for (int i = 0; i < NI; ++i) top = fmaxf(top, key[i]);
            top = warp_max(top);
        }
        if (!by_logit || (!p.sigmoid && !p.renormalize)) {
            float score[NI];
            if (p.sigmoid) {
#pragma unroll
                for (int i = 0; i < NI; ++i) score[i] = fast_sigmoid(key[i]);
            } else {
                total = 0.0f;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    // (an infinite top takes all; equal ones share)
                    score[i] = key[i] == top ? 1.0f : __expf(key[i] - top);
                    score[i] = key[i] > kNone ? score[i] : 0.0f;
                    total += score[i];
                }
                total = warp_sum(total);
                total = total > 0.0f ? total : 1.0f;
                const float inv = 1.0f / total;
#pragma unroll
                for (int i = 0; i < NI; ++i) score[i] *= inv;
            }
            if (!by_logit) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const float v = score[i] + bias[i];
                    key[i] = key[i] > kNone && v > kNone ? v : kNone;
                }
            }
        }
        bool close = false;
        if (p.groups > 1 && r.lanes) {
            float b1 = kNone, b2 = kNone;   // the lane's two best keys
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                b2 = fmaxf(b2, fminf(b1, key[i]));
                b1 = fmaxf(b1, key[i]);
            }
            bool keep = keep_group<float>(b1, b2, r, p.E / p.groups / NI, lane, !by_logit, close);
            if (close && p.sigmoid) {
                unsigned need = 0u;
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (key[i] > kNone && (key[i] >= b2 || close_call(b2, key[i], kStep))) need |= 1u << i;
                keep = keep_group_in_64<T, NI>(row, p.bias, need, r, lane);
                close = false;
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) key[i] = keep ? key[i] : kNone;
        } else if (p.groups > 1) {
            close = keep_best_groups<NI, float>(key, r, lane, !by_logit);
        }
        uint32_t item[NI];
        pack_items<NI>(key, item);
        int id = -1;
        uint32_t mine = 0u, last = 0u;   // lane j: the j-th largest key
        int taken = 0;
        for (; taken < 32; ++taken) {
            const uint32_t head = item[0] & ~static_cast<uint32_t>(NI - 1);
            const uint32_t m = __reduce_max_sync(kAll, head);
            if (m == 0u) break;
            // past the k-th: only while it may be one of them
            if (taken >= p.k && (exact || !close_call(unordered(last), unordered(m), kStep))) break;
            last = m;
            const int w = __ffs(__ballot_sync(kAll, head == m)) - 1;   // the lowest lane with it
            const uint32_t from_end = __shfl_sync(kAll, item[0], w) & static_cast<uint32_t>(NI - 1);
            if (lane == w) {
#pragma unroll
                for (int i = 0; i + 1 < NI; ++i) item[i] = item[i + 1];
                item[NI - 1] = 0u;
            }
            if (lane == taken) {
                mine = m;
                id = w * NI + NI - 1 - static_cast<int>(from_end);
            }
        }
        // all 32 lanes taken: the next key may still be one of the k
        bool more = false;
        if (!exact && taken == 32) {
            const uint32_t m = __reduce_max_sync(kAll, item[0] & ~static_cast<uint32_t>(NI - 1));
            more = m != 0u && close_call(unordered(last), unordered(m), kStep);
        }
        float x = id >= 0 ? as_float(row[id]) : kNone;
        if (!exact) {
            // neighbours too close to tell, unless their logits and biases are equal (a true tie)
            const uint32_t next = __shfl_down_sync(kAll, mine, 1);
            const float next_x = __shfl_down_sync(kAll, x, 1);
            const float b = id >= 0 && p.bias != nullptr ? p.bias[id] : 0.0f, next_b = __shfl_down_sync(kAll, b, 1);
            const bool tight = lane < 31 && mine != 0u && next != 0u && close_call(unordered(mine), unordered(next), kStep) &&
                               !(x == next_x && b == next_b);
            const bool any = __any_sync(kAll, tight);
            if (any && !close && !more && (p.sigmoid || by_logit)) {
                // every expert that may be among the k is in a lane: put them in the order of their keys in 64 bits
                order_in_64(x, b, by_logit, taken, lane, id);
                x = id >= 0 ? as_float(row[id]) : kNone;
            } else if (any || close || more) {
                id = choose_in_64<T, NI>(row, p.bias, p.sigmoid, by_logit, top, r, lane);
                x = id >= 0 ? as_float(row[id]) : kNone;
            }
        }
        if (lane >= p.k) id = -1;
        float weight = 0.0f;
        if (id >= 0) {
            if (p.sigmoid) weight = 1.0f / (1.0f + expf(-x));
            else weight = (x == top ? 1.0f : expf(x - top)) / total;
        }
        if (p.renormalize) {
            float sum = warp_sum(weight);
            if (sum < 1e-30f) {
                // scores about or below FP32's smallest: both kinds are e^x times the same factor there, so the largest
                // is taken out of it (scores that are 0 in 64 bits too, below e^-745, stay 0)
                const float best = warp_max(id >= 0 ? x : kNone), depth = (p.sigmoid ? 0.0f : top) - best;
                if (depth < 745.0f) {
                    weight = id >= 0 ? expf(x - best) : 0.0f;
                    sum = warp_sum(weight);
                }
            }
            weight = sum > 0.0f ? weight / sum : 0.0f;
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = weight * p.scale;
        }
    }
}

template <typename T, int NI>
cudaError_t route_as(const RouteArgs& a, cudaStream_t stream) {
    const int per = a.E / a.groups, width = per / NI;
    const Rules r{a.E, a.k, a.groups, a.top_groups, a.group_top,
                  a.E == 32 * NI && per % NI == 0 && (width & (width - 1)) == 0};
    const bool vec = a.E == 32 * NI && a.ldl * static_cast<int64_t>(sizeof(T)) % 16 == 0 &&
                     (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0;
    const int64_t ctas = (a.T + 3) / 4;
    const int grid = static_cast<int>(ctas < 1216 ? ctas : 1216);   // 8 CTAs an SM: a warp keeps its biases
    if (vec) route_kernel<T, NI, true><<<grid, 128, 0, stream>>>(a, r);
    else route_kernel<T, NI, false><<<grid, 128, 0, stream>>>(a, r);
    return cudaGetLastError();
}

template <typename T>
cudaError_t route_as(const RouteArgs& a, cudaStream_t stream) {
    if (a.E <= 32) return route_as<T, 1>(a, stream);
    if (a.E <= 64) return route_as<T, 2>(a, stream);
    if (a.E <= 128) return route_as<T, 4>(a, stream);
    if (a.E <= 256) return route_as<T, 8>(a, stream);
    return route_as<T, 16>(a, stream);
}

// ---------------------------------------------------------------- the plan
// A stable counting sort of the pairs by expert, without atomics on positions: chunks of 1024
// pairs, a CTA each. With several chunks a first launch counts every chunk's pairs per expert; the
// CTA of chunk c then adds up the counts before it. Latency bounds it: 32768 pairs and 128 experts, 3.2 + 8.5 us
// (the ids and the plan are 0.4 MB); one chunk, 3.5 us. It ranks by __match_any_sync because positions taken by atomics
// would change from run to run, and with them the rows, though not the results.
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
                                                            const int32_t* __restrict__ counts, int32_t* __restrict__ plan) {
    extern __shared__ int32_t sm[];
    int32_t* total = sm;
    int32_t* base = sm + E;
    uint16_t* per_warp = reinterpret_cast<uint16_t*>(sm + 2 * E);
    __shared__ int32_t carry[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    dev::pdl_launch_dependents();   // (the quantizer after it waits for all of it)
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
__device__ __forceinline__ void load8(const float* d, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(d)[0], b = reinterpret_cast<const float4*>(d)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* d, float (&v)[8]) {
    const uint4 raw = *reinterpret_cast<const uint4*>(d);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = as_float(reinterpret_cast<const T*>(&raw)[c]);
}

// Eight columns a thread, the slots in order, FP32 sums, rounded once to T. DRAM bounds it: 4096 tokens of 8 rows of 4096
// FP32 values, 570 MB (84 us at the copy rate) in 83.5 us; of 16-bit values, 302 MB (44.5 us) in 49.7. Four rows in
// flight: one at a time, each waited for its row's number too.
template <typename S, typename T, bool kVec>
__global__ void __launch_bounds__(256) combine_kernel(const S* __restrict__ D, int64_t ldd, const int32_t* __restrict__ row_of,
                                                      int64_t tokens, int k, int N, T* __restrict__ Y, int64_t ldy) {
    dev::pdl_wait();
    dev::pdl_launch_dependents();
    const int n = static_cast<int>(blockIdx.x * 256 + threadIdx.x) * 8;
    if (n >= N) return;
    for (int64_t t = blockIdx.y; t < tokens; t += gridDim.y) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const bool whole = kVec && n + 8 <= N;
        for (int j0 = 0; j0 < k; j0 += 4) {   // four rows in flight
            int32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = j0 + j < k ? row_of[t * k + j0 + j] : -1;
            if (whole) {
                float v[4][8];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r[j] >= 0) load8(D + r[j] * ldd + n, v[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r[j] >= 0) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) acc[c] += v[j][c];
                    }
            } else {
                for (int j = 0; j < 4; ++j)
                    for (int c = 0; c < 8; ++c)
                        if (r[j] >= 0 && n + c < N) acc[c] += as_float(D[r[j] * ldd + n + c]);
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

template <typename S, typename T>
cudaError_t combine_as(const void* D, int64_t ldd, const int32_t* row_of, int64_t tokens, int k, int N, void* Y, int64_t ldy,
                       bool pdl, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(((N + 7) / 8 + 255) / 256), static_cast<unsigned>(tokens < 65535 ? tokens : 65535));
    const bool vec = ldd * static_cast<int64_t>(sizeof(S)) % 16 == 0 && ldy % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(D) | reinterpret_cast<uintptr_t>(Y)) & 15u) == 0;
    auto fn = vec ? combine_kernel<S, T, true> : combine_kernel<S, T, false>;
    return launch_after(fn, grid, 256, 0, pdl, stream, static_cast<const S*>(D), ldd, row_of, tokens, k, N,
                        static_cast<T*>(Y), ldy);
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
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(plan_place_kernel), 1024 * 72);   // E <= 1024
    if (e != cudaSuccess) return e;
    plan_place_kernel<<<chunks, kChunk, smem, stream>>>(ids, P, E, chunks, counts, plan);
    return cudaGetLastError();
}

cudaError_t launch_moe_combine(const void* D, int d_dtype, int64_t ldd, const int32_t* row_of, int64_t T, int k, int N,
                               void* Y, int dtype, int64_t ldy, bool pdl, cudaStream_t stream) {
    auto fn = d_dtype == kF32 ? (dtype == kF16 ? combine_as<float, __half> : combine_as<float, __nv_bfloat16>)
                              : (dtype == kF16 ? combine_as<__half, __half> : combine_as<__nv_bfloat16, __nv_bfloat16>);
    return fn(D, ldd, row_of, T, k, N, Y, ldy, pdl, stream);
}

}  // namespace fmpq
