// What the two E4M3 product kernels share: parameters, the tiles and their order, epilogue pieces.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fmpq_device.cuh"
#include "fmpq_internal.h"
#include "fp8_internal.h"

namespace fmpq {
namespace fp8 {

constexpr int kScChunk = 4;     // blocks of token scales per copy
constexpr int kScSlots = 3;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 384;   // 4 warps of other roles, 8 of the epilogue
constexpr int kGroupM = 8;      // dense order: bands of 8 token tiles, weight tiles inside a band
constexpr uint32_t kTmemCols = 512;

struct Params {
    const uint8_t* A;
    const uint8_t* W;
    const float* w_scales;
    const int32_t* start;      // experts (nullptr: dense)
    const int32_t* count;
    const int32_t* pair_of;
    const float* pair_weight;
    int64_t rows, sstride;
    void* Y;
    int64_t ldy;
    int bf16, f32;             // output type (neither: fp16)
    int vec;                   // columns a store may write at once: 8 (16 bits), 4 or 1
    uint8_t* H;
    float* h_scales;
    int M, N, nb, pairs, scale_rows, experts, splits;
    float* partial;            // split-K: [tile][split][CTA][warp][vector][lane] FP32 sums
    int32_t* arrivals;         // [tile][CTA]
    int32_t* status;
};

// The experts' tiles, staged in shared memory: units before each expert's, its first row and tokens.
struct Tables {
    int32_t first_unit[kMaxFp8Experts + 1], start[kMaxFp8Experts], count[kMaxFp8Experts];
};

// A unit of work: the 256 packed weight rows `pair` of expert e, `n` tokens from row `row0`, blocks
// [b0, b1).
struct Unit {
    int e, pair, n, b0, b1, tile, split;
    int64_t row0;
};

// Every thread calls it; a barrier must follow. All threads load, then warp 3 sums up the units (kT tokens
// a tile): lane l those of the run of experts [l * run, l * run + run).
template <int kT>
__device__ __forceinline__ void fill_tables(const Params& p, Tables& s, int warp, int lane) {
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) {
        s.start[e] = p.start[e];
        s.count[e] = p.count[e];
    }
    __syncthreads();
    if (warp != 3) return;
    const int run = (p.experts + 31) / 32;
    auto units_of = [&](int e) { return e < p.experts ? (s.count[e] + kT - 1) / kT * p.pairs : 0; };
    int sum = 0;
    for (int i = 0; i < run; ++i) sum += units_of(lane * run + i);
    int before = sum;
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += o;
    }
    before -= sum;
    for (int i = 0; i < run; ++i) {
        const int e = lane * run + i;
        if (e <= p.experts) s.first_unit[e] = before;
        before += units_of(e);
    }
    if (lane == 31 && p.experts == 32 * run) s.first_unit[p.experts] = before;
}

template <int kT>
__device__ __forceinline__ int unit_count(const Params& p, const Tables& s) {
    if (p.start != nullptr) return s.first_unit[p.experts];
    return p.pairs * ((p.M + kT - 1) / kT) * p.splits;
}

// An expert's (or the layer's) tokens in full tiles and a rest.
template <int kT>
__device__ __forceinline__ Unit unit_of(const Params& p, const Tables& s, int u) {
    Unit r;
    int tokens = p.M, tiles, t;
    int64_t row = 0;
    r.e = 0;
    r.split = 0;
    r.b0 = 0;
    r.b1 = p.nb;
    if (p.start != nullptr) {
        int lo = 0, hi = p.experts;   // the expert with first_unit[e] <= u < first_unit[e + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s.first_unit[mid] <= u) lo = mid;
            else hi = mid;
        }
        r.e = lo;
        tokens = s.count[lo];
        row = s.start[lo];
        tiles = (tokens + kT - 1) / kT;
        const int i = u - s.first_unit[lo];
        t = i % tiles;
        r.pair = i / tiles;
        r.tile = u;
    } else {
        tiles = (p.M + kT - 1) / kT;
        r.tile = u / p.splits;
        r.split = u % p.splits;
        const int band = r.tile / (kGroupM * p.pairs), in_band = r.tile - band * kGroupM * p.pairs;
        const int gm = min(kGroupM, tiles - band * kGroupM);
        t = band * kGroupM + in_band % gm;
        r.pair = in_band / gm;
        r.b0 = static_cast<int>(static_cast<int64_t>(r.split) * p.nb / p.splits);
        r.b1 = static_cast<int>(static_cast<int64_t>(r.split + 1) * p.nb / p.splits);
    }
    r.row0 = row + t * kT;
    r.n = min(kT, tokens - t * kT);
    return r;
}

// dev::mbar_wait on a shared-memory address.
__device__ __forceinline__ bool wait_at(uint32_t bar, uint32_t parity, const volatile int* abort) {
    for (uint32_t i = 0; i < dev::kMaxPolls; ++i) {
        uint32_t done;
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n"
            "}\n"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if ((i & 255u) == 255u && *abort) return false;
    }
    return false;
}

__device__ __forceinline__ void fail(const Params& p, volatile int* abort_flag) {
    *abort_flag = 1;
    dev::report(p.status, dev::kStatusTimeout);
}

__device__ __forceinline__ const uint8_t* weight_block(const Params& p, const Unit& t, uint32_t rank) {
    return p.W + ((static_cast<int64_t>(t.e) * p.pairs * 2 + 2 * t.pair + rank) * p.nb + t.b0) * kTileBytes;
}

// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// The larger of two magnitudes, compared as bits: NaN is above every number, so a block's scale does not lose it.
__device__ __forceinline__ float max_magnitude(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
// silu(g) * u = g u / (1 + e^-g): the exponential and the quotient to 2 of their last places, the value and the scale
// made of it within 4 steps of 2^-23 for every g. The E4M3 codes that follow change where the value crosses the middle
// between two codes, so the hardware's exponential, whose error grows with |g| (15 steps at 49), is not used: it saves
// 19 of 798 us for 4096 tokens through 8 of 128 experts of 4096 x 1024. A rounded division costs 48 more. (Where
// 1 + e^-g passes 2^126, silu(g) is below 1e-36 in magnitude, the quotient is 0.)
__device__ __forceinline__ float silu_times(float g, float u) { return __fdividef(g, 1.0f + expf(-g)) * u; }

}  // namespace fp8

// The token scales as a 2-D tensor [nb][rows]: boxes of `blocks` blocks x `tokens` rows. The codes as a
// 3-D one [nb][rows][128 bytes], boxes of kScChunk blocks x `tokens` rows.
bool encode_scale_map(CUtensorMap* map, const float* scales, int64_t sstride, int nb, int tokens, int blocks);
bool encode_code_map(CUtensorMap* map, const void* codes, int64_t rows, int nb, int tokens);

// Launch a kernel of CTA pairs; pdl: as the programmatic dependent of the launch before it.
template <typename... P, typename... A>
cudaError_t launch_pairs(void (*fn)(P...), int grid, int threads, size_t smem, bool pdl, cudaStream_t stream, const A&... args) {
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_after(fn, dim3(static_cast<unsigned>(grid)), threads, smem, pdl, stream, args...);
}

// The kernel for many tokens, with the tokens on the tensor core's M side (few_tokens chooses).
cudaError_t launch_fp8_wide(const fp8_layer& L, const fp8::Params& p, const float* a_scales, int64_t tiles, bool pdl,
                            cudaStream_t stream);
// Pairs of CTAs that are resident at once (one CTA per SM).
int fp8_resident_pairs(const fp8_layer& L);

}  // namespace fmpq
