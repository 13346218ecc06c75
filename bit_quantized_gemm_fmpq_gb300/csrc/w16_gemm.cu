// Products with weights kept in 16 bits (sm_103a): a linear layer, or experts whose rows lie one group after another,
//
//   Y[r][n] = act(sum_k X[r][k] W_e[n][k] + bias_e[n]) * row_weight[r] + residual[r][n],   e the group of row r,
//   gated: act(gate sum + bias) * (up sum + bias) in place of act(sum + bias).
//
// FP32 sums on the tensor cores (tcgen05 kind::f16, FP32 accumulators in TMEM), one rounding. A pair of CTAs computes 256
// packed weight rows (128 each, the tensor core's M side, 16 KB a block of 64 channels, laid out beforehand so that a block is
// one bulk copy) x up to 512 rows of X (the N side, 256 an MMA, half of them from each CTA, TMA boxes with the 128-byte swizzle).
// The N side takes any multiple of 32, so a group's rest costs MMAs only for its own rows, and few rows are the same
// kernel with a narrower tile and more weight blocks in flight: for one row it streams weights, for many it is bound by
// the tensor pipe.
//   * A unit's whole K is summed in TMEM; two accumulators, so that a unit's epilogue runs under the next one's MMAs (above 256 rows a
//     unit takes both, and reads its weights once).
//   * The epilogue turns 8 rows at a time through shared memory in FP32, so that a thread has 8 neighbouring outputs of a row:
//     activation, residual (16-byte loads, on their way before the sums are there) and one 16-byte store. The bias is added as the sums are
//     turned, where a thread has one weight row.
//   * Units too few for the pairs: K is split over the pairs of a cluster; the others leave their sums in the first one's
//     shared memory, which adds them in order, so results do not depend on timing. What a dense product's units leave over of full
//     rounds has a launch of its own, cut finer and along K, under the first one's end.
//
// Warp roles (640 threads, one CTA per SM, pairs persistent over units):
//   warp 0      producer of weight blocks and X boxes
//   warp 1      even CTA of a pair: MMA issuer; odd CTA: reports its operands to the even one
//   warp 2      allocates and frees TMEM
//   warp 3      sums up the groups' units
//   warps 4-19  epilogue: TMEM lane quarter warp % 4; four groups take the unit's 8-row chunks in turn
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.cuh"
#include "fmpq_device.cuh"
#include "fmpq_internal.h"
#include "pieces.cuh"
#include "w16_internal.h"

namespace fmpq {
namespace w16 {
namespace {

constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kGroups = kEpiWarps / 4;   // of epilogue warps, one for each TMEM lane quarter, that take the chunks in turn
constexpr int kMaxStages = 12;
constexpr int kPartRows = 256;    // of a part: the N side of an MMA, and an accumulator's columns
constexpr int kMostRows = 512;    // of a unit: two parts
constexpr int kChunk = 8;         // rows of X that a group turns at a time
constexpr int kStageLd = 136;     // floats of a row there: 128 outputs, and up to 7 in front of them
// Epilogues: any outputs and any split of K; put_out_whole, without a residual, with one, and for FP32.
enum { kAnyForm, kWholeBare, kWholeAdded, kWholeF32 };
constexpr int kAhead = 2;         // chunks of a group whose residual is on its way (put_out_whole), 16 bytes a thread and a row's end
constexpr int kAheadBytes = kGroups * kAhead * (128 + kChunk) * 16;
constexpr int kBandTiles = 8;     // dense order: bands of 8 row tiles, weight tiles inside a band
constexpr int kMaxSplits = 4;
constexpr int kTileChoices = kMostRows / 32;
constexpr int kBigBox = 64, kSmallBox = 16;   // rows of the two TMA boxes

struct Params {
    const uint8_t* W;
    const int32_t* start;
    const int32_t* count;
    const float* row_weight;
    const int32_t* pair_of;
    Epilogue e;
    void* Y;
    int64_t ldy;
    int bf16, f32;       // operands (and Y, unless f32) are bf16
    int vec;             // columns that Y and the residual take at once: 8, 4 (16 bits; FP32: 4 and 4), or 1
    int rows, N, out_n;  // out_n: columns of Y (gated: N / 2)
    int nb, pairs, experts, splits;
    int tile;            // rows of a unit, at most: a multiple of 32
    int most_tile;       // groups, K not split: what the device may choose (0: tile)
    int cut, cuts;       // rows of the units that a dense product's rows are cut into, and units of this launch in one of them
    int tiles;           // those units, for a pair of weight tiles
    int first_cut;       // this launch's first
    int last_launch;     // the rest of a product, behind the launch of its full rounds
    int units;           // dense: of this launch
    int others;          // bytes behind the operands' ring
    int32_t* status;
    uint32_t polls;      // (kernels with kTest) after how many polls a wait gives up,
    int withheld_cta, withheld_copy;   // and the copy of weights, counted from 0, that this CTA leaves out
};

struct Tables {
    int32_t first_unit[kMaxFp8Experts + 1], start[kMaxFp8Experts], count[kMaxFp8Experts];
    uint16_t per[kMaxFp8Experts];   // rows of its units
    int32_t units[kTileChoices], cost[kTileChoices];   // with tiles of 32, 64, ..
    int32_t tile, stages, stage_bytes;   // the operands' ring, for units of `tile` rows
};

struct __align__(1024) Smem {
    float turn[kGroups][2][kChunk][kStageLd];   // a group's chunks, two in turn
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_free[2];
    uint64_t split_full;   // first pair of a cluster: the others' sums are here
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
    Tables tables;
    // then the ring of operand stages (16 KB of weights, tile / 2 rows of X), and with K split the sums of the other pairs:
    // [split - 1][chunk][2 vectors][128 weight rows] of 4 floats, or (K not split) kAheadBytes of the residual
};
constexpr int kHeadBytes = (sizeof(Smem) + 1023) / 1024 * 1024;
constexpr int kSmemBytes = 232448;                  // 227 KB: what a CTA may use
constexpr int kRingBytes = kSmemBytes - 1024 - kHeadBytes;

// `rows` of X for the 256 weight rows `pair` of expert e, blocks [b0, b1). More than 256 rows are two parts of about half each, which
// share the weight blocks and take both accumulators.
struct Unit {
    int e, pair, rows, row0, b0, b1;
    __device__ int parts() const { return rows > kPartRows ? 2 : 1; }
    __device__ int first_rows() const { return rows > kPartRows ? ((rows + 1) / 2 + 31) & ~31 : rows; }
    __device__ int part_row0(int i) const { return i == 0 ? row0 : row0 + first_rows(); }
    __device__ int part_rows(int i) const { return i == 0 ? first_rows() : rows - first_rows(); }
    __device__ int columns(int i) const { return max(32, (part_rows(i) + 31) & ~31); }   // of the MMAs
};

// Rows of a unit where `count` rows are cut evenly into as few units as tiles of `tile` allow.
__host__ __device__ inline int even_rows(int count, int tile) {
    const int tiles = (count + tile - 1) / tile;
    return tiles == 0 ? tile : ((count + tiles - 1) / tiles + 31) / 32 * 32;
}
__host__ __device__ inline int tiles_of(int count, int per) { return (count + per - 1) / per; }

__host__ __device__ inline int stage_bytes_of(int tile) { return kTileBytes + tile / 2 * 128; }
__host__ __device__ inline int stages_of(int tile, int others) {
    const int stages = (kRingBytes - others) / stage_bytes_of(tile);
    return stages < kMaxStages ? stages : kMaxStages;
}
__device__ __forceinline__ void set_ring(const Params& p, Tables& s, int tile) {
    s.tile = tile;
    s.stage_bytes = stage_bytes_of(tile);
    s.stages = stages_of(tile, p.others);
}
// What a block of 64 channels costs a pair, in clk (shape_of has what it is made of).
__host__ __device__ inline float block_of(int rows) { return rows > kPartRows ? 2.25f * rows : 400.0f + 0.65f * rows; }

// The tile for the groups as they are (the host knows only their mean): all of a CTA's threads count the units that each tile would make, a
// choice each and every 40th group; then the one with the least time by shape_of's count. All CTAs find the same. 6436 rows of 39 of 59
// experts, 896 -> 4608: 115 to 82 us; 23784 of 60 of 66, 256 -> 10624: 225 to 216 (251 with an epilogue's 30 clk a row counted where they are
// more than the blocks). It takes about 1 us, and few rows an expert gain nothing: 357 of 36 of 55, 1408 -> 128, 12.3 to 13.1.
__device__ __forceinline__ void count_units(const Params& p, Tables& s, int lane) {
    const int i = threadIdx.x % kTileChoices, tile = 32 * (i + 1);
    int units = 0, cost = 0;
    if (tile <= p.most_tile) {
        for (int e = threadIdx.x / kTileChoices; e < p.experts; e += blockDim.x / kTileChoices) {
            const int count = s.count[e];
            if (count == 0) continue;
            const int per = even_rows(count, tile), n = tiles_of(count, per);
            units += n;
            cost += n * static_cast<int>(block_of(per) + (per > kPartRows ? 14.0f * per / p.nb : 0.0f));
        }
    }
    units += __shfl_xor_sync(0xFFFFFFFFu, units, 16);
    cost += __shfl_xor_sync(0xFFFFFFFFu, cost, 16);
    if (lane < kTileChoices) {
        atomicAdd(&s.units[i], units);
        atomicAdd(&s.cost[i], cost);
    }
}
__device__ __forceinline__ int best_tile(const Params& p, const Tables& s, int clusters, int lane) {
    const int i = lane % kTileChoices, tile = 32 * (i + 1), units = s.units[i];
    float time = 3e38f;
    if (units > 0) {
        const int rounds = (units * p.pairs + clusters - 1) / clusters;
        time = rounds * (static_cast<float>(s.cost[i]) / units) * p.nb + 14.0f * min(tile, kPartRows);
    }
    int best = tile;
    for (int d = 8; d > 0; d >>= 1) {
        const float t = __shfl_xor_sync(0xFFFFFFFFu, time, d);
        const int b = __shfl_xor_sync(0xFFFFFFFFu, best, d);
        if (t < time || (t == time && b < best)) time = t, best = b;
    }
    return best;
}

// Every thread calls it; a barrier must follow. Group bounds outside [0, rows] are cut to it, and a group begins no earlier than those
// before it end: no row is in two, so there are never more units than the host counts with.
__device__ __forceinline__ void fill_tables(const Params& p, Tables& s, int clusters, int warp, int lane) {
    if (threadIdx.x < kTileChoices) s.units[threadIdx.x] = 0, s.cost[threadIdx.x] = 0;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) {
        const int64_t from = p.start[e], to = p.count != nullptr ? from + p.count[e] : p.start[e + 1];
        const int a = static_cast<int>(min(max(from, INT64_C(0)), static_cast<int64_t>(p.rows)));
        const int b = static_cast<int>(min(max(to, INT64_C(0)), static_cast<int64_t>(p.rows)));
        s.start[e] = a;
        s.count[e] = max(0, b - a);
    }
    __syncthreads();
    if (p.most_tile > 0) {
        count_units(p, s, lane);
        __syncthreads();
    }
    if (warp != 3) return;
    const int tile = p.most_tile > 0 ? best_tile(p, s, clusters, lane) : p.tile;
    if (lane == 0) set_ring(p, s, tile);
    // lane l: the run of experts [l * run, l * run + run)
    const int run = (p.experts + 31) / 32, begin = lane * run, end = min(begin + run, p.experts);
    int last = 0;   // where the groups so far end
    for (int e = begin; e < end; ++e)
        if (s.count[e] > 0) last = max(last, s.start[e] + s.count[e]);
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, last, d);
        if (lane >= d) last = max(last, o);
    }
    last = __shfl_up_sync(0xFFFFFFFFu, last, 1);
    if (lane == 0) last = 0;
    int sum = 0;
    for (int e = begin; e < end; ++e) {
        const int cut = min(s.count[e], max(0, last - s.start[e]));
        s.start[e] += cut;
        s.count[e] -= cut;
        if (s.count[e] > 0) last = max(last, s.start[e] + s.count[e]);
        s.per[e] = static_cast<uint16_t>(even_rows(s.count[e], tile));
        const int units = tiles_of(s.count[e], s.per[e]) * p.pairs;
        s.first_unit[e] = sum;   // (of this lane's)
        sum += units;
    }
    int before = sum;
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += o;
    }
    if (lane == 31) s.first_unit[p.experts] = before;
    before -= sum;
    for (int e = begin; e < end; ++e) s.first_unit[e] += before;
}

__device__ __forceinline__ int unit_count(const Params& p, const Smem& s) {
    return p.start != nullptr ? s.tables.first_unit[p.experts] : p.units;
}

__device__ __forceinline__ Unit unit_of(const Params& p, const Smem& s, int u, int split) {
    Unit r;
    int count = p.rows, first = 0, t, per;
    r.e = 0;
    if (p.start != nullptr) {
        int lo = 0, hi = p.experts;   // the expert with first_unit[e] <= u < first_unit[e + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s.tables.first_unit[mid] <= u) lo = mid;
            else hi = mid;
        }
        r.e = lo;
        count = s.tables.count[lo];
        first = s.tables.start[lo];
        per = s.tables.per[lo];
        const uint32_t tiles = (static_cast<uint32_t>(s.tables.first_unit[lo + 1]) - s.tables.first_unit[lo]) / static_cast<uint32_t>(p.pairs);
        const uint32_t i = u - s.tables.first_unit[lo];
        r.pair = static_cast<int>(i / tiles);
        t = static_cast<int>(i - r.pair * tiles);
    } else {
        per = p.cut;
        const uint32_t v = p.first_cut + (p.cuts == 1 ? u : u / p.cuts), of_band = kBandTiles * p.pairs;
        const uint32_t band = v / of_band, in_band = v - band * of_band;
        const uint32_t high = min(kBandTiles, p.tiles - static_cast<int>(band) * kBandTiles);
        r.pair = static_cast<int>(high == kBandTiles ? in_band / kBandTiles : in_band / high);
        t = static_cast<int>(band * kBandTiles + in_band - r.pair * high);
    }
    r.row0 = first + t * per;
    r.rows = min(per, count - t * per);
    if (p.cuts > 1) {   // (nothing may be left for the last of them)
        const int skip = u % p.cuts * p.tile;
        r.row0 += skip;
        r.rows = max(0, min(p.tile, r.rows - skip));
    }
    r.b0 = p.splits == 1 ? 0 : split * p.nb / p.splits;
    r.b1 = p.splits == 1 ? p.nb : (split + 1) * p.nb / p.splits;
    return r;
}

__device__ __forceinline__ void fail(const Params& p, volatile int* abort_flag) {
    *abort_flag = 1;
    dev::report(p.status, dev::kStatusTimeout);
}
// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// Where a CTA stands: its number in the cluster, in its pair, the pair's first CTA, the pair's K split, the cluster.
struct Place {
    uint32_t cluster_rank, rank, leader;
    int split, cluster, clusters;
};

// ---------------------------------------------------------------- producer (warp 0)
template <bool kTest>
__device__ __forceinline__ void producer(const Params& p, const CUtensorMap* big, const CUtensorMap* small, Smem& s, uint8_t* ring,
                                         const Place& at, volatile int* abort_flag) {
    const uint32_t polls = kTest ? p.polls : dev::kMaxPolls;
    const bool withholds = kTest && static_cast<int>(blockIdx.x) == p.withheld_cta;
    const int units = unit_count(p, s);
    const uint32_t stages = s.tables.stages, stage_bytes = s.tables.stage_bytes;
    uint32_t it = 0, st = 0, phase = 1;
    bool ok = true;
    for (int u = at.cluster; ok && u < units; u += at.clusters) {
        const Unit t = unit_of(p, s, u, at.split);
        if (t.rows == 0) continue;
        // this CTA's half of each part's rows
        const int parts = t.parts(), half0 = t.columns(0) >> 1, half1 = parts > 1 ? t.columns(1) >> 1 : 0;
        const int from0 = t.part_row0(0) + static_cast<int>(at.rank) * half0, from1 = t.part_row0(1) + static_cast<int>(at.rank) * half1;
        const uint8_t* w = p.W + (((static_cast<int64_t>(t.e) * p.pairs + t.pair) * 2 + at.rank) * p.nb + t.b0) * kTileBytes;
        for (int b = t.b0; b < t.b1; ++b, ++it, w += kTileBytes) {
            ok = __all_sync(0xFFFFFFFFu, dev::mbar_wait(&s.empty[st], phase, abort_flag, polls));
            if (!ok) break;
            if (elect_one()) {
                uint64_t* bar = &s.full[st];
                uint8_t* to = ring + st * stage_bytes;
                dev::mbar_arrive_expect_tx(bar, kTileBytes + (half0 + half1) * 128u);
                if (!withholds || static_cast<int>(it) != p.withheld_copy) dev::bulk_g2s(to, w, kTileBytes, bar);
                to += kTileBytes;
                auto rows_to = [&](int half, int row) {
                    int i = 0;
                    for (; i + kBigBox <= half; i += kBigBox) dev::tma_load_2d(to + i * 128, big, b * kW16Block, row + i, bar);
                    for (; i < half; i += kSmallBox) dev::tma_load_2d(to + i * 128, small, b * kW16Block, row + i, bar);
                    to += half * 128;
                };
                rows_to(half0, from0);
                rows_to(half1, from1);
            }
            __syncwarp();
            if (++st == stages) {
                st = 0;
                phase ^= 1;
            }
        }
    }
    if (!ok && elect_one()) fail(p, abort_flag);
    // the copies in flight must land before the CTA's shared memory is given up
    for (uint32_t k = 0; k < stages && k < it; ++k) {
        const uint32_t i = it - 1 - k;
        dev::mbar_drain(&s.full[i % stages], (i / stages) & 1, abort_flag, polls);
    }
}

// ---------------------------------------------------------------- MMA (warp 1)
// kind::f16, A and B both F16 or both BF16, D = F32, both K-major.
__device__ __forceinline__ uint32_t idesc16(uint32_t M, uint32_t N, uint32_t bf16) {
    return (1u << 4) | (bf16 << 7) | (bf16 << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the barrier at `bar`'s offset in both CTAs of this pair once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t leader) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            dev::smem_u32(bar)),
        "h"(static_cast<uint16_t>(3u << leader))
        : "memory");
}

template <bool kTest>
__device__ __forceinline__ void mma_issuer(const Params& p, Smem& s, uint8_t* ring, const Place& at, uint32_t tmem,
                                           volatile int* abort_flag) {
    const uint32_t polls = kTest ? p.polls : dev::kMaxPolls;
    const uint32_t stages = s.tables.stages, stage_bytes = s.tables.stage_bytes;
    const int units = unit_count(p, s);
    const uint32_t remote = dev::mapa(&s.full[0], at.leader);
    const uint64_t w0 = dev::sdesc_k_sw128(dev::smem_u32(ring));
    uint32_t st = 0, phase = 0, np = 0;   // np: parts so far; accumulator np & 1 is the next one's
    bool ok = true;
    for (int u = at.cluster; ok && u < units; u += at.clusters) {
        const Unit t = unit_of(p, s, u, at.split);
        if (t.rows == 0) continue;
        const int parts = t.parts();
        const uint32_t idesc0 = idesc16(256, static_cast<uint32_t>(t.columns(0)), static_cast<uint32_t>(p.bf16));
        const uint32_t idesc1 = idesc16(256, static_cast<uint32_t>(t.columns(1)), static_cast<uint32_t>(p.bf16));
        const uint32_t acc = np & 1, d0 = tmem + acc * kPartRows, d1 = tmem + (acc ^ 1) * kPartRows;
        const uint32_t to1 = static_cast<uint32_t>(t.columns(0)) * 4;   // the second part's rows in a stage, in 16 bytes
        if (at.rank == 0) {
            bool free = dev::mbar_wait(&s.acc_free[acc], ((np >> 1) & 1) ^ 1, abort_flag, polls);
            if (parts > 1) free = free && dev::mbar_wait(&s.acc_free[acc ^ 1], (((np + 1) >> 1) & 1) ^ 1, abort_flag, polls);
            ok = __all_sync(0xFFFFFFFFu, free);
            if (!ok) break;
        }
        for (int b = t.b0; b < t.b1; ++b) {
            ok = __all_sync(0xFFFFFFFFu, dev::mbar_wait(&s.full[st], phase, abort_flag, polls));
            if (!ok) break;
            if (at.rank != 0) {
                if (elect_one()) dev::mbar_arrive_remote(remote + st * 8u);
            } else {
                dev::tc_fence_after();
                // (a descriptor's address field counts 16 bytes)
                const uint64_t ad = w0 + st * (stage_bytes >> 4), bd = ad + kTileBytes / 16;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_16_pair(d0, ad + 2 * k, bd + 2 * k, idesc0, b > t.b0 || k > 0 ? 1u : 0u);
                    if (parts > 1)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_16_pair(d1, ad + 2 * k, bd + to1 + 2 * k, idesc1, b > t.b0 || k > 0 ? 1u : 0u);
                    commit_pair(&s.empty[st], at.leader);
                    if (b + 1 == t.b1) {
                        commit_pair(&s.acc_full[acc], at.leader);
                        if (parts > 1) commit_pair(&s.acc_full[acc ^ 1], at.leader);
                    }
                }
            }
            __syncwarp();
            if (++st == stages) {
                st = 0;
                phase ^= 1;
            }
        }
        np += parts;
    }
    if (elect_one()) {
        if (!ok) fail(p, abort_flag);
        if (at.rank == 0) {   // every MMA must finish before TMEM is released
            commit_pair(&s.mma_done, at.leader);
            dev::mbar_wait(&s.mma_done, 0, nullptr);
        }
    }
    __syncwarp();
}

// ---------------------------------------------------------------- epilogue (warps 4-19)

// kW (8, or 4 of a gated layer) neighbouring outputs of a row, from column n on (columns of them exist): 16 bits or FP32, in
// accesses of p.vec columns.
template <int kW>
__device__ __forceinline__ void store_piece(const Params& p, int64_t row, int n, int columns, const float (&f)[kW]) {
    if (p.f32) {
        float* y = static_cast<float*>(p.Y) + row * p.ldy + n;
#pragma unroll
        for (int i = 0; i < kW; i += 4) {
            if (columns >= kW) *reinterpret_cast<float4*>(y + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
            else
#pragma unroll
                for (int j = i; j < i + 4; ++j)
                    if (j < columns) y[j] = f[j];
        }
        return;
    }
    uint16_t* y = static_cast<uint16_t*>(p.Y) + row * p.ldy + n;
    uint32_t o[kW / 2];
#pragma unroll
    for (int i = 0; i < kW / 2; ++i) {
        if (p.bf16) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
            const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    if (columns < kW) {
#pragma unroll
        for (int i = 0; i < kW; ++i)
            if (i < columns) y[i] = static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1)));
    } else if (kW == 8 && p.vec == 8) {
        *reinterpret_cast<uint4*>(y) = make_uint4(o[0], o[1], o[kW / 2 - 2], o[kW / 2 - 1]);
    } else {
#pragma unroll
        for (int i = 0; i < kW; i += 4) *reinterpret_cast<uint2*>(y + i) = make_uint2(o[i / 2], o[i / 2 + 1]);
    }
}
// The residual there, as it is in memory: 16 bits in raw[0 .. kW / 2 - 1], FP32 in all of it.
template <int kW>
__device__ __forceinline__ void load_residual(const Params& p, int64_t row, int n, int columns, uint32_t (&raw)[kW]) {
    if (p.f32) {
        const uint32_t* r = static_cast<const uint32_t*>(p.e.residual) + row * p.e.ldr + n;
#pragma unroll
        for (int i = 0; i < kW; i += 4) {
            if (columns >= kW) {
                const uint4 a = *reinterpret_cast<const uint4*>(r + i);
                raw[i] = a.x, raw[i + 1] = a.y, raw[i + 2] = a.z, raw[i + 3] = a.w;
            } else {
#pragma unroll
                for (int j = i; j < i + 4; ++j) raw[j] = j < columns ? r[j] : 0u;
            }
        }
        return;
    }
    const uint16_t* r = static_cast<const uint16_t*>(p.e.residual) + row * p.e.ldr + n;
    if (columns < kW) {
#pragma unroll
        for (int i = 0; i < kW / 2; ++i)
            raw[i] = (2 * i < columns ? r[2 * i] : 0u) | (2 * i + 1 < columns ? static_cast<uint32_t>(r[2 * i + 1]) << 16 : 0u);
    } else if (kW == 8 && p.vec == 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(r);
        raw[0] = a.x, raw[1] = a.y, raw[2] = a.z, raw[3] = a.w;
    } else {
#pragma unroll
        for (int i = 0; i < kW; i += 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(r + i);
            raw[i / 2] = a.x, raw[i / 2 + 1] = a.y;
        }
    }
}
template <int kW>
__device__ __forceinline__ void add_residual(const Params& p, const uint32_t (&raw)[kW], float (&f)[kW]) {
    if (p.f32) {
#pragma unroll
        for (int i = 0; i < kW; ++i) f[i] += __uint_as_float(raw[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < kW / 2; ++i) {
        const float2 a = epi::values16(raw[i], p.bf16 != 0);
        f[2 * i] += a.x;
        f[2 * i + 1] += a.y;
    }
}
template <int kW>
__device__ __forceinline__ void activate_piece(int act, float (&f)[kW]) {
    auto all = [&](auto one) {
#pragma unroll
        for (int i = 0; i < kW; ++i) f[i] = one(f[i]);
    };
    if (act == kActRelu) all([](float v) { return epi::activate(kActRelu, v); });
    else if (act == kActSilu) all([](float v) { return epi::activate(kActSilu, v); });
    else if (act == kActGelu) all([](float v) { return epi::activate(kActGelu, v); });
    else if (act == kActGeluTanh) all([](float v) { return epi::activate(kActGeluTanh, v); });
}
__device__ __forceinline__ float weight_of(const Params& p, int64_t row) {
    return __ldg(p.row_weight + (p.pair_of != nullptr ? __ldg(p.pair_of + row) : row));
}
// One output, and its residual.
__device__ __forceinline__ void store1(const Params& p, int64_t row, int n, float f) {
    const int64_t at = row * p.ldy + n;
    if (p.f32) static_cast<float*>(p.Y)[at] = f;
    else static_cast<uint16_t*>(p.Y)[at] = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
}
__device__ __forceinline__ uint32_t residual1(const Params& p, int64_t row, int n) {
    const int64_t at = row * p.e.ldr + n;
    return p.f32 ? static_cast<const uint32_t*>(p.e.residual)[at] : static_cast<const uint16_t*>(p.e.residual)[at];
}
// Where a chunk's sums of another pair begin for a weight row (16 bytes each).
__device__ __forceinline__ int other_sums(const Params& p, int split, int chunk, int row) {
    return ((split - 1) * (p.tile / kChunk) + chunk) * (kChunk / 4) * 128 + row;
}

// Of outputs of 16 bits that rows may hold anywhere (gated: on 8-byte boundaries): where a thread's piece of a row lies. A CTA's row of
// kCols columns begins `past` elements behind a boundary, and a piece is kW elements between two boundaries; the first thread's is the row's
// two ends: its last `past` columns and its first kW - past. (Rows kW apart begin at the same place of their pieces, so it is the same in each chunk.)
template <int kW, int kCols>
struct Piece {
    int first, columns;   // the column of its first element (negative: the row's last ones), how many columns there are
    bool whole;           // all of it exists, in a row

    __device__ __forceinline__ Piece(int i, int past, int columns) : first(kW * i - past), columns(columns), whole(first >= 0 && first + kW <= columns) {}
    __device__ __forceinline__ int column(int c) const { return first + c < 0 ? first + c + kCols : first + c; }
    __device__ __forceinline__ bool has(int c) const { return column(c) < columns; }
};
// Elements between the 16-byte boundary before a row's outputs and them.
template <bool kNone>   // the rows are known to start on boundaries
__device__ __forceinline__ int row_past(const Params& p, int64_t row) {
    const uint32_t first = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.Y) >> 1) + static_cast<uint32_t>(row) * static_cast<uint32_t>(p.ldy);
    return kNone ? 0 : static_cast<int>(first & 7u);
}

// The epilogue's chunks of a part: outputs of 16 bits (or FP32), K not split. What costs time here is a group's chain through a chunk (TMEM, shared
// memory, barrier, output) and the size of the loop's code, so the rows are shifted to their place in memory as they are turned, the residual
// of a thread's next two rows is on its way by cp.async (no register waits for it), and this is a kernel of its own, with a residual or
// without. 8192 x 512 -> 4096 bf16: plain 33 us, with bias, silu and residual 51 (by the form below, with a bias for each of a piece's
// columns, 49 and 91); 4096 x 1024 -> 4096 31 and 36 (35 and 53), -> 4095 35 and 44 (57 and 88). No faster: the residual 3 or 4
// rows ahead, or its lines sent for to the L2 before; two chunks a turn of the loop (8192 x 512: 51 and 79); one kernel for both (38 and 55).
// FP32 outputs on 16-byte boundaries without a residual go the same way (8192 x 512 -> 4096 52 to 45, 32768 x 512 -> 2000 in 64 groups 104 to 92).
template <bool kGated, int kForm, int kW, int kCols, typename Wait>
__device__ __forceinline__ void put_out_whole(const Params& p, float (*turn)[kChunk][kStageLd], uint8_t* residuals, uint32_t from_tmem, int g, int tid, int64_t row0, int rows,
                                              int n0, const Piece<kW, kCols>& piece, float bias, const Wait& wait, int& buffer) {
    constexpr bool kAdded = kForm == kWholeAdded, kF32 = kForm == kWholeF32;
    constexpr int kPieces = kCols / kW;
    const int chunks = (rows + kChunk - 1) / kChunk, sub = tid / kPieces, i = tid % kPieces;
    // of every 32 packed rows of a gated layer, 16 are gates and 16 the ups of the same hidden channels
    const int place = kGated ? 32 * (kW * i >> 4) + (kW * i & 15) : kW * i;
    int to[kChunk];
#pragma unroll
    for (int j = 0; j < kChunk; ++j) to[j] = j * kStageLd + tid + row_past<kGated || kF32>(p, row0 + j);
    int64_t row = row0 + kChunk * g + sub;
    using Out = std::conditional_t<kF32, float, uint16_t>;
    Out* y = static_cast<Out*>(p.Y) + row * p.ldy + n0;
    const uint16_t* r = static_cast<const uint16_t*>(p.e.residual) + row * p.e.ldr + n0;
    const int64_t y_step = p.ldy * (kGroups * kChunk), r_step = p.e.ldr * (kGroups * kChunk);
    int left = rows - kChunk * g - sub;   // this thread's row of a chunk exists where more than 0 are left
    uint32_t d[kChunk];
    // the residual's pieces of this thread's next rows (whole ones, which hold one of the piece's elements at least), and for the first thread
    // of a row those of its last columns
    const bool head = max(piece.first, 0) < piece.columns, tail = piece.first < 0 && piece.first + kCols < piece.columns;
    uint4* slot = reinterpret_cast<uint4*>(residuals) + g * kAhead * 128 + tid;
    uint4* ends = reinterpret_cast<uint4*>(residuals) + kGroups * kAhead * 128 + g * kAhead * kChunk + sub;
    auto ask = [&](int i, int left) {
        if (left > 0 && head) dev::cp_async_if<2 * kW>(dev::smem_u32(slot + i * 128), r + piece.first, true);
        if (left > 0 && tail) dev::cp_async_if<2 * kW>(dev::smem_u32(ends + i * kChunk), r + piece.first + kCols, true);
        dev::cp_async_commit();
        r += r_step;
    };
    const bool bf16 = p.bf16 != 0;
    if (kAdded)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ask(i, left - i * kGroups * kChunk);
    int turns = 0;   // so far
    if (!wait()) left = 0;
    dev::tmem_ld8(from_tmem + kChunk * min(g, chunks - 1), d);
#pragma unroll 1
    for (int c = g; c < chunks; c += kGroups) {
        float* here = &turn[buffer][0][0];
        buffer ^= 1;
        dev::tmem_ld_wait8(d);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) here[to[j]] = __uint_as_float(d[j]) + bias;
        // (whoever writes this buffer again has passed the next barrier, behind which the others have read it)
        dev::named_bar_sync(2 + g, 128);
        dev::tmem_ld8(from_tmem + kChunk * min(c + kGroups, chunks - 1), d);
        const int held = turns++ % kAhead;   // where this row's residual is
        if (kAdded) dev::cp_async_wait<kAhead - 1>();
        if (left > 0) {
            const float* from = here + sub * kStageLd + place;
            float f[kW];
#pragma unroll
            for (int i = 0; i < kW; i += 4) *reinterpret_cast<float4*>(&f[i]) = *reinterpret_cast<const float4*>(from + i);
            if (!kGated && piece.first < 0) {
                float e[kW];
#pragma unroll
                for (int i = 0; i < kW; i += 4) *reinterpret_cast<float4*>(&e[i]) = *reinterpret_cast<const float4*>(from + kCols + i);
#pragma unroll
                for (int c = 0; c < kW; ++c) f[c] = piece.first + c < 0 ? e[c] : f[c];
            }
            activate_piece(p.e.act, f);
            if constexpr (kGated) {
                const float4 v = *reinterpret_cast<const float4*>(from + 16);
                const float up[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < kW; ++i) f[i] *= up[i];
            }
            if (p.row_weight != nullptr) {
                const float w = weight_of(p, row);
#pragma unroll
                for (int i = 0; i < kW; ++i) f[i] *= w;
            }
            if (kAdded) {
                const uint4 now = slot[held * 128];
                uint32_t raw[4] = {now.x, now.y, now.z, now.w};
                if (!kGated && piece.first < 0) {
                    const uint4 last = ends[held * kChunk];
                    const uint32_t e[4] = {last.x, last.y, last.z, last.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        raw[c] = (piece.first + 2 * c < 0 ? e[c] & 0xFFFFu : raw[c] & 0xFFFFu) | (piece.first + 2 * c + 1 < 0 ? e[c] & 0xFFFF0000u : raw[c] & 0xFFFF0000u);
                }
#pragma unroll
                for (int c = 0; c < kW / 2; ++c) {
                    const float2 a = epi::values16(raw[c], bf16);
                    f[2 * c] += a.x;
                    f[2 * c + 1] += a.y;
                }
            }
            if constexpr (kF32) {
                if (piece.whole) {
#pragma unroll
                    for (int i = 0; i < kW; i += 4) *reinterpret_cast<float4*>(y + piece.first + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
                } else {
#pragma unroll
                    for (int c = 0; c < kW; ++c)
                        if (piece.has(c)) y[piece.column(c)] = f[c];
                }
            } else {
                uint32_t o[kW / 2];
#pragma unroll
                for (int i = 0; i < kW / 2; ++i) {
                    if (bf16) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                        o[i] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                        o[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
                if (!kGated && piece.first == -4 && piece.columns == kCols) {
                    *reinterpret_cast<uint2*>(y) = make_uint2(o[kW / 2 - 2], o[kW / 2 - 1]);
                    *reinterpret_cast<uint2*>(y + kCols - 4) = make_uint2(o[0], o[1]);
                } else if (!piece.whole) {
#pragma unroll
                    for (int c = 0; c < kW; ++c)
                        if (piece.has(c)) y[piece.column(c)] = static_cast<uint16_t>(o[c >> 1] >> (16 * (c & 1)));
                } else if constexpr (kW == 8) {
                    *reinterpret_cast<uint4*>(y + piece.first) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
                    *reinterpret_cast<uint2*>(y + piece.first) = make_uint2(o[0], o[1]);
                }
            }
        }
        if (kAdded) ask(held, left - kAhead * kGroups * kChunk);
        y += y_step;
        row += kGroups * kChunk;
        left -= kGroups * kChunk;
    }
    dev::tmem_ld_wait8(d);   // (the last one's is of no use)
}

// Any outputs, any split of K: a thread's sums, a chunk's 8 rows for one packed weight row, go through shared memory; then it has one piece of neighbouring
// columns of one row: 8, or gate and up of 4 hidden channels. Where rows of Y or of the residual do not start on 8-byte boundaries
// (FP32: 16) a thread has one column instead, of all 8 rows (gated: of 4), so that a warp's accesses are still neighbours. A chunk's
// sums leave TMEM while the chunk before is put out.
template <bool kGated, int kForm, bool kTest>
__device__ __forceinline__ void epilogue(const Params& p, Smem& s, float4* others, const Place& at, int warp, int lane, uint32_t tmem,
                                         volatile int* abort_flag) {
    constexpr bool kWhole = kForm != kAnyForm;
    const uint32_t polls = kTest ? p.polls : dev::kMaxPolls;
    constexpr int kCols = kGated ? 64 : 128;              // of this CTA
    constexpr int kW = kCols * kChunk / 128, kPieces = kCols / kW;
    constexpr int kColumnRows = 128 / kCols;              // rows that the threads cover at once, a column each
    const int units = unit_count(p, s);
    const int q = warp & 3, g = (warp - 4) >> 2, tid = 32 * q + lane;
    const bool pieces = p.vec > 1;
    // column inside the CTA's, first row of a chunk, and the place of the column's gate in a turned row: of every 32 packed rows, 16
    // are gates and 16 the ups of the same hidden channels
    const int col = pieces ? tid % kPieces * kW : tid % kCols, sub = pieces ? tid / kPieces : tid / kCols;
    const int place = kGated ? 32 * (col >> 4) + (col & 15) : col;
    const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t leader_free = dev::mapa(&s.acc_free[0], at.leader);
    const bool first = kWhole || at.split == 0;
    uint32_t np = 0;   // parts so far
    bool ok = true;
    int part = 0, buffer = 0;   // (of turn: which a chunk writes)
    for (int u = at.cluster; u < units; ++np) {
        const Unit whole = unit_of(p, s, u, at.split);
        if (whole.rows == 0) {
            u += at.clusters;
            --np;
            continue;
        }
        struct {
            int e, pair, rows, row0;
        } const t{whole.e, whole.pair, whole.part_rows(part), whole.part_row0(part)};
        if (++part == whole.parts()) {
            part = 0;
            u += at.clusters;
        }
        const uint32_t acc = np & 1;
        const int n0 = (2 * t.pair + static_cast<int>(at.rank)) * kCols, n = n0 + col;
        const int columns = p.out_n - n;
        const Piece<kW, kCols> piece(tid % kPieces, kWhole ? row_past<kGated || kForm == kWholeF32>(p, t.row0 + tid / kPieces) : 0, min(kCols, p.out_n - n0));
        const int chunks = (t.rows + kChunk - 1) / kChunk;
        float bias = -0.0f;   // of this thread's packed row: added to its sums (-0: nothing is)
        if (first && p.e.bias != nullptr) {
            const int c = kGated ? n0 + 16 * (tid >> 5) + (tid & 15) : n0 + tid;   // (16 gates, 16 ups)
            if (c < p.out_n) bias = epi::bias_at(p.e, static_cast<int64_t>(t.e) * p.N + (kGated && (tid & 16) != 0 ? p.out_n : 0) + c, p.bf16 != 0);
        }
        if (!kWhole && first && p.e.residual != nullptr) {   // the part's lines of the residual to the L2, under its MMAs
            const int size = p.f32 ? 4 : 2, bytes = min(kCols, p.out_n - n0) * size;
            for (int r = (warp - 4) * 32 + lane; r < t.rows; r += kEpiWarps * 32) {
                const uint8_t* line = static_cast<const uint8_t*>(p.e.residual) + ((static_cast<int64_t>(t.row0) + r) * p.e.ldr + n0) * size;
                for (int b = 0; b < bytes; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + b));
                if (bytes > 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + bytes - 1));
            }
        }
        auto wait = [&] {
            ok = ok && dev::mbar_wait(&s.acc_full[acc], (np >> 1) & 1, abort_flag, polls);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!kWhole && first && p.splits > 1 && ok) ok = __all_sync(0xFFFFFFFFu, dev::mbar_wait_cluster(&s.split_full, 0, polls));
            dev::tc_fence_after();
            return ok;
        };
        const uint32_t from_tmem = base + acc * kPartRows;
        if (!kWhole) wait();

        if constexpr (kWhole) {
            put_out_whole<kGated, kForm>(p, s.turn[g], reinterpret_cast<uint8_t*>(others), from_tmem, g, tid, t.row0, t.rows, n0, piece, bias, wait, buffer);
        } else if (!first) {   // to the first pair's CTA of this rank
            const uint32_t to = dev::mapa(others, at.rank) + other_sums(p, at.split, 0, tid) * 16u;
            for (int c = g; c < chunks; c += kGroups) {
                uint32_t d[kChunk];
                dev::tmem_ld8(from_tmem + kChunk * c, d);
                dev::tmem_ld_wait8(d);
                if (!ok) continue;
#pragma unroll
                for (int v = 0; v < kChunk / 4; ++v)
                    dev::st_cluster_v4(to + (c * (kChunk / 4) + v) * 128 * 16u, __uint_as_float(d[4 * v]), __uint_as_float(d[4 * v + 1]),
                                       __uint_as_float(d[4 * v + 2]), __uint_as_float(d[4 * v + 3]));
            }
        } else {
            const bool mine = ok && columns > 0;
            // one chunk behind the sums
            auto put_out = [&](int c, const float (*turn)[kStageLd]) {
                const int rows = t.rows - kChunk * c;   // of this chunk, and behind
                const int64_t row0 = static_cast<int64_t>(t.row0) + kChunk * c;
                if (!mine) return;
                if (pieces) {
                    if (sub >= rows) return;
                    uint32_t raw[kW];
                    if (p.e.residual != nullptr) load_residual(p, row0 + sub, n, columns, raw);
                    const float* from = &turn[sub][place];
                    float f[kW];
#pragma unroll
                    for (int i = 0; i < kW; i += 4) *reinterpret_cast<float4*>(&f[i]) = *reinterpret_cast<const float4*>(from + i);
                    activate_piece(p.e.act, f);
                    if constexpr (kGated) {
                        const float4 v = *reinterpret_cast<const float4*>(from + 16);
                        const float up[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < kW; ++i) f[i] *= up[i];
                    }
                    if (p.row_weight != nullptr) {
                        const float w = weight_of(p, row0 + sub);
#pragma unroll
                        for (int i = 0; i < kW; ++i) f[i] *= w;
                    }
                    if (p.e.residual != nullptr) add_residual(p, raw, f);
                    store_piece(p, row0 + sub, n, columns, f);
                    return;
                }
                uint32_t raw[kW];
                if (p.e.residual != nullptr)
#pragma unroll
                    for (int i = 0; i < kW; ++i)
                        if (sub + kColumnRows * i < rows) raw[i] = residual1(p, row0 + sub + kColumnRows * i, n);
                float f[kW];
#pragma unroll
                for (int i = 0; i < kW; ++i) f[i] = turn[sub + kColumnRows * i][place];
                activate_piece(p.e.act, f);
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    const int j = sub + kColumnRows * i;
                    if (j >= rows) continue;
                    if constexpr (kGated) f[i] *= turn[j][place + 16];
                    if (p.row_weight != nullptr) f[i] *= weight_of(p, row0 + j);
                    if (p.e.residual != nullptr) f[i] += p.f32 ? __uint_as_float(raw[i]) : epi::value16(static_cast<uint16_t>(raw[i]), p.bf16 != 0);
                    store1(p, row0 + j, n, f[i]);
                }
            };
            for (int c = g; c < chunks + kGroups; c += kGroups) {
                uint32_t d[kChunk];
                const int here = min(c, chunks - 1);   // (the last turn only puts out: its load is of no use, and not behind a branch)
                dev::tmem_ld8(from_tmem + kChunk * here, d);
                if (c >= kGroups) put_out(c - kGroups, s.turn[g][buffer ^ 1]);
                dev::tmem_ld_wait8(d);
                float f[kChunk];
#pragma unroll
                for (int j = 0; j < kChunk; ++j) f[j] = __uint_as_float(d[j]);
                for (int sp = 1; sp < p.splits; ++sp) {
                    const float4* from = others + other_sums(p, sp, here, tid);
#pragma unroll
                    for (int v = 0; v < kChunk / 4; ++v) {
                        const float4 o = from[v * 128];
                        f[4 * v] += o.x, f[4 * v + 1] += o.y, f[4 * v + 2] += o.z, f[4 * v + 3] += o.w;
                    }
                }
#pragma unroll
                for (int j = 0; j < kChunk; ++j) s.turn[g][buffer][j][tid] = f[j] + bias;
                // (whoever writes this buffer again has passed the next barrier, behind which the others have read it)
                dev::named_bar_sync(2 + g, 128);
                buffer ^= 1;
            }
        }
        // all of it has been read: the accumulator is free
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive_remote(leader_free + acc * 8u);
        if (!first) {
            __syncwarp();
            if (lane == 0 && ok) dev::mbar_arrive_remote_release(dev::mapa(&s.split_full, at.rank));
        }
    }
    if (kForm == kWholeAdded) dev::cp_async_wait_all();   // (none is under way but after a wait that gave up)
    if (!ok && lane == 0) fail(p, abort_flag);
}

// kTest: the failure-detection test (Params::polls); the others bound every wait by dev::kMaxPolls.
template <bool kGated, int kForm, bool kTest = false>
__global__ void __launch_bounds__(kThreads, 1)
w16_kernel(const Params p, const __grid_constant__ CUtensorMap big, const __grid_constant__ CUtensorMap small) {
    extern __shared__ uint8_t smem_raw[];
    // (an offset from the array, so that the compiler still knows the accesses to be shared memory's)
    uint8_t* head = smem_raw + ((1024u - (dev::smem_u32(smem_raw) & 1023u)) & 1023u);
    Smem& s = *reinterpret_cast<Smem*>(head);
    uint8_t* ring = head + kHeadBytes;
    float4* others = reinterpret_cast<float4*>(ring + kRingBytes - p.others);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Place at;
    at.cluster_rank = dev::cluster_ctarank();
    at.rank = at.cluster_rank & 1;
    at.leader = at.cluster_rank & ~1u;
    at.split = static_cast<int>(at.cluster_rank >> 1);
    at.cluster = static_cast<int>(blockIdx.x) / (2 * p.splits);
    at.clusters = static_cast<int>(gridDim.x) / (2 * p.splits);
    if (threadIdx.x == 0) {
        dev::tma_prefetch_map(&big);
        dev::tma_prefetch_map(&small);
        for (int i = 0; i < kMaxStages; ++i) {
            dev::mbar_init(&s.full[i], at.rank == 0 ? 2 : 1);
            dev::mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            dev::mbar_init(&s.acc_full[i], 1);
            dev::mbar_init(&s.acc_free[i], 2 * kEpiWarps);
        }
        dev::mbar_init(&s.split_full, kEpiWarps * (p.splits > 1 ? p.splits - 1 : 1));
        dev::mbar_init(&s.mma_done, 1);
        s.abort_flag = 0;
        dev::fence_barrier_init();
    }
    if (warp == 2) dev::tmem_alloc_pair(&s.tmem_base, 512);
    // (launched as the programmatic dependent of whatever is before it: everything up to here runs under that one's end. The rest
    // of a product works before it waits for the launch before it, the full rounds. Two conditions make that sound: every thread of the full rounds
    // triggers behind its own wait, so that all before them is done and seen when the rest starts; and the rest reads nothing that they write,
    // and writes other units. Its own wait and trigger come last, so whatever is launched behind it finds both done. A trigger ahead of the wait here, or a rest
    // that reads an output of the full rounds, would be a race.)
    if (p.last_launch) {
        __threadfence();
    } else {
        dev::pdl_wait();
        dev::pdl_launch_dependents();
    }
    if (p.start != nullptr) fill_tables(p, s.tables, at.clusters, warp, lane);
    else if (threadIdx.x == 0) set_ring(p, s.tables, p.tile);
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // every CTA's barriers and TMEM exist before any traffic between them
    dev::tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    volatile int* abort_flag = &s.abort_flag;

    if (warp == 0) {
        producer<kTest>(p, &big, &small, s, ring, at, abort_flag);
    } else if (warp == 1) {
        mma_issuer<kTest>(p, s, ring, at, tmem, abort_flag);
    } else if (warp >= 4) {
        epilogue<kGated, kForm, kTest>(p, s, others, at, warp, lane, tmem, abort_flag);
    }
    __syncwarp();
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // the other CTAs' MMAs, commits, sums and arrivals on this one are done
    if (p.last_launch) {
        dev::pdl_wait();
        dev::pdl_launch_dependents();
    }
    if (warp == 2) {
        dev::tc_fence_after();
        dev::tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- layout

// W [N] x [K] at strides (ld_n, ld_k) into the packed tiles, 16 bytes (8 channels) a thread.
__global__ void __launch_bounds__(256) pack_kernel(const uint16_t* __restrict__ W, int64_t ld_n, int64_t ld_k, int K, int N, int gated,
                                                   int nb, int tiles, uint8_t* __restrict__ Wp) {
    const int64_t pieces = static_cast<int64_t>(tiles) * nb * 1024;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < pieces; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int c = static_cast<int>(i & 7), r = static_cast<int>((i >> 3) & 127);
        const int64_t tb = i >> 10;
        const int b = static_cast<int>(tb % nb), t = static_cast<int>(tb / nb);
        const int n = fp8_source_row(t, r, N, gated), k = b * kW16Block + ((c ^ (r & 7)) << 3);
        uint4 out = make_uint4(0u, 0u, 0u, 0u);
        if (n >= 0) {
            const uint16_t* from = W + n * ld_n + k * ld_k;
            if (ld_k == 1 && k + 8 <= K && (reinterpret_cast<uintptr_t>(from) & 15u) == 0) {
                out = *reinterpret_cast<const uint4*>(from);
            } else {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k + j < K) w[j >> 1] |= static_cast<uint32_t>(from[j * ld_k]) << (16 * (j & 1));
                out = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        reinterpret_cast<uint4*>(Wp)[i] = out;
    }
}

// Rows to rows of ld8 pieces of 8 elements, a piece a thread; elements past K are 0.
template <bool kVec>
__global__ void __launch_bounds__(256) rows_kernel(const uint16_t* __restrict__ X, int64_t ldx, int64_t rows, int K,
                                                   const int32_t* __restrict__ row_of, int slots, uint4* __restrict__ out, int64_t ld8) {
    dev::pdl_wait();
    dev::pdl_launch_dependents();
    const int64_t pieces = rows * ld8;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < pieces; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t m = i / ld8, c = i - m * ld8;
        const int k = static_cast<int>(c) * 8;
        const uint16_t* from = X + m * ldx + k;
        uint4 v;
        if (k + 8 <= K) {
            v = kVec ? *reinterpret_cast<const uint4*>(from) : eight_at(from, 0);
        } else {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < K) w[j >> 1] |= static_cast<uint32_t>(from[j]) << (16 * (j & 1));
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (row_of == nullptr) {
            out[i] = v;
        } else {
            for (int j = 0; j < slots; ++j) {
                const int64_t r = row_of[m * slots + j];
                if (r >= 0) out[r * ld8 + c] = v;
            }
        }
    }
}

// ---------------------------------------------------------------- launch

bool encode_rows(CUtensorMap* map, const W16Args& a, const w16_layer& L, int box_rows) {
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(L.K), static_cast<cuuint64_t>(a.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldx) * 2};
    const cuuint32_t box[2] = {kW16Block, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    return encode(map, L.dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(a.X),
                  dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t config(int grid, int cluster, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// Clusters of `splits` pairs that are resident at once; asked once per device.
int resident_clusters(const w16_layer& L, int splits) {
    static int cached[64][kMaxSplits + 1] = {};
    const bool known = L.device >= 0 && L.device < 64;
    if (known && cached[L.device][splits] > 0) return cached[L.device][splits];
    int most = L.num_sms / (2 * splits) > 0 ? L.num_sms / (2 * splits) : 1;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(most * 2 * splits, 2 * splits, kSmemBytes, nullptr, attr);
    int got = 0;
    if (ensure_smem_limit(reinterpret_cast<const void*>(w16_kernel<false, kAnyForm>), kSmemBytes) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&got, w16_kernel<false, kAnyForm>, &cfg) == cudaSuccess && got > 0 && got < most)
        most = got;
    cudaGetLastError();   // a failed query leaves no error behind
    if (known) cached[L.device][splits] = most;
    return most;
}

// The units that are left of full rounds, in a launch of their own: each cut into `cuts` of `tile` rows, K in `splits` parts.
struct Rest {
    int units, tile, cuts, splits;   // units: of the product, 0: there is no such launch
    double time;
};
struct Shape {
    int tile, splits, grid, stages, others, most_tile;
    Rest rest;
};

// (`ahead`: of the residual, where K is not split)
Shape with_ring(int tile, int splits, int64_t units, int clusters, int ahead) {
    Shape s{tile, splits, 0, 0, 0, 0, {}};
    s.grid = static_cast<int>(units < clusters ? units : clusters) * 2 * splits;
    s.others = splits > 1 ? (splits - 1) * tile * 128 * 4 : ahead;
    s.stages = stages_of(tile, s.others);
    return s;
}

// The best such launch for `units` of `per` rows, all of it resident at once. It starts under the full rounds' end and still costs about
// 6000 clk, the exchange 1500 more: 300 x 4096 -> 20480 62 to 55 us, 1 x 8192 -> 28672 82 to 77, 2048 x 4096 -> 12288 127 to 123; counted at
// 1500, 300 x 1024 -> 20000 lost 3 of 24 and 520 x 4096 -> 11008 3 of 48.
Rest rest_of(const w16_layer& L, int units, int per, int ahead) {
    Rest best{0, 0, 0, 0, 1e30};
    for (int splits = 1; splits <= kMaxSplits; splits *= 2) {
        if (splits > 1 && L.nb < 4 * splits) break;
        const int clusters = resident_clusters(L, splits);
        for (int tile = 32; tile <= kPartRows && tile <= per; tile += 32) {
            const int cuts = (per + tile - 1) / tile;
            if (units * cuts > clusters || with_ring(tile, splits, 1, 1, ahead).stages < 4) continue;
            const double time = (L.nb + splits - 1) / splits * block_of(tile) + (splits > 1 ? 1500.0 : 0.0) + 6000.0 + 14.0 * tile;
            if (time < best.time) best = Rest{units, tile, cuts, splits, time};
        }
    }
    return best;
}

// No more units than these, whatever the groups: even_rows cuts none that is not the last of its group below half a tile.
int64_t most_units(const w16_layer& L, int used, int rows, int tile) {
    return (static_cast<int64_t>(used) + rows / (tile / 2)) * L.pairs;
}

// Rows of a unit, and in how many parts K is taken, by the rounds of units over the resident clusters. A block of 64 channels costs
// a pair about 400 clk and 0.65 more for each row of X: the copies from the L2 bound it, not the MMAs' 2 clk a row (2048 x 4096 -> 12288 in
// tiles of 64, 128, 192 and 256: 345, 172, 142 and 124 us; 777 x 2048 -> 5632: 51, 31, 25 and 29). Above 256 rows it is the MMAs, and
// the epilogue, which has no accumulator left to run beside: worth it where it saves a round (777 x 2048 -> 5632 in 320: 22) or where
// an expert's load is a little above 256 (32768 rows of 128, 4096 -> 2048: 463 us in tiles of 256, 439 in 320).
// Units that leave half the pairs idle split K: 1 x 8192 -> 8192 in 1, 2 and 4 parts 33.5, 25.2 and 25.4 us, 16 x 8192 -> 1024 33.2,
// 20.1 and 13.3, 128 x 8192 -> 8192 35.6 and 31.4, one row of 65 experts, 6400 -> 512, 29.5 and 14.4 in 4; the exchange takes about 1500
// clk. (The last round's blocks cut evenly over all pairs, their sums in global memory and the last to arrive adding them: 31.6 in place of 25.2, 17.2 of 13.3, 64
// units of a token's 8 experts 35.8 of 28.3, and 2048 x 4096 -> 12288, 4 units in the last round, no faster.)
Shape shape_of(const w16_layer& L, const W16Args& a, int ahead) {
    const bool grouped = a.start != nullptr;
    const int rows = static_cast<int>(a.rows);
    // the experts' loads are known on the device only: every one in use is taken to have the mean, and a sixth more for the spread. From 24
    // rows an expert on the device chooses the tile (count_units; 1554 rows of 10 uneven experts, 1404 -> 2012, in tiles of 64, 128, 192 and 256:
    // 37, 28, 32 and 36 us), and this says only whether K is split.
    const int used = grouped ? (L.experts < rows ? L.experts : rows) : 1, load = grouped ? (7 * rows / used + 5) / 6 : rows;
    Shape best{};
    double least = 0.0;
    for (int splits = 1; splits <= kMaxSplits; splits *= 2) {
        const int clusters = resident_clusters(L, splits);
        if (splits > 1 && L.nb < 4 * splits) break;
        for (int tile = 32; tile <= (splits > 1 ? kPartRows : kMostRows); tile += 32) {
            const int per = even_rows(load, tile);
            if (per != tile) continue;
            const int64_t tiles = (load + per - 1) / per, units = tiles * L.pairs * used, rounds = (units + clusters - 1) / clusters;
            const int64_t most = grouped ? most_units(L, used, rows, tile) : units;
            if (splits > 1 && most > clusters) continue;   // (a cluster that splits K takes one unit)
            Shape s = with_ring(tile, splits, most, clusters, ahead);
            if (s.stages < 4) continue;
            const double round = L.nb * block_of(per) + (per > kPartRows ? 14.0 * per : 0.0);
            double time = splits > 1 ? (L.nb + splits - 1) / splits * block_of(per) + 1500.0 + 14.0 * per : rounds * round + 14.0 * per;
            if (!grouped && splits == 1 && rounds > 1 && units % clusters != 0) {
                const Rest r = rest_of(L, static_cast<int>(units % clusters), per, ahead);
                if (r.time < round) {
                    s.rest = r;
                    time += r.time - round;
                }
            }
            if (best.grid == 0 || time < least) {
                best = s;
                least = time;
            }
        }
    }
    if (grouped && best.splits == 1 && rows >= 24 * used) {   // the device chooses the tile
        for (best.most_tile = kMostRows; stages_of(best.most_tile, best.others) < 4;) best.most_tile -= 32;
        const int64_t most = most_units(L, used, rows, 32);
        const int clusters = resident_clusters(L, 1);
        best.grid = static_cast<int>(most < clusters ? most : clusters) * 2;
    }
    return best;
}

}  // namespace
}  // namespace w16

cudaError_t launch_w16_gemm(const w16_layer& L, const W16Args& a, cudaStream_t stream) {
    w16::Params p{};
    p.W = static_cast<const uint8_t*>(a.W);
    p.start = a.start;
    p.count = a.count;
    p.row_weight = a.row_weight;
    p.pair_of = a.pair_of;
    p.e = a.epilogue;
    p.Y = a.Y;
    p.ldy = a.ldy;
    p.bf16 = L.dtype == kBF16;
    p.f32 = a.dtype == kF32;
    auto takes = [&](const void* v, int64_t ld, int bytes) {
        return (reinterpret_cast<uintptr_t>(v) & (bytes - 1)) == 0 && ld * (p.f32 ? 4 : 2) % bytes == 0;
    };
    auto both = [&](int bytes) { return takes(a.Y, a.ldy, bytes) && (p.e.residual == nullptr || takes(p.e.residual, p.e.ldr, bytes)); };
    p.vec = both(16) ? 8 : !p.f32 && both(8) ? 4 : 1;
    // put_out_whole does it where K is not split (a residual's rows begin at the same place of their 16 bytes as the outputs')
    const bool unsplit = !p.f32 && (L.gated ? p.vec >= 4
                                            : p.e.residual == nullptr ||
                                                  (((reinterpret_cast<uintptr_t>(a.Y) ^ reinterpret_cast<uintptr_t>(p.e.residual)) & 15u) == 0 &&
                                                   (p.ldy - p.e.ldr) % 8 == 0));
    const int ahead = unsplit && p.e.residual != nullptr ? w16::kAheadBytes : 0;
    const w16::Shape shape = w16::shape_of(L, a, ahead);
    p.rows = static_cast<int>(a.rows);
    p.N = L.N;
    p.out_n = L.gated ? L.N / 2 : L.N;
    p.nb = L.nb;
    p.pairs = L.pairs;
    p.experts = L.experts;
    p.status = L.d_status;
    p.polls = a.polls;
    p.withheld_cta = a.withheld_cta;
    p.withheld_copy = a.withheld_copy;
    CUtensorMap big, small;
    if (!w16::encode_rows(&big, a, L, w16::kBigBox) || !w16::encode_rows(&small, a, L, w16::kSmallBox)) return cudaErrorInvalidValue;
    auto launch = [&](const w16::Shape& s) {
        p.tile = s.tile;
        p.most_tile = s.most_tile;
        p.splits = s.splits;
        const bool whole = unsplit && s.splits == 1;
        // (FP32: on 16-byte boundaries)
        const bool whole32 = p.f32 && s.splits == 1 && p.vec == 8 && p.e.residual == nullptr;
        auto form = [&](auto gated) {
            return whole32 ? w16::w16_kernel<gated.value, w16::kWholeF32> : !whole ? w16::w16_kernel<gated.value, w16::kAnyForm>
                          : p.e.residual == nullptr ? w16::w16_kernel<gated.value, w16::kWholeBare> : w16::w16_kernel<gated.value, w16::kWholeAdded>;
        };
        auto fn = L.gated ? form(std::true_type{}) : form(std::false_type{});
        if (a.polls != 0) fn = whole ? w16::w16_kernel<false, w16::kWholeBare, true> : w16::w16_kernel<false, w16::kAnyForm, true>;
        const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), w16::kSmemBytes);
        if (e != cudaSuccess) return e;
        p.others = s.others;
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = w16::config(s.grid, 2 * s.splits, w16::kSmemBytes, stream, attr);
        return cudaLaunchKernelEx(&cfg, fn, p, big, small);
    };
    const w16::Rest& rest = shape.rest;
    p.cut = shape.tile;
    p.cuts = 1;
    p.tiles = w16::tiles_of(p.rows, p.cut);
    p.units = static_cast<int>((a.rows + p.cut - 1) / p.cut * L.pairs - rest.units);   // (experts: not used)
    const cudaError_t first = launch(shape);
    if (first != cudaSuccess || rest.units == 0) return first;
    p.first_cut = p.units;
    p.cuts = rest.cuts;
    p.units = rest.units * rest.cuts;
    p.last_launch = 1;
    p.withheld_cta = -1;
    return launch(w16::with_ring(rest.tile, rest.splits, p.units, p.units, ahead));
}

cudaError_t launch_w16_pack(const w16_layer& L, int expert, const void* W, int64_t ld_n, int64_t ld_k, void* Wp, cudaStream_t stream) {
    uint8_t* out = static_cast<uint8_t*>(Wp) + static_cast<int64_t>(expert) * L.pairs * 2 * L.nb * kTileBytes;
    const int64_t ctas = static_cast<int64_t>(L.pairs) * 2 * L.nb * 4;
    w16::pack_kernel<<<static_cast<int>(ctas < L.num_sms * 32LL ? ctas : L.num_sms * 32LL), 256, 0, stream>>>(
        static_cast<const uint16_t*>(W), ld_n, ld_k, L.K, L.N, L.gated, L.nb, L.pairs * 2, out);
    return cudaGetLastError();
}

cudaError_t launch_w16_rows(const void* X, int64_t ldx, int64_t rows, int K, const int32_t* row_of, int slots, void* out, int64_t ld,
                            int num_sms, cudaStream_t stream) {
    const int64_t ctas = (rows * (ld / 8) + 255) / 256;
    const bool vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && ldx % 8 == 0;
    return launch_after(vec ? w16::rows_kernel<true> : w16::rows_kernel<false>,
                        dim3(static_cast<unsigned>(ctas < num_sms * 32LL ? ctas : num_sms * 32LL)), 256, 0, true, stream,
                        static_cast<const uint16_t*>(X), ldx, rows, K, row_of, slots, static_cast<uint4*>(out), ld / 8);
}

}  // namespace fmpq
