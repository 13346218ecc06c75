// E4M3 product with a scale for each block of 128 (sm_103a), for a linear layer and for routed
// experts:
//
//   Y[m][n] = sum_b a_scale[b][m] * w_scale[n / 128][b] * P[m][n][b],
//   P[m][n][b] = sum over the 128 channels of block b of a_code * w_code.
//
// One kernel serves one token and thousands. The tensor core's M side is the weights: a pair of
// CTAs covers 256 packed weight rows (128 each, a 16 KB bulk copy a block), its N side the tokens
// of a tile, 32 to 256 of them in steps of 32. So a tile costs tensor time in proportion to its tokens
// (an expert's 150 tokens cost 160 columns, not 256), few tokens leave a pure weight stream, and the
// 256 x 256 pair tile of long prompts reads each operand byte half as often as two single CTAs.
//   * P is an FP32 accumulator tile in TMEM for one block of 128 (4 MMAs); 2, 4 or 8 of them, so that
//     the next blocks' MMAs run while the epilogue scales this one into FP32 registers.
//   * The epilogue reads 16 lanes x 64 columns at a time; a thread holds two rows and column
//     pairs, so a pair of token scales (one 8-byte shared load) serves both rows and, with packed
//     FP32 arithmetic, costs a multiply by the block's weight scale and two multiply-adds.
//   * The packed order of the weight rows (fp8_source_row) makes the transposed accumulator give a
//     thread 8 consecutive output channels of a token (one 16-byte store), or, for a gated layer,
//     the gate and up values of the same hidden channels: SwiGLU and the E4M3 quantization of the
//     hidden vector happen in registers, with one absmax per token exchanged inside the pair.
//
// Warp roles (384 threads, one CTA per SM, pairs persistent over tiles):
//   warp 0      producer: weight block, token codes, token scales (a chunk of blocks at a time)
//   warp 1      even CTA: MMA issuer; odd CTA: reports its operands to the even one
//   warp 2      allocates and frees TMEM
//   warps 4-11  epilogue: TMEM lane quarter warp % 4, half of the tile's columns each
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fmpq_device.cuh"
#include "fmpq_internal.h"
#include "fp8_internal.h"

namespace fmpq {
namespace {

constexpr int kThreads = 384;
constexpr int kStages = 6;
constexpr int kScChunk = 4;     // blocks of token scales per copy
constexpr int kScSlots = 3;
constexpr int kMaxAcc = 8;
constexpr int kEpiWarps = 8;
constexpr int kMaxExperts = 1024;
constexpr int kGroupM = 8;      // dense order: bands of token tiles, weight tiles inside a band
constexpr uint32_t kTmemCols = 512;

// kC: 32-column chunks of a half tile: token tiles of up to 64 (1), 128 (2) or 256 (4) tokens.
template <int kC>
struct Shape {
    static constexpr int kTokens = 64 * kC;
    static constexpr int kAcc = kC == 1 ? 8 : 8 / kC;   // accumulators of kTokens columns in 512
    static constexpr int kCols = kC == 1 ? 32 : 64;     // columns of one TMEM load
    static constexpr int kParts = 32 * kC / kCols;      // loads of each lane half per block
};

template <int kC>
struct __align__(1024) Smem {
    uint8_t w[kStages][kTileBytes];                 // weight block: this CTA's 128 rows
    uint8_t x[kStages][Shape<kC>::kTokens * 64];    // token codes: this CTA's half of the tile
    float sx[kScSlots][kScChunk][Shape<kC>::kTokens];
    float amax[2][8][Shape<kC>::kTokens];           // gated: absmax of 16 hidden channels (CTA, quarter)
    uint64_t full[kStages], empty[kStages], peer_full[kStages];
    uint64_t acc_full[kMaxAcc], acc_empty[kMaxAcc];
    uint64_t sc_full[kScSlots], sc_empty[kScSlots];
    uint64_t amax_full[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
    int fixup_last;
    int32_t first_unit[kMaxExperts + 1];            // experts: units before each expert's
};

struct Params {
    const uint8_t* A;
    const uint8_t* W;
    const float* w_scales;
    const int32_t* start;      // experts (nullptr: dense)
    const int32_t* count;
    const int32_t* pair_of;
    const float* pair_weight;
    int64_t rows, sstride;
    uint16_t* Y;
    int64_t ldy;
    int bf16, vec;             // output type; 16-byte stores allowed
    uint8_t* H;
    float* h_scales;
    int M, N, nb, pairs, scale_rows, experts, splits;
    float* partial;            // split-K: [tile][split][CTA][warp][vector][lane] FP32 sums
    int32_t* arrivals;         // [tile][CTA]
    int32_t* status;
};

// A unit of work: the 256 packed weight rows `pair` of expert e, `n` tokens from row `row0`, blocks
// [b0, b1).
struct Unit {
    int e, pair, n, cols, b0, b1, tile, split;
    int64_t row0;
};

// Tile t of `tiles` over an expert's tokens, all of about the same size (a multiple of 32).
__device__ __forceinline__ void token_tile(int tokens, int tiles, int t, int& first, int& n) {
    const int size = ((tokens + tiles - 1) / tiles + 31) & ~31;
    first = t * size;
    n = min(size, tokens - first);
}

template <int kC>
__device__ __forceinline__ int unit_count(const Params& p, const Smem<kC>& s) {
    if (p.start != nullptr) return s.first_unit[p.experts];
    return p.pairs * ((p.M + Shape<kC>::kTokens - 1) / Shape<kC>::kTokens) * p.splits;
}

template <int kC>
__device__ __forceinline__ Unit unit_of(const Params& p, const Smem<kC>& s, int u) {
    constexpr int kT = Shape<kC>::kTokens;
    Unit r;
    int tokens = p.M, t, first;
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
        tokens = p.count[lo];
        const int tiles = (tokens + kT - 1) / kT, i = u - s.first_unit[lo];
        t = i % tiles;
        r.pair = i / tiles;
        r.tile = u;
        token_tile(tokens, tiles, t, first, r.n);
        r.row0 = p.start[lo] + first;
    } else {
        const int tiles = (p.M + kT - 1) / kT;
        r.e = 0;
        r.tile = u / p.splits;
        r.split = u % p.splits;
        const int band = r.tile / (kGroupM * p.pairs), in_band = r.tile - band * kGroupM * p.pairs;
        const int gm = min(kGroupM, tiles - band * kGroupM);
        t = band * kGroupM + in_band % gm;
        r.pair = in_band / gm;
        token_tile(tokens, tiles, t, first, r.n);
        r.row0 = first;
        r.b0 = static_cast<int>(static_cast<int64_t>(r.split) * p.nb / p.splits);
        r.b1 = static_cast<int>(static_cast<int64_t>(r.split + 1) * p.nb / p.splits);
    }
    r.cols = max(32, (r.n + 31) & ~31);
    return r;
}

__device__ __forceinline__ void fail(const Params& p, volatile int* abort_flag) {
    *abort_flag = 1;
    dev::report(p.status, dev::kStatusTimeout);
}

// ---------------------------------------------------------------- producer (warp 0, one thread)
template <int kC>
__device__ __forceinline__ void producer(const Params& p, const CUtensorMap* scales, Smem<kC>& s, uint32_t rank,
                                         volatile int* abort_flag) {
    const int units = unit_count<kC>(p, s);
    uint32_t it = 0, ch = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        const Unit t = unit_of<kC>(p, s, u);
        const int half = t.cols >> 1, local = static_cast<int>(rank) * half;
        const uint32_t xbytes = static_cast<uint32_t>(max(0, min(half, t.n - local))) * 128u;
        const uint8_t* w = p.W + (static_cast<int64_t>(t.e) * p.pairs * 2 + 2 * t.pair + rank) * p.nb * kTileBytes;
        const uint8_t* x = p.A + (t.row0 + local) * 128;
        for (int b = t.b0; b < t.b1; ++b, ++it) {
            if ((b - t.b0) % kScChunk == 0) {
                const int sl = ch % kScSlots;
                ok = dev::mbar_wait(&s.sc_empty[sl], ((ch / kScSlots) & 1) ^ 1, abort_flag);
                if (!ok) break;
                dev::mbar_arrive_expect_tx(&s.sc_full[sl], sizeof(s.sx[0]));
                dev::tma_load_2d(s.sx[sl], scales, static_cast<int>(t.row0), b, &s.sc_full[sl]);
                ++ch;
            }
            const int st = it % kStages;
            ok = dev::mbar_wait(&s.empty[st], ((it / kStages) & 1) ^ 1, abort_flag);
            if (!ok) break;
            dev::mbar_arrive_expect_tx(&s.full[st], kTileBytes + xbytes);
            dev::bulk_g2s(s.w[st], w + static_cast<int64_t>(b) * kTileBytes, kTileBytes, &s.full[st]);
            if (xbytes > 0) dev::bulk_g2s(s.x[st], x + static_cast<int64_t>(b) * p.rows * 128, xbytes, &s.full[st]);
        }
    }
    if (!ok) fail(p, abort_flag);
    // the copies in flight must land before the CTA's shared memory is given up
    for (uint32_t k = 0; k < kStages && k < it; ++k) {
        const uint32_t i = it - 1 - k;
        dev::mbar_wait(&s.full[i % kStages], (i / kStages) & 1, nullptr);
    }
    for (uint32_t k = 0; k < kScSlots && k < ch; ++k) {
        const uint32_t i = ch - 1 - k;
        dev::mbar_wait(&s.sc_full[i % kScSlots], (i / kScSlots) & 1, nullptr);
    }
}

// ---------------------------------------------------------------- MMA (warp 1, one thread)
template <int kC>
__device__ __forceinline__ void mma_issuer(const Params& p, Smem<kC>& s, uint32_t rank, uint32_t tmem,
                                           volatile int* abort_flag) {
    constexpr int kAcc = Shape<kC>::kAcc;
    const int units = unit_count<kC>(p, s);
    const uint32_t leader = dev::mapa(&s.peer_full[0], 0);
    uint32_t it = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        const Unit t = unit_of<kC>(p, s, u);
        const uint32_t idesc = dev::idesc_e4m3_f32(256, static_cast<uint32_t>(t.cols));
        for (int b = t.b0; b < t.b1; ++b, ++it) {
            const int st = it % kStages;
            const uint32_t phase = (it / kStages) & 1;
            ok = dev::mbar_wait(&s.full[st], phase, abort_flag);
            if (!ok) break;
            if (rank != 0) {
                dev::mbar_arrive_remote(leader + static_cast<uint32_t>(st) * 8u);
                continue;
            }
            const int acc = it % kAcc;
            ok = dev::mbar_wait(&s.peer_full[st], phase, abort_flag) &&
                 dev::mbar_wait(&s.acc_empty[acc], ((it / kAcc) & 1) ^ 1, abort_flag);
            if (!ok) break;
            dev::tc_fence_after();
            const uint64_t ad = dev::sdesc_k_sw128(dev::smem_u32(s.w[st]));
            const uint64_t bd = dev::sdesc_k_sw128(dev::smem_u32(s.x[st]));
            const uint32_t d = tmem + static_cast<uint32_t>(acc * Shape<kC>::kTokens);
#pragma unroll
            for (int k = 0; k < 4; ++k) dev::mma_e4m3_pair(d, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
            dev::mma_commit_pair(&s.empty[st]);
            dev::mma_commit_pair(&s.acc_full[acc]);
        }
    }
    if (!ok) fail(p, abort_flag);
    if (rank == 0) {   // every MMA must finish before TMEM is released
        dev::mma_commit_pair(&s.mma_done);
        dev::mbar_wait(&s.mma_done, 0, nullptr);
    }
}

// ---------------------------------------------------------------- epilogue (warps 4-11)
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
    uint32_t r;
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        r = *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        r = *reinterpret_cast<const uint32_t*>(&v);
    }
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int N>
__device__ __forceinline__ void load_acc(uint32_t addr, uint32_t (&d)[N]) {
    if constexpr (N == 32) dev::tmem_ld16x256b_x8(addr, d);
    else dev::tmem_ld16x256b_x4(addr, d);
}
template <int N>
__device__ __forceinline__ void wait_acc(uint32_t (&d)[N]) {
    if constexpr (N == 32) dev::tmem_ld_wait32(d);
    else dev::tmem_ld_wait16(d);
}

// Warp ew covers TMEM lanes 32 (ew % 4) .. + 31 and the columns (ew / 4) * cols / 2 .. + cols / 2 of a
// tile. In a load of 16 lanes (half v of the quarter), thread t holds rows t / 4 and t / 4 + 8 and
// columns 8i + 2 (t % 4) + {0, 1}: acc[v][i][0] and acc[v][i][1].
template <int kC, bool kGated>
__device__ __forceinline__ void epilogue(const Params& p, Smem<kC>& s, uint32_t rank, int warp, int lane, uint32_t tmem,
                                         volatile int* abort_flag) {
    using S = Shape<kC>;
    constexpr int kGroups = 4 * kC;          // 8-column groups of a half tile
    constexpr int kPer = S::kCols / 8;       // of one load
    const int units = unit_count<kC>(p, s);
    const int ew = warp - 4, q = ew & 3, h = ew >> 2;
    const int tq = lane & 3, tr = lane >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t leader_empty = dev::mapa(&s.acc_empty[0], 0);
    uint32_t v = 0, ch = 0, nu = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; u < units; u += gridDim.x >> 1) {
        const Unit t = unit_of<kC>(p, s, u);
        const int half = t.cols >> 1, c0 = h * half;
        const int parts = (half + S::kCols - 1) / S::kCols;
        // weight scales of 32 blocks, one a lane: this CTA's 128 channels, or gate and up
        const int srow = kGated ? t.pair : 2 * t.pair + static_cast<int>(rank);
        const float* ws = p.w_scales + static_cast<int64_t>(t.e) * p.scale_rows * p.nb;
        const float* ws0 = ws + static_cast<int64_t>(min(srow, p.scale_rows - 1)) * p.nb;
        const float* ws1 = kGated ? ws0 + static_cast<int64_t>(p.scale_rows / 2) * p.nb : ws0;
        auto scale_of = [&](const float* w, int b) { return b < t.b1 ? __ldg(w + b) : 0.0f; };
        float next0 = scale_of(ws0, t.b0 + lane), next1 = kGated ? scale_of(ws1, t.b0 + lane) : 0.0f;
        float cur0 = 0.0f, cur1 = 0.0f;
        float wgt[kC];                        // a row's weight: columns c0 + lane + 32 j
#pragma unroll
        for (int j = 0; j < kC; ++j) {
            wgt[j] = 1.0f;
            const int col = c0 + lane + 32 * j;
            if (!kGated && p.pair_weight != nullptr && col < t.n) wgt[j] = __ldg(p.pair_weight + p.pair_of[t.row0 + col]);
        }
        float2 acc[2][kGroups][2];
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j >> 1][i][j & 1] = make_float2(0.0f, 0.0f);

        for (int b = t.b0; b < t.b1; ++b, ++v) {
            const int i32 = (b - t.b0) & 31;
            if (i32 == 0) {
                cur0 = next0;
                cur1 = next1;
                next0 = scale_of(ws0, b + 32 + lane);
                if (kGated) next1 = scale_of(ws1, b + 32 + lane);
            }
            const float w0 = __shfl_sync(0xFFFFFFFFu, cur0, i32);
            const float w1 = kGated ? __shfl_sync(0xFFFFFFFFu, cur1, i32) : w0;
            const int in_chunk = (b - t.b0) % kScChunk, sl = ch % kScSlots;
            const int slot = v % S::kAcc;
            if (ok) {
                ok = (in_chunk != 0 || dev::mbar_wait(&s.sc_full[sl], (ch / kScSlots) & 1, abort_flag)) &&
                     dev::mbar_wait(&s.acc_full[slot], (v / S::kAcc) & 1, abort_flag);
                ok = __all_sync(0xFFFFFFFFu, ok);
            }
            if (ok) {
                dev::tc_fence_after();
                const uint32_t base = tmem + lane_addr + static_cast<uint32_t>(slot * S::kTokens + c0);
                const float* sx = s.sx[sl][in_chunk] + c0 + 2 * tq;
                uint32_t d[2][S::kCols / 2];
                load_acc(base, d[0]);
#pragma unroll
                for (int st = 0; st < 2 * S::kParts; ++st) {
                    const int part = st >> 1, lh = st & 1;
                    if (part >= parts) break;
                    wait_acc(d[st & 1]);
                    const bool more = st + 1 < 2 * S::kParts && ((st + 1) >> 1) < parts;
                    if (more) {
                        load_acc(base + static_cast<uint32_t>(((st + 1) >> 1) * S::kCols) + (((st + 1) & 1) ? (16u << 16) : 0u),
                                 d[(st + 1) & 1]);
                    } else {
                        // all of it is in registers: the next MMAs may have the accumulator
                        dev::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) dev::mbar_arrive_remote(leader_empty + static_cast<uint32_t>(slot) * 8u);
                    }
                    const float wl = lh ? w1 : w0;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const float2 sc = dev::fmul2(*reinterpret_cast<const float2*>(sx + part * S::kCols + 8 * i), make_float2(wl, wl));
                        const uint32_t* r = d[st & 1] + 4 * i;
                        float2* a = acc[lh][part * kPer + i];
                        a[0] = dev::ffma2(make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])), sc, a[0]);
                        a[1] = dev::ffma2(make_float2(__uint_as_float(r[2]), __uint_as_float(r[3])), sc, a[1]);
                    }
                }
            }
            if (in_chunk == kScChunk - 1 || b + 1 == t.b1) {
                __syncwarp();
                if (lane == 0 && ok) dev::mbar_arrive(&s.sc_empty[sl]);
                ++ch;
            }
        }

        if constexpr (kGated) {
            // h = silu(gate) * up and the absmax of each token over the pair's 128 hidden channels: 16
            // channels a warp, exchanged through both CTAs' shared memory. Two buffers: a warp writes
            // the next tile's only after every warp has arrived for the tile in between.
            const int par = nu & 1;
            const uint32_t mine = dev::mapa(&s.amax[par][rank * 4 + q][0], rank), other = dev::mapa(&s.amax[par][rank * 4 + q][0], rank ^ 1u);
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                float2 m = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float2& g = acc[0][i][r];
                    const float2 up = acc[1][i][r];
                    g.x = g.x / (1.0f + expf(-g.x)) * up.x;
                    g.y = g.y / (1.0f + expf(-g.y)) * up.y;
                    m.x = fmaxf(m.x, fabsf(g.x));
                    m.y = fmaxf(m.y, fabsf(g.y));
                }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    m.x = fmaxf(m.x, __shfl_xor_sync(0xFFFFFFFFu, m.x, d));
                    m.y = fmaxf(m.y, __shfl_xor_sync(0xFFFFFFFFu, m.y, d));
                }
                if (tr == 0 && 8 * i < half) {
                    const uint32_t at = static_cast<uint32_t>(c0 + 8 * i + 2 * tq) * 4u;
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mine + at), "f"(m.x), "f"(m.y) : "memory");
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(other + at), "f"(m.x), "f"(m.y) : "memory");
                }
            }
            __syncwarp();
            if (lane == 0) {
                dev::mbar_arrive_remote_release(dev::mapa(&s.amax_full[par], 0));
                dev::mbar_arrive_remote_release(dev::mapa(&s.amax_full[par], 1));
            }
            if (ok) ok = dev::mbar_wait_cluster(&s.amax_full[par], (nu >> 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                if (8 * i >= half) break;
                const int col = c0 + 8 * i + 2 * tq;
                float2 m = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 o = *reinterpret_cast<const float2*>(&s.amax[par][j][col]);
                    m.x = fmaxf(m.x, o.x);
                    m.y = fmaxf(m.y, o.y);
                }
                const float sx = __fdiv_rn(m.x, 448.0f), sy = __fdiv_rn(m.y, 448.0f);
                auto quot = [](float a, float b) { return b > 0.0f ? __fdiv_rn(a, b) : 0.0f; };
                const float2 a = acc[0][i][0], bb = acc[0][i][1];
                // rows r and r + 8 of a column in one 16-bit element, transposed as 8 x 8 elements
                const uint32_t r = transpose8x8(e4m3x2(quot(a.x, sx), quot(bb.x, sx)) | (e4m3x2(quot(a.y, sy), quot(bb.y, sy)) << 16));
                const int tok = c0 + 8 * i + tr;
                if (ok && tok < t.n) {
                    const int64_t row = t.row0 + tok;
                    uint8_t* o = p.H + (static_cast<int64_t>(t.pair) * p.rows + row) * 128;
                    *reinterpret_cast<uint32_t*>(o + (((static_cast<int>(rank) * 4 + q) ^ static_cast<int>(row & 7)) << 4) + 4 * tq) =
                        __byte_perm(r, 0u, 0x3120);
                }
                if (ok && rank == 0 && q == 0 && tr == 0) {
                    float* hs = p.h_scales + t.pair * p.sstride + t.row0;
                    if (col < t.n) hs[col] = sx;
                    if (col + 1 < t.n) hs[col + 1] = sy;
                }
            }
            ++nu;
        } else {
            const int n0 = 256 * t.pair + 128 * static_cast<int>(rank) + 32 * q + 8 * tq;
            auto store = [&]() {
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    if (8 * i >= half) break;
                    const float wx = __shfl_sync(0xFFFFFFFFu, wgt[i >> 2], (8 * i + 2 * tq) & 31);
                    const float wy = __shfl_sync(0xFFFFFFFFu, wgt[i >> 2], (8 * i + 2 * tq + 1) & 31);
                    uint32_t o[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float2 f = acc[g >> 1][i][g & 1];
                        o[g] = transpose8x8(pack16(f.x * wx, f.y * wy, p.bf16));
                    }
                    const int tok = c0 + 8 * i + tr;
                    if (!ok || tok >= t.n) continue;
                    uint16_t* y = p.Y + (t.row0 + tok) * p.ldy + n0;
                    if (p.vec && n0 + 8 <= p.N) {
                        *reinterpret_cast<uint4*>(y) = make_uint4(o[0], o[1], o[2], o[3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (n0 + j < p.N) y[j] = static_cast<uint16_t>(o[j >> 1] >> (16 * (j & 1)));
                    }
                }
            };
            if (p.splits == 1) {
                store();
            } else {
                // publish this split's sums; the last split to arrive adds all of them in split order
                const int64_t per_warp = kGroups * 2 * 32;   // float4s
                auto slot_of = [&](int sp) {
                    return reinterpret_cast<float4*>(p.partial) +
                           (((static_cast<int64_t>(t.tile) * p.splits + sp) * 2 + rank) * kEpiWarps + ew) * per_warp + lane;
                };
                float4* out = slot_of(t.split);
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    if (8 * i >= half) break;
#pragma unroll
                    for (int l = 0; l < 2; ++l)
                        __stcg(out + (2 * i + l) * 32, make_float4(acc[l][i][0].x, acc[l][i][0].y, acc[l][i][1].x, acc[l][i][1].y));
                }
                __threadfence();
                dev::named_bar_sync(1, kEpiWarps * 32);
                if (ew == 0 && lane == 0) {
                    int32_t* cnt = p.arrivals + t.tile * 2 + static_cast<int>(rank);
                    const int last = atomicAdd(cnt, 1) == p.splits - 1;
                    if (last) *cnt = 0;   // ready for the next call
                    s.fixup_last = last;
                }
                dev::named_bar_sync(1, kEpiWarps * 32);
                if (s.fixup_last) {
                    __threadfence();
#pragma unroll
                    for (int i = 0; i < kGroups; ++i) {
                        if (8 * i >= half) break;
#pragma unroll
                        for (int l = 0; l < 2; ++l) {
                            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            for (int sp = 0; sp < p.splits; ++sp) {
                                const float4 f = __ldcg(slot_of(sp) + (2 * i + l) * 32);
                                sum.x += f.x;
                                sum.y += f.y;
                                sum.z += f.z;
                                sum.w += f.w;
                            }
                            acc[l][i][0] = make_float2(sum.x, sum.y);
                            acc[l][i][1] = make_float2(sum.z, sum.w);
                        }
                    }
                    store();
                }
                dev::named_bar_sync(1, kEpiWarps * 32);   // fixup_last is read before the next unit writes it
            }
        }
    }
    if (!ok && lane == 0) fail(p, abort_flag);
}

template <int kC, bool kGated>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
fp8_gemm_kernel(const Params p, const __grid_constant__ CUtensorMap scales) {
    extern __shared__ uint8_t smem_raw[];
    Smem<kC>& s = *reinterpret_cast<Smem<kC>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = dev::cluster_ctarank();
    if (threadIdx.x == 0) {
        dev::tma_prefetch_map(&scales);
        for (int i = 0; i < kStages; ++i) {
            dev::mbar_init(&s.full[i], 1);
            dev::mbar_init(&s.empty[i], 1);
            dev::mbar_init(&s.peer_full[i], 1);
        }
        for (int i = 0; i < kMaxAcc; ++i) {
            dev::mbar_init(&s.acc_full[i], 1);
            dev::mbar_init(&s.acc_empty[i], 2 * kEpiWarps);
        }
        for (int i = 0; i < kScSlots; ++i) {
            dev::mbar_init(&s.sc_full[i], 1);
            dev::mbar_init(&s.sc_empty[i], kEpiWarps);
        }
        for (int i = 0; i < 2; ++i) dev::mbar_init(&s.amax_full[i], 2 * kEpiWarps);
        dev::mbar_init(&s.mma_done, 1);
        s.abort_flag = 0;
        dev::fence_barrier_init();
    }
    if (warp == 2) dev::tmem_alloc_pair(&s.tmem_base, kTmemCols);
    if (warp == 3 && p.start != nullptr) {
        // units before each expert's: lane l sums the run of experts [l * run, l * run + run)
        const int run = (p.experts + 31) / 32;
        auto units_of = [&](int e) {
            return e < p.experts ? (p.count[e] + Shape<kC>::kTokens - 1) / Shape<kC>::kTokens * p.pairs : 0;
        };
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
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // both CTAs' barriers and TMEM exist before any traffic between them
    dev::tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    volatile int* abort_flag = &s.abort_flag;

    if (warp < 4) {
        dev::setmaxnreg_dec<72>();
        if (warp == 0 && lane == 0) producer<kC>(p, &scales, s, rank, abort_flag);
        else if (warp == 1 && lane == 0) mma_issuer<kC>(p, s, rank, tmem, abort_flag);
        __syncwarp();
    } else {
        dev::setmaxnreg_inc<216>();
        epilogue<kC, kGated>(p, s, rank, warp, lane, tmem, abort_flag);
    }
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // the peer's MMAs, commits, stores and arrivals on this CTA are done
    if (warp == 2) {
        dev::tc_fence_after();
        dev::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

template <int kC>
constexpr size_t smem_bytes() { return sizeof(Smem<kC>) + 1024; }
static_assert(smem_bytes<4>() <= 232448, "shared memory exceeds the 227 KB a CTA may use");

// Pairs that can be resident at once, asked once per device: the persistent grid never launches more.
int max_pairs(const fp8_layer& L) {
    static int cached[64] = {};
    if (L.device >= 0 && L.device < 64 && cached[L.device] > 0) return cached[L.device];
    int pairs = L.num_sms / 2 > 0 ? L.num_sms / 2 : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<4>();
    int clusters = 0;
    if (ensure_smem_limit(reinterpret_cast<const void*>(fp8_gemm_kernel<4, false>), static_cast<int>(smem_bytes<4>())) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, fp8_gemm_kernel<4, false>, &cfg) == cudaSuccess && clusters > 0 && clusters < pairs)
        pairs = clusters;
    cudaGetLastError();   // a failed query leaves no error behind
    if (L.device >= 0 && L.device < 64) cached[L.device] = pairs;
    return pairs;
}

// Chunks of a half tile: the smallest token tile that holds a dense layer's tokens, or that holds
// an expert's share of them with room for an uneven load.
int chunks_for(int64_t tokens, int experts) {
    const int64_t share = experts > 1 ? (tokens * 4 / 3 + experts - 1) / experts : tokens;
    return share <= 64 ? 1 : share <= 128 ? 2 : 4;
}

// Dense tiles too few for the pairs: K is split, at least 4 blocks a split.
int splits_for(const fp8_layer& L, int64_t M) {
    if (L.experts > 1 || L.gated) return 1;
    const int most = 64 * chunks_for(M, 1);
    const int64_t tiles = L.pairs * ((M + most - 1) / most);
    const int pairs = max_pairs(L);
    if (tiles * 2 > pairs) return 1;
    int64_t s = pairs / tiles;
    if (s > L.nb / 4) s = L.nb / 4;
    if (s > 8) s = 8;
    return s < 1 ? 1 : static_cast<int>(s);
}

template <int kC, bool kGated>
cudaError_t launch_as(const fp8_layer& L, const Params& p, int grid, const CUtensorMap& map, cudaStream_t stream) {
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fp8_gemm_kernel<kC, kGated>), static_cast<int>(smem_bytes<kC>()));
    if (e != cudaSuccess) return e;
    fp8_gemm_kernel<kC, kGated><<<grid, kThreads, smem_bytes<kC>(), stream>>>(p, map);
    return cudaGetLastError();
}

size_t partial_bytes(const fp8_layer& L, int64_t M, int splits) {
    const int c = chunks_for(M, 1);
    const int64_t tiles = L.pairs * ((M + 64 * c - 1) / (64 * c));
    return static_cast<size_t>(tiles) * splits * 2 * kEpiWarps * (4 * c * 2 * 32) * sizeof(float4);
}

}  // namespace

// The arrival counters come first, so that every size that shares a buffer finds zeros there.
size_t fp8_gemm_workspace(const fp8_layer& L, int64_t M) {
    const int splits = splits_for(L, M);
    if (splits == 1) return 0;
    return static_cast<size_t>(L.num_sms) * 2 * sizeof(int32_t) + 256 + partial_bytes(L, M, splits);
}

cudaError_t launch_fp8_gemm(const fp8_layer& L, const Fp8GemmArgs& a, cudaStream_t stream) {
    const bool routed = a.start != nullptr;
    const int c = chunks_for(a.pairs_routed, routed ? L.experts : 1);
    const int most = 64 * c;
    Params p{};
    p.A = static_cast<const uint8_t*>(a.A);
    p.W = static_cast<const uint8_t*>(a.W);
    p.w_scales = a.w_scales;
    p.start = a.start;
    p.count = a.count;
    p.pair_of = a.pair_of;
    p.pair_weight = a.pair_weight;
    p.rows = a.rows;
    p.sstride = scale_stride(a.rows);
    p.Y = static_cast<uint16_t*>(a.Y);
    p.ldy = a.ldy;
    p.bf16 = a.dtype == kBF16;
    p.vec = a.ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(a.Y) & 15u) == 0;
    p.H = static_cast<uint8_t*>(a.H);
    p.h_scales = a.h_scales;
    p.M = static_cast<int>(a.rows);
    p.N = L.N;
    p.nb = L.nb;
    p.pairs = L.pairs;
    p.scale_rows = L.scale_rows;
    p.experts = L.experts;
    p.splits = a.workspace != nullptr ? splits_for(L, a.rows) : 1;
    p.status = L.d_status;
    if (p.splits > 1) {
        p.arrivals = static_cast<int32_t*>(a.workspace);
        p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                             ((static_cast<size_t>(L.num_sms) * 2 * sizeof(int32_t) + 255) & ~size_t(255)));
    }
    // the token scales as a 2-D tensor [nb][rows], boxes of kScChunk blocks x a tile's tokens
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;
    CUtensorMap map;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.sstride), static_cast<cuuint64_t>(L.nb)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.sstride) * sizeof(float)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(most), kScChunk}, step[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(a.a_scales), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    // an upper bound of the units: a partial token tile per expert in use
    const int64_t experts_used = routed ? (L.experts < a.pairs_routed ? L.experts : a.pairs_routed) : 0;
    const int64_t tiles = routed ? experts_used + a.pairs_routed / most : (a.rows + most - 1) / most;
    const int64_t units = tiles * L.pairs * p.splits;
    const int grid = 2 * static_cast<int>(units < max_pairs(L) ? units : max_pairs(L));
    if (L.gated)
        return c == 1 ? launch_as<1, true>(L, p, grid, map, stream) : c == 2 ? launch_as<2, true>(L, p, grid, map, stream) : launch_as<4, true>(L, p, grid, map, stream);
    return c == 1 ? launch_as<1, false>(L, p, grid, map, stream) : c == 2 ? launch_as<2, false>(L, p, grid, map, stream) : launch_as<4, false>(L, p, grid, map, stream);
}

}  // namespace fmpq
