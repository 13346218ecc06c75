// E4M3 product with a scale for each block of 128 (sm_103a), for a linear layer and for routed
// experts:
//
//   Y[m][n] = sum_b a_scale[b][m] * w_scale[n / 128][b] * P[m][n][b],
//   P[m][n][b] = sum over the 128 channels of block b of a_code * w_code.
//
// This file: few tokens a matrix (a decode step, an expert's share of one), and the choice between this
// kernel and the one for many (fp8_gemm_wide.cu). Reading the weights bounds it. The tensor core's M
// side is the weights: a pair of CTAs covers 256 packed weight rows (128 each, a 16 KB bulk copy a
// block, 128 KB in flight per SM); its N side is a tile of 32 or 64 tokens.
//   * P is an FP32 accumulator tile in TMEM for one block of 128 (4 MMAs), eight of them, so that the
//     next blocks' MMAs run while the epilogue scales this one into FP32 registers.
//   * An epilogue thread owns one weight row (a TMEM lane) and 32 tokens. A scaler warp multiplies the
//     block's token scales by its weight scale beforehand, so that a pair of sums costs one packed
//     multiply-add and half a broadcast shared load. Up to 32 tokens, the two warps of a lane quarter
//     take the blocks in turn: the chain of a block through one warp (wait, TMEM load, arithmetic,
//     release: about 650 clk) is as long as a 16 KB copy takes at the HBM's rate.
//   * A gated layer's rows are packed so that a warp holds the gate and the up rows of the same 16
//     hidden channels in its two halves: SwiGLU and the E4M3 quantization of the hidden vector
//     happen in registers, with one absmax per token exchanged inside the pair.
//   * The weights' stream starts before the codes are there (the kernel is launched as the quantizer's
//     programmatic dependent); token codes come four blocks a box, one copy per block being what the
//     copy engine and the issuing warp keep up with.
// Measured (quantizer included): one token of 8192 x 8192 21.8 us, 67.1 MB = 3.1 TB/s (a stream this short does
// not reach the copy rate); 64 tokens through 8 of 128 experts of 4096 x 1024, 1.59 GB in 272 us = 5.8 TB/s, 86% of
// the measured copy rate.
//
// Warp roles (384 threads, one CTA per SM, pairs persistent over tiles):
//   warp 0      weight producer (a 16 KB block a copy)
//   warp 1      even CTA: MMA issuer; odd CTA: reports its operands to the even one
//   warp 2      scaler; also allocates and frees TMEM
//   warp 3      token producer: codes and scales of four blocks at a time
//   warps 4-11  epilogue: TMEM lane quarter warp % 4, half of the tile's tokens (or of the blocks) each
#include <type_traits>

#include "fp8_gemm.cuh"

namespace fmpq {
namespace fp8 {
namespace {

constexpr int kRing = 16;      // blocks whose readiness may be in flight (> kStages, > 2 kAcc - 1)
constexpr int kProd = 4;       // blocks of scale products
constexpr int kTokens = 64;    // of a tile, at most
constexpr int kAcc = 8;        // accumulators of kTokens columns in 512
constexpr int kStages = 8;     // weight blocks in flight

struct __align__(1024) Smem {
    uint8_t w[kStages][kTileBytes];                // weight block: this CTA's 128 rows
    uint8_t x[kScSlots][kScChunk][kTokens * 64];   // token codes of a chunk of blocks: this CTA's half of the tile
    float sx[kScSlots][kScChunk][kTokens];         // token scales of the chunk
    // token scales times the block's weight scale; gated: [0] gate, [1] up (the 16-byte skew keeps
    // the two halves of a warp in different banks)
    float prod[kProd][2][kTokens + 4];
    // gated: absmax of 16 hidden channels (a quarter's), of this CTA's 64 and the peer's 64, the
    // tokens' scales
    float amax[4][kTokens], amax_peer[2][kTokens], hscale[kTokens];
    float2 other_turn[16][128];   // up to 32 tokens: the sums of every second block
    // ready[b % kRing], even CTA: block b's weights have landed in both CTAs, the odd one's token codes
    // too, and its accumulator has been read (by both CTAs' epilogue warps). Odd CTA: its weights have
    // landed. sc_full: a chunk's token codes and scales have landed here; sc_empty: the scaler has read the
    // scales and the chunk's MMAs are done.
    uint64_t ready[kRing];
    uint64_t empty[kStages];
    uint64_t acc_full[kAcc];
    uint64_t sc_full[kScSlots], sc_empty[kScSlots];
    uint64_t prod_full[kProd], prod_empty[kProd];
    uint64_t amax_full[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
    int fixup_last;
    Tables tables;
};

__device__ __forceinline__ Unit unit(const Params& p, const Smem& s, int u) {
    return unit_of<kTokens>(p, s.tables, u);
}
// Columns of a tile's MMAs: its tokens rounded up to 32.
__device__ __forceinline__ int columns(const Unit& t) { return max(32, (t.n + 31) & ~31); }

// ---------------------------------------------------------------- producers (warps 0 and 3)
// Whole warps, one elected lane issuing: with one lane alone in the loop the addresses leave the uniform
// registers and a block took about 600 clk of issue. Warp 0 streams the weights, which no earlier kernel
// writes, from the start.
__device__ __forceinline__ void weight_producer(const Params& p, Smem& s, uint32_t rank, volatile int* abort_flag) {
    const int units = unit_count<kTokens>(p, s.tables);
    uint32_t it = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        const Unit t = unit(p, s, u);
        const uint8_t* w = weight_block(p, t, rank);
        for (int b = t.b0; b < t.b1; ++b, ++it, w += kTileBytes) {
            const int st = it % kStages;
            ok = __all_sync(0xFFFFFFFFu, dev::mbar_wait(&s.empty[st], ((it / kStages) & 1) ^ 1, abort_flag));
            if (!ok) break;
            if (elect_one()) {
                uint64_t* bar = &s.ready[it % kRing];
                dev::mbar_arrive_expect_tx(bar, kTileBytes);
                dev::bulk_g2s(s.w[st], w, kTileBytes, bar);
            }
            __syncwarp();
        }
    }
    if (!ok && elect_one()) fail(p, abort_flag);
    // the copies in flight must land before the CTA's shared memory is given up (after an abort the
    // even CTA's readiness may never be complete: a short bound, far longer than a copy)
    for (uint32_t k = 0; k < kStages && k < it; ++k) {
        const uint32_t i = it - 1 - k;
        dev::mbar_wait(&s.ready[i % kRing], (i / kRing) & 1, nullptr, ok ? dev::kMaxPolls : 1u << 16);
    }
}

// Warp 3: the token codes and scales of kScChunk blocks at a time, one box each.
__device__ __forceinline__ void token_producer(const Params& p, const CUtensorMap* codes, const CUtensorMap* scales,
                                               Smem& s, uint32_t rank, volatile int* abort_flag) {
    const int units = unit_count<kTokens>(p, s.tables);
    uint32_t ch = 0;
    bool ok = true;
    dev::pdl_wait();                // the codes and scales come from the kernel before
    dev::pdl_launch_dependents();   // (after the wait: see Fp8GemmArgs::pdl)
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        const Unit t = unit(p, s, u);
        const int row = static_cast<int>(t.row0), mine = row + static_cast<int>(rank) * (columns(t) >> 1);
        for (int b = t.b0; b < t.b1; b += kScChunk, ++ch) {
            const int sl = ch % kScSlots;
            ok = __all_sync(0xFFFFFFFFu, dev::mbar_wait(&s.sc_empty[sl], ((ch / kScSlots) & 1) ^ 1, abort_flag));
            if (!ok) break;
            if (elect_one()) {
                dev::mbar_arrive_expect_tx(&s.sc_full[sl], sizeof(s.sx[0]) + sizeof(s.x[0]));
                dev::tma_load_3d(s.x[sl], codes, 0, mine, b, &s.sc_full[sl]);
                dev::tma_load_2d(s.sx[sl], scales, row, b, &s.sc_full[sl]);
            }
            __syncwarp();
        }
    }
    if (!ok && elect_one()) fail(p, abort_flag);
    for (uint32_t k = 0; k < kScSlots && k < ch; ++k) {
        const uint32_t i = ch - 1 - k;
        dev::mbar_wait(&s.sc_full[i % kScSlots], (i / kScSlots) & 1, nullptr);
    }
}

// ---------------------------------------------------------------- MMA (warp 1)
__device__ __forceinline__ void mma_issuer(const Params& p, Smem& s, uint32_t rank, uint32_t tmem,
                                           volatile int* abort_flag) {
    const int units = unit_count<kTokens>(p, s.tables);
    const uint32_t leader = dev::mapa(&s.ready[0], 0);
    const uint64_t w0 = dev::sdesc_k_sw128(dev::smem_u32(s.w[0])), x0 = dev::sdesc_k_sw128(dev::smem_u32(s.x[0][0]));
    uint32_t it = 0, st = 0, ch = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        const Unit t = unit(p, s, u);
        const uint32_t idesc = dev::idesc_e4m3_f32(256, static_cast<uint32_t>(columns(t)));
        for (int b = t.b0; b < t.b1; ++b, ++it) {
            const int in_chunk = (b - t.b0) % kScChunk, sl = ch % kScSlots;
            const bool chunk_ends = in_chunk == kScChunk - 1 || b + 1 == t.b1;
            bool there = in_chunk != 0 || dev::mbar_wait(&s.sc_full[sl], (ch / kScSlots) & 1, abort_flag);
            there = there && dev::mbar_wait(&s.ready[it % kRing], (it / kRing) & 1, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, there);
            if (!ok) break;
            if (chunk_ends) ++ch;
            if (rank != 0) {
                if (elect_one()) dev::mbar_arrive_remote(leader + (it % kRing) * 8u);
                __syncwarp();
                continue;
            }
            dev::tc_fence_after();
            // (a descriptor's address field counts 16 bytes)
            const uint64_t ad = w0 + st * (kTileBytes / 16), bd = x0 + (sl * kScChunk + in_chunk) * (kTokens * 4);
            const uint32_t d = tmem + (it % kAcc) * kTokens;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) dev::mma_e4m3_pair(d, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
                dev::mma_commit_pair(&s.acc_full[it % kAcc]);
                dev::mma_commit_pair(&s.empty[st]);
                if (chunk_ends) dev::mma_commit_pair(&s.sc_empty[sl]);
            }
            __syncwarp();
            if (++st == kStages) st = 0;
        }
    }
    if (elect_one()) {
        if (!ok) fail(p, abort_flag);
        if (rank == 0) {   // every MMA must finish before TMEM is released
            dev::mma_commit_pair(&s.mma_done);
            dev::mbar_wait(&s.mma_done, 0, nullptr);
        }
    }
    __syncwarp();
}

// ---------------------------------------------------------------- scaler (warp 2)
template <bool kGated>
__device__ __forceinline__ void scaler(const Params& p, Smem& s, uint32_t rank, int lane,
                                       volatile int* abort_flag) {
    constexpr int kPer = kTokens / 32;   // tokens a lane
    const int units = unit_count<kTokens>(p, s.tables);
    uint32_t v = 0, ch = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        const Unit t = unit(p, s, u);
        // weight scales of 32 blocks, one a lane: this CTA's 128 channels, or gate and up
        const int srow = kGated ? t.pair : 2 * t.pair + static_cast<int>(rank);
        const float* ws = p.w_scales + static_cast<int64_t>(t.e) * p.scale_rows * p.nb;
        const float* ws0 = ws + static_cast<int64_t>(min(srow, p.scale_rows - 1)) * p.nb;
        const float* ws1 = kGated ? ws0 + static_cast<int64_t>(p.scale_rows / 2) * p.nb : ws0;
        auto scale_of = [&](const float* w, int b) { return b < t.b1 ? __ldg(w + b) : 0.0f; };
        float next0 = scale_of(ws0, t.b0 + lane), next1 = kGated ? scale_of(ws1, t.b0 + lane) : 0.0f;
        float cur0 = 0.0f, cur1 = 0.0f;
        for (int b = t.b0; b < t.b1; ++b, ++v) {
            const int i = b - t.b0, i32 = i & 31, in_chunk = i % kScChunk, sl = ch % kScSlots;
            if (i32 == 0) {
                cur0 = next0;
                cur1 = next1;
                next0 = scale_of(ws0, b + 32 + lane);
                if (kGated) next1 = scale_of(ws1, b + 32 + lane);
            }
            const float w0 = __shfl_sync(0xFFFFFFFFu, cur0, i32);
            const float w1 = kGated ? __shfl_sync(0xFFFFFFFFu, cur1, i32) : 0.0f;
            const int slot = v % kProd;
            bool there = in_chunk != 0 || dev::mbar_wait(&s.sc_full[sl], (ch / kScSlots) & 1, abort_flag);
            there = there && dev::mbar_wait(&s.prod_empty[slot], ((v / kProd) & 1) ^ 1, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, there);
            if (!ok) break;
            float x[kPer];
#pragma unroll
            for (int j = 0; j < kPer; j += 2)
                *reinterpret_cast<float2*>(x + j) = *reinterpret_cast<const float2*>(&s.sx[sl][in_chunk][lane * kPer + j]);
#pragma unroll
            for (int j = 0; j < kPer; j += 2) {
                *reinterpret_cast<float2*>(&s.prod[slot][0][lane * kPer + j]) = make_float2(x[j] * w0, x[j + 1] * w0);
                if (kGated)
                    *reinterpret_cast<float2*>(&s.prod[slot][1][lane * kPer + j]) = make_float2(x[j] * w1, x[j + 1] * w1);
            }
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(&s.prod_full[slot]);
            if (in_chunk == kScChunk - 1 || b + 1 == t.b1) {
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(&s.sc_empty[sl]);
                ++ch;
            }
        }
    }
    if (!ok && lane == 0) fail(p, abort_flag);
}

// ---------------------------------------------------------------- epilogue (warps 4-11)

// acc[c] += d * (scale product) for 32 tokens.
__device__ __forceinline__ void accumulate(const uint32_t (&d)[32], const float* prod, float2 (&acc)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(prod + 4 * i);
        acc[2 * i] = dev::ffma2(make_float2(__uint_as_float(d[4 * i]), __uint_as_float(d[4 * i + 1])), make_float2(f.x, f.y), acc[2 * i]);
        acc[2 * i + 1] = dev::ffma2(make_float2(__uint_as_float(d[4 * i + 2]), __uint_as_float(d[4 * i + 3])), make_float2(f.z, f.w), acc[2 * i + 1]);
    }
}

// The blocks of a unit for one epilogue warp: P of 32 tokens from TMEM, times the scale products, into
// acc. Straight-line inside a block: a TMEM load's 32 registers are one fixed run, and a load under a
// condition makes the compiler move all 32 of them at every join. Returns false when a wait gave up. v
// counts the blocks of this CTA. kTurns: the warp takes every second block (v % 2 == turn) and arrives
// for the warp that takes the others.
template <bool kTurns>
__device__ __forceinline__ bool sum_blocks(Smem& s, uint32_t base, const float* prod0, uint32_t leader_ready, int blocks,
                                           int lane, int turn, uint32_t& v, float2 (&acc)[16], volatile int* abort_flag) {
    constexpr uint32_t kArrivals = kTurns ? 2 : 1;
    constexpr int kProdFloats = sizeof(s.prod[0]) / sizeof(float);
    for (int left = blocks; left > 0; --left, ++v) {
        if (kTurns && static_cast<int>(v & 1) != turn) continue;
        const uint32_t slot = v % kProd;
        const bool there = dev::mbar_wait(&s.acc_full[v % kAcc], (v / kAcc) & 1, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, there)) return false;
        dev::tc_fence_after();
        uint32_t d[32];
        dev::tmem_ld32(base + (v % kAcc) * kTokens, d);
        if (!__all_sync(0xFFFFFFFFu, dev::mbar_wait(&s.prod_full[slot], (v / kProd) & 1, abort_flag))) return false;
        dev::tmem_ld_wait32(d);
        // all of it is in registers: the accumulator is free for block v + kAcc
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive_remote_n(leader_ready + ((v + kAcc) % kRing) * 8u, kArrivals);
        accumulate(d, prod0 + slot * kProdFloats, acc);
        __syncwarp();
        if (lane == 0) dev::mbar_arrive_n(&s.prod_empty[slot], kArrivals);
    }
    return true;
}

// Warp w covers TMEM lanes 32 (w % 4) .. + 31, one packed weight row a thread, and half of the
// tile's tokens (up to 32): acc[i] holds tokens c0 + 2i and + 1.
template <bool kGated>
__device__ __forceinline__ void epilogue(const Params& p, Smem& s, uint32_t rank, int warp, int lane, uint32_t tmem,
                                         volatile int* abort_flag) {
    const int units = unit_count<kTokens>(p, s.tables);
    const int ew = warp - 4, q = warp & 3, h = ew >> 2;
    const uint32_t leader_ready = dev::mapa(&s.ready[0], 0);
    uint32_t v = 0, nu = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; u < units; u += gridDim.x >> 1) {
        const Unit t = unit(p, s, u);
        // up to 32 tokens: the two warps of a quarter take the blocks in turn, each with all the columns
        const bool turns = columns(t) == 32;
        const int half = turns ? 32 : columns(t) >> 1, c0 = turns ? 0 : h * half;
        const int own = turns && h == 1 ? 0 : max(0, min(half, t.n - c0));   // tokens that this warp puts out
        const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c0);
        const float* prod0 = &s.prod[0][kGated ? lane >> 4 : 0][c0];
        float weight = 1.0f;   // of token c0 + lane
        if (!kGated && p.pair_weight != nullptr && lane < own) weight = __ldg(p.pair_weight + p.pair_of[t.row0 + c0 + lane]);
        float2 acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = make_float2(0.0f, 0.0f);

        if (ok) {
            const int blocks = t.b1 - t.b0;
            if (turns) ok = sum_blocks<true>(s, base, prod0, leader_ready, blocks, lane, h, v, acc, abort_flag);
            else ok = sum_blocks<false>(s, base, prod0, leader_ready, blocks, lane, 0, v, acc, abort_flag);
        }
        if (turns) {
            if (h == 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (2 * i < t.n) s.other_turn[i][32 * q + lane] = acc[i];
            }
            dev::named_bar_sync(4 + q, 64);
            if (h == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (2 * i < t.n) {
                        const float2 f = s.other_turn[i][32 * q + lane];
                        acc[i] = make_float2(acc[i].x + f.x, acc[i].y + f.y);
                    }
            }
            dev::named_bar_sync(4 + q, 64);   // read before the next unit's sums come
        }

        if constexpr (kGated) {
            // Lanes 0-15 hold the gate rows and lanes 16-31 the up rows of the same hidden channels. A
            // lane of the first half takes the even token of each pair, one of the second half the odd
            // one: h = silu(gate) * up for 16 tokens, kept in acc[i].x.
            const int l16 = lane & 15;
            const bool odd = lane >= 16;
            const unsigned mine = odd ? 0xFFFF0000u : 0x0000FFFFu;
            const int par = nu & 1;
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (2 * i >= own) break;   // (the same for the whole warp)
                const float2 f = acc[i];
                const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? f.x : f.y, 16);
                const float g = odd ? got : f.x, up = odd ? f.y : got;
                const float hv = silu_times(g, up);
                acc[i].x = hv;
                const float m = __uint_as_float(__reduce_max_sync(mine, __float_as_uint(fabsf(hv))));
                if (l16 == i) top = m;
            }
            // this lane's maximum is of token 2 l16 (+ 1)
            if (2 * l16 < own) s.amax[q][c0 + 2 * l16 + (odd ? 1 : 0)] = top;
            dev::named_bar_sync(2 + h, 128);
            // the four quarters' maximum of a token to the peer
            const int col = c0 + lane;
            if (q == 0 && lane < own) {
                const float m = max_magnitude(max_magnitude(s.amax[0][col], s.amax[1][col]), max_magnitude(s.amax[2][col], s.amax[3][col]));
                s.hscale[col] = m;
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dev::mapa(&s.amax_peer[par][col], rank ^ 1u)), "f"(m) : "memory");
            }
            __syncwarp();
            if (lane == 0) dev::mbar_arrive_remote_release(dev::mapa(&s.amax_full[par], rank ^ 1u));
            if (ok) ok = dev::mbar_wait_cluster(&s.amax_full[par], (nu >> 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (q == 0 && lane < own) {
                const float sc = __fdiv_rn(max_magnitude(s.hscale[col], s.amax_peer[par][col]), 448.0f);
                s.hscale[col] = sc;
                if (ok && rank == 0 && col < t.n) p.h_scales[t.pair * p.sstride + t.row0 + col] = sc;
            }
            dev::named_bar_sync(2 + h, 128);
            const int chunk16 = static_cast<int>(rank) * 4 + q;
            uint8_t* out = p.H + (static_cast<int64_t>(t.pair) * p.rows + t.row0) * 128 + l16;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (2 * i >= own) break;
                const int tok = c0 + 2 * i + (odd ? 1 : 0);
                if (!ok || tok >= t.n) continue;
                const float sc = s.hscale[tok];
                const uint32_t code = e4m3x2(sc > 0.0f ? __fdiv_rn(acc[i].x, sc) : 0.0f, 0.0f);
                out[static_cast<int64_t>(tok) * 128 + ((chunk16 ^ static_cast<int>((t.row0 + tok) & 7)) << 4)] = static_cast<uint8_t>(code);
            }
            ++nu;
        } else {
            const int n = 256 * t.pair + 128 * static_cast<int>(rank) + 32 * q + lane;
            auto store = [&](auto f32) {   // (FP32 outputs are the experts', whose K is not split)
                int64_t at = (t.row0 + c0) * p.ldy + n;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (i >= own) break;   // (the same for the whole warp)
                    const float w = __shfl_sync(0xFFFFFFFFu, weight, i);
                    if (ok && n < p.N) {
                        const float f = ((i & 1) ? acc[i >> 1].y : acc[i >> 1].x) * w;
                        if constexpr (f32.value) static_cast<float*>(p.Y)[at] = f;
                        else static_cast<uint16_t*>(p.Y)[at] = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
                    }
                    at += p.ldy;
                }
            };
            if (p.splits == 1 && p.f32) {
                store(std::true_type{});
            } else if (p.splits == 1) {
                store(std::false_type{});
            } else {
                // publish this split's sums; the last split to arrive adds all of them in split order
                auto slot_of = [&](int sp) {
                    return reinterpret_cast<float4*>(p.partial) +
                           (((static_cast<int64_t>(t.tile) * p.splits + sp) * 2 + rank) * kEpiWarps + ew) * (8 * 32) + lane;
                };
                float4* out = slot_of(t.split);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (4 * i < own)
                        __stcg(out + i * 32, make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y));
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
                    for (int i = 0; i < 16; ++i) acc[i] = make_float2(0.0f, 0.0f);
                    for (int sp = 0; sp < p.splits; ++sp) {
                        const float4* in = slot_of(sp);
                        float4 f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (4 * i < own) f[i] = __ldcg(in + i * 32);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (4 * i < own) {
                                acc[2 * i].x += f[i].x;
                                acc[2 * i].y += f[i].y;
                                acc[2 * i + 1].x += f[i].z;
                                acc[2 * i + 1].y += f[i].w;
                            }
                    }
                    store(std::false_type{});
                }
            }
        }
    }
    if (!ok) {
        dev::tmem_ld_wait();   // none in flight when TMEM is freed
        if (lane == 0) fail(p, abort_flag);
    }
}

template <bool kGated>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
fp8_few_kernel(const Params p, const __grid_constant__ CUtensorMap codes, const __grid_constant__ CUtensorMap scales) {
    extern __shared__ uint8_t smem_raw[];
    // (an offset from the array, so that the compiler still knows the accesses to be shared memory's)
    Smem& s = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (dev::smem_u32(smem_raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = dev::cluster_ctarank();
    if (threadIdx.x == 0) {
        dev::tma_prefetch_map(&codes);
        dev::tma_prefetch_map(&scales);
        for (int i = 0; i < kRing; ++i) dev::mbar_init(&s.ready[i], rank == 0 ? 2 + 2 * kEpiWarps : 1);
        for (int i = 0; i < kStages; ++i) dev::mbar_init(&s.empty[i], 1);
        for (int i = 0; i < kAcc; ++i) dev::mbar_init(&s.acc_full[i], 1);
        for (int i = 0; i < kScSlots; ++i) {
            dev::mbar_init(&s.sc_full[i], 1);
            dev::mbar_init(&s.sc_empty[i], 2);   // the scaler and the MMAs
        }
        for (int i = 0; i < kProd; ++i) {
            dev::mbar_init(&s.prod_full[i], 1);
            dev::mbar_init(&s.prod_empty[i], kEpiWarps);
        }
        for (int i = 0; i < 2; ++i) dev::mbar_init(&s.amax_full[i], kEpiWarps);
        dev::mbar_init(&s.mma_done, 1);
        s.abort_flag = 0;
        if (rank == 0)   // the first blocks find their accumulators free
            for (int i = 0; i < kAcc; ++i)
                for (int k = 0; k < 2 * kEpiWarps; ++k) dev::mbar_arrive(&s.ready[i]);
        dev::fence_barrier_init();
    }
    if (warp == 2) dev::tmem_alloc_pair(&s.tmem_base, kTmemCols);
    if (p.start != nullptr) fill_tables<kTokens>(p, s.tables, warp, lane);
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // both CTAs' barriers and TMEM exist before any traffic between them
    dev::tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    volatile int* abort_flag = &s.abort_flag;

    if (warp < 4) {
        if (warp == 0) {
            weight_producer(p, s, rank, abort_flag);
        } else if (warp == 1) {
            mma_issuer(p, s, rank, tmem, abort_flag);
        } else if (warp == 2) {
            scaler<kGated>(p, s, rank, lane, abort_flag);
        } else {
            token_producer(p, &codes, &scales, s, rank, abort_flag);
        }
        __syncwarp();
    } else {
        epilogue<kGated>(p, s, rank, warp, lane, tmem, abort_flag);
    }
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // the peer's MMAs, commits, stores and arrivals on this CTA are done
    if (warp == 2) {
        dev::tc_fence_after();
        dev::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory exceeds the 227 KB a CTA may use");

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Which kernel, from the rounds of tiles over the resident pairs of CTAs. A round of 256-token tiles takes 1.2
// to 1.4 times as long as one of 64-token tiles, so these are taken while they need less than 1.5 times the
// rounds. Measured, quantizer included: 128 tokens of 8192 x 8192 (one round each) 27.6 against 32.6 us, 256 tokens (two
// against one) 46.9 against 33.7; all of a routed feed-forward, 16 experts of 4096 x 2048 with 48 tokens each (4 rounds
// each) 111 against 120 us, with 96 (7 against 4) 170 against 131; 10 of 2012 x 1404 with 96 (3 against 2) 86 against 62.
// 128-token tiles, tried between the two, were slower than the better of them everywhere, and the last few tokens of an
// expert in a second launch of small tiles gained or lost 2%. Experts: their mean load, and a sixth more for its
// spread.
bool few_tokens(const fp8_layer& L, int64_t tokens, bool routed) {
    int64_t tiles64 = ceil_div(tokens, kTokens), tiles256 = ceil_div(tokens, 256);
    if (routed) {
        const int64_t used = tokens < L.experts ? tokens : L.experts, load = ceil_div(tokens * 7, used * 6);
        tiles64 = used * ceil_div(load, kTokens);
        tiles256 = used * ceil_div(load, 256);
    }
    const int pairs = fp8_resident_pairs(L);
    return 2 * ceil_div(tiles64 * L.pairs, pairs) < 3 * ceil_div(tiles256 * L.pairs, pairs);
}

// Dense tiles too few for the pairs: K is split, at least 4 blocks a split and at most 8 splits. Measured at
// 32 tokens: 1024 x 8192 in 1, 4, 8 and 16 splits 23.5, 16.5, 16.8 and 21.4 us; 8192 x 8192 in 1 and 2 25.3 and 23.5.
int splits_for(const fp8_layer& L, int64_t M) {
    if (L.experts > 1 || L.gated || !few_tokens(L, M, false)) return 1;
    const int64_t tiles = L.pairs * ceil_div(M, kTokens);
    const int pairs = fp8_resident_pairs(L);
    if (tiles * 2 > pairs) return 1;
    int64_t s = pairs / tiles;
    if (s > L.nb / 4) s = L.nb / 4;
    if (s > 8) s = 8;
    return s < 1 ? 1 : static_cast<int>(s);
}

size_t counter_bytes(const fp8_layer& L) { return (static_cast<size_t>(L.num_sms) * 2 * sizeof(int32_t) + 255) & ~size_t(255); }

}  // namespace
}  // namespace fp8

// The arrival counters come first, so that every size that shares a buffer finds zeros there.
size_t fp8_gemm_workspace(const fp8_layer& L, int64_t M) {
    const int splits = fp8::splits_for(L, M);
    if (splits == 1) return 0;
    const size_t tile_bytes = fp8::kTokens * 256 * sizeof(float);
    return fp8::counter_bytes(L) + static_cast<size_t>(L.pairs) * fp8::ceil_div(M, fp8::kTokens) * splits * tile_bytes;
}

cudaError_t launch_fp8_gemm(const fp8_layer& L, const Fp8GemmArgs& a, cudaStream_t stream) {
    const bool routed = a.start != nullptr;
    fp8::Params p{};
    p.A = static_cast<const uint8_t*>(a.A);
    p.W = static_cast<const uint8_t*>(a.W);
    p.w_scales = a.w_scales;
    p.start = a.start;
    p.count = a.count;
    p.pair_of = a.pair_of;
    p.pair_weight = a.pair_weight;
    p.rows = a.rows;
    p.sstride = scale_stride(a.rows);
    p.Y = a.Y;
    p.ldy = a.ldy;
    p.bf16 = a.dtype == kBF16;
    p.f32 = a.dtype == kF32;
    const uintptr_t y = reinterpret_cast<uintptr_t>(a.Y);
    if (p.f32) p.vec = a.ldy % 4 == 0 && (y & 15u) == 0 ? 4 : 1;
    else p.vec = a.ldy % 8 == 0 && (y & 15u) == 0 ? 8 : a.ldy % 4 == 0 && (y & 7u) == 0 ? 4 : 1;
    p.H = static_cast<uint8_t*>(a.H);
    p.h_scales = a.h_scales;
    p.M = static_cast<int>(a.rows);
    p.N = L.N;
    p.nb = L.nb;
    p.pairs = L.pairs;
    p.scale_rows = L.scale_rows;
    p.experts = L.experts;
    p.splits = a.workspace != nullptr ? fp8::splits_for(L, a.rows) : 1;
    p.status = L.d_status;
    if (p.splits > 1) {
        p.arrivals = static_cast<int32_t*>(a.workspace);
        p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + fp8::counter_bytes(L));
    }
    // an upper bound of the token tiles: a partial one per expert in use
    const bool few = fp8::few_tokens(L, a.pairs_routed, routed);
    const int most = few ? fp8::kTokens : 256;
    const int64_t used = routed ? (L.experts < a.pairs_routed ? L.experts : a.pairs_routed) : 0;
    const int64_t tiles = routed ? used + a.pairs_routed / most : fp8::ceil_div(a.rows, most);
    if (!few) return launch_fp8_wide(L, p, a.a_scales, tiles, a.pdl, stream);
    CUtensorMap codes, scales;
    if (!encode_code_map(&codes, a.A, a.rows, L.nb, fp8::kTokens / 2) ||
        !encode_scale_map(&scales, a.a_scales, p.sstride, L.nb, fp8::kTokens, fp8::kScChunk))
        return cudaErrorInvalidValue;
    const int64_t units = tiles * L.pairs * p.splits;
    const int grid = 2 * static_cast<int>(units < fp8_resident_pairs(L) ? units : fp8_resident_pairs(L));
    auto fn = L.gated ? fp8::fp8_few_kernel<true> : fp8::fp8_few_kernel<false>;
    return launch_pairs(fn, grid, fp8::kThreads, fp8::kSmemBytes, a.pdl, stream, p, codes, scales);
}

}  // namespace fmpq
