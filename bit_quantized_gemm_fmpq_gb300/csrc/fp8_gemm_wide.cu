// E4M3 product with a scale for each block of 128, for many tokens (sm_103a).
//
// A pair of CTAs computes 256 tokens x 256 packed weight rows. The tokens are on the tensor core's M
// side, so an epilogue thread owns one token: per block of 128 channels its partial sums P (FP32, in
// TMEM) take one factor, a_scale[b][m] * w_scale[.][b] (a gated layer: two), and cost nothing but a
// TMEM read and a packed multiply-add for two of them. With the weights on the M side (fp8_gemm.cu)
// every pair of sums needs its own factor from shared memory, and costs twice as much.
//
// Per block and CTA: 4 MMAs of 128 clk, 128 KB of TMEM reads, 32 K multiply-adds (256 clk of the FP32
// pipe), 32 KB of operands from L2. Measured at 4096 x 28672 x 8192: 0.68 ms with the quantizer, 2.8 PFLOP/s, 750 clk a
// block, of which the tensor pipe works 512; back to back the card reaches its power limit. The per-block work
// of the epilogue bounds it, not the tensor pipe or the copies. Tried and no faster: single-CTA MMAs with the weights
// multicast to both CTAs, 8 warps of 128 sums, 16-column loads, the sums kept as packed pairs, 2 blocks a loop iteration
// (it spills), waits with a time hint. Factors by chunks of 8 blocks, not 2: 0.83 to 0.75 ms; shared memory reached
// without generic addresses: 0.73 to 0.68; 5 operand stages cost nothing against 6, 3 cost 2%. The compiler spills 76
// bytes a thread in either form (96 registers at launch, before the roles take their shares).
//
// Warp roles (640 threads, one CTA per SM, pairs persistent over tiles):
//   warp 0      producer: token codes and weight block, token scales (a chunk of blocks at a time)
//   warps 1, 3  even CTA: MMA issuers of one half of the columns each; odd CTA: warp 1 reports its operands
//   warp 2      scaler: a chunk's token scales times its weight scales; also allocates and frees TMEM
//   warps 4-19  epilogue: TMEM lane quarter warp % 4 (32 tokens), 64 of the 256 columns each
#include "fp8_gemm.cuh"
#include "pieces.cuh"

namespace fmpq {
namespace fp8 {
namespace {

constexpr int kT = 256;      // tokens of a tile, 128 a CTA
constexpr int kAcc = 2;      // blocks with accumulators, two halves of 128 columns each
constexpr int kWideEpi = 16; // epilogue warps
constexpr int kWideThreads = 640;
constexpr int kChunk = 8;    // blocks of token scales per copy
constexpr int kSlots = 2;    // chunks of scales, and of factors

// kEpi: one operand block less in flight, for the whole tile of the residual
template <bool kEpi>
struct __align__(1024) Smem {
    static constexpr int kStages = kEpi ? 4 : 5;   // operand blocks in flight
    uint8_t x[kStages][kTileBytes];   // token codes: this CTA's 128 rows
    uint8_t w[kStages][kTileBytes];   // weight block: this CTA's tile, half of the pair's columns
    float sx[kSlots][kChunk][128];        // token scales
    float factor[kSlots][kChunk][2][128]; // times the weight scales: of the pair's two tiles, or gate and up
    union {
        float amax[2][4][128];        // gated: absmax of each quarter of a token's 128 hidden channels (units in turn)
        // of a warp's 32 tokens x 64 columns: 16 tokens of 16-bit outputs (kEpi: all), or 16 columns of FP32
        uint4 out[kWideEpi][(kEpi ? 32 : 16) * 8];
    };
    // full: a stage's operands have landed (even CTA: in both CTAs). empty: both halves' MMAs have read it.
    uint64_t full[kStages], empty[kStages];
    // [2 (b % kAcc) + half] of block b's accumulator: summed up; read by both CTAs' warps (even CTA)
    uint64_t acc_full[2 * kAcc], acc_free[2 * kAcc];
    uint64_t sc_full[kSlots], sc_empty[kSlots], factor_full[kSlots], factor_empty[kSlots];
    uint64_t mma_done[2];
    uint32_t tmem_base;
    int abort_flag;
    int4 unit[2];        // first row, tokens and pair tile of the epilogue's units (in turn), with their first factors
    Tables tables;
};

template <bool kEpi>
__device__ __forceinline__ Unit unit(const Params& p, const Smem<kEpi>& s, int u) { return unit_of<kT>(p, s.tables, u); }

template <bool kEpi>
__device__ __forceinline__ void producer(const Params& p, const CUtensorMap* scales, Smem<kEpi>& s, uint32_t rank,
                                         volatile int* abort_flag) {
    constexpr uint32_t kStages = Smem<kEpi>::kStages;
    const int units = unit_count<kT>(p, s.tables);
    uint32_t it = 0, ch = 0;
    bool ok = true;
    dev::pdl_wait();                // the codes and scales come from the kernel before
    dev::pdl_launch_dependents();   // (after the wait: see Fp8GemmArgs::pdl)
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        const Unit t = unit(p, s, u);
        const int local = static_cast<int>(rank) * 128;
        const uint32_t xbytes = static_cast<uint32_t>(max(0, min(128, t.n - local))) * 128u;
        const uint8_t* w = weight_block(p, t, rank);
        const uint8_t* x = p.A + (t.row0 + local + t.b0 * p.rows) * 128;
        for (int b = t.b0; b < t.b1; ++b, ++it) {
            if ((b - t.b0) % kChunk == 0) {
                const int sl = ch % kSlots;
                ok = dev::mbar_wait(&s.sc_empty[sl], ((ch / kSlots) & 1) ^ 1, abort_flag);
                if (!ok) break;
                dev::mbar_arrive_expect_tx(&s.sc_full[sl], sizeof(s.sx[0]));
                dev::tma_load_2d(s.sx[sl], scales, static_cast<int>(t.row0) + local, b, &s.sc_full[sl]);
                ++ch;
            }
            const uint32_t st = it % kStages;
            ok = dev::mbar_wait(&s.empty[st], ((it / kStages) & 1) ^ 1, abort_flag);
            if (!ok) break;
            uint64_t* bar = &s.full[st];
            dev::mbar_arrive_expect_tx(bar, kTileBytes + xbytes);
            dev::bulk_g2s(s.w[st], w, kTileBytes, bar);
            if (xbytes > 0) dev::bulk_g2s(s.x[st], x, xbytes, bar);
            w += kTileBytes;
            x += p.rows * 128;
        }
    }
    if (!ok) fail(p, abort_flag);
    // the copies in flight must land before the CTA's shared memory is given up
    for (uint32_t k = 0; k < kStages && k < it; ++k) {
        const uint32_t i = it - 1 - k;
        dev::mbar_drain(&s.full[i % kStages], (i / kStages) & 1, abort_flag);
    }
    for (uint32_t k = 0; k < kSlots && k < ch; ++k) {
        const uint32_t i = ch - 1 - k;
        dev::mbar_wait(&s.sc_full[i % kSlots], (i / kSlots) & 1, nullptr);
    }
}

// Even CTA: warps 1 and 3 issue the MMAs of one half of the columns each (weight rows 0-63 and 64-127 of both
// tiles), as its operands and its accumulator allow. Odd CTA: warp 1 reports its operands.
template <bool kEpi>
__device__ __forceinline__ void mma_issuer(const Params& p, Smem<kEpi>& s, uint32_t rank, int half, uint32_t tmem,
                                           volatile int* abort_flag) {
    constexpr uint32_t kStages = Smem<kEpi>::kStages;
    const int units = unit_count<kT>(p, s.tables);
    constexpr uint32_t kIdesc = dev::idesc_e4m3_f32(256, 128);
    const uint32_t leader = dev::mapa(&s.full[0], 0);
    // (a descriptor's address field counts 16 bytes; 64 weight rows are 8 KB)
    const uint64_t x0 = dev::sdesc_k_sw128(dev::smem_u32(s.x[0])), w0 = dev::sdesc_k_sw128(dev::smem_u32(s.w[0])) + half * 512;
    uint32_t it = 0, st = 0, phase = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1) {
        for (int b = 0; b < p.nb; ++b, ++it) {
            bool there = dev::mbar_wait(&s.full[st], phase, abort_flag);
            const uint32_t acc = 2 * (it % kAcc) + half;
            if (rank == 0) there = there && dev::mbar_wait(&s.acc_free[acc], ((it / kAcc) & 1) ^ 1, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, there);
            if (!ok) break;
            if (rank != 0) {
                if (elect_one()) dev::mbar_arrive_remote(leader + st * 8u);
            } else {
                dev::tc_fence_after();
                const uint64_t ad = x0 + st * (kTileBytes / 16), bd = w0 + st * (kTileBytes / 16);
                const uint32_t d = tmem + acc * 128u;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) dev::mma_e4m3_pair(d, ad + 2 * k, bd + 2 * k, kIdesc, k > 0 ? 1u : 0u);
                    dev::mma_commit_pair(&s.acc_full[acc]);
                    dev::mma_commit_pair(&s.empty[st]);
                }
            }
            __syncwarp();
            if (++st == kStages) {
                st = 0;
                phase ^= 1;
            }
        }
    }
    if (elect_one()) {
        if (!ok) fail(p, abort_flag);
        if (rank == 0) {   // every MMA must finish before TMEM is released
            dev::mma_commit_pair(&s.mma_done[half]);
            dev::mbar_wait(&s.mma_done[half], 0, nullptr);
        }
    }
    __syncwarp();
}

// ---------------------------------------------------------------- scaler (warp 2)
template <bool kGated, bool kEpi>
__device__ __forceinline__ void scaler(const Params& p, Smem<kEpi>& s, int lane, volatile int* abort_flag) {
    const int units = unit_count<kT>(p, s.tables);
    uint32_t ch = 0, nu = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok && u < units; u += gridDim.x >> 1, ++nu) {
        const Unit t = unit(p, s, u);
        // weight scales of 32 blocks, one a lane, of the pair's two tiles, or of gate and up
        const int srow = kGated ? t.pair : 2 * t.pair;
        const float* ws0 = p.w_scales + (static_cast<int64_t>(t.e) * p.scale_rows + srow) * p.nb + t.b0 + lane;
        const int to1 = kGated ? p.scale_rows / 2 * p.nb : (srow + 1 < p.scale_rows ? p.nb : 0);
        const int blocks = t.b1 - t.b0;
        auto scale_of = [&](int i, int off) { return i + lane < blocks ? __ldg(ws0 + i + off) : 0.0f; };
        float next0 = scale_of(0, 0), next1 = scale_of(0, to1), cur0 = 0.0f, cur1 = 0.0f;
        for (int i = 0; i < blocks; i += kChunk, ++ch) {
            const int sl = ch % kSlots;
            const uint32_t phase = (ch / kSlots) & 1;
            if ((i & 31) == 0) {
                cur0 = next0;
                cur1 = next1;
                next0 = scale_of(i + 32, 0);
                next1 = scale_of(i + 32, to1);
            }
            ok = dev::mbar_wait(&s.sc_full[sl], phase, abort_flag) && dev::mbar_wait(&s.factor_empty[sl], phase ^ 1, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
                const float w0 = __shfl_sync(0xFFFFFFFFu, cur0, (i + j) & 31), w1 = __shfl_sync(0xFFFFFFFFu, cur1, (i + j) & 31);
                const float4 x = *reinterpret_cast<const float4*>(&s.sx[sl][j][4 * lane]);
                *reinterpret_cast<float4*>(&s.factor[sl][j][0][4 * lane]) = make_float4(x.x * w0, x.y * w0, x.z * w0, x.w * w0);
                *reinterpret_cast<float4*>(&s.factor[sl][j][1][4 * lane]) = make_float4(x.x * w1, x.y * w1, x.z * w1, x.w * w1);
            }
            __syncwarp();
            if (lane == 0) {
                // (the unit two before has been read: its first factors have)
                if (i == 0) s.unit[nu & 1] = make_int4(static_cast<int>(t.row0), t.n, t.pair, 0);
                dev::mbar_arrive(&s.factor_full[sl]);
                dev::mbar_arrive(&s.sc_empty[sl]);
            }
        }
    }
    if (!ok && lane == 0) fail(p, abort_flag);
}

// acc += d * f for 32 columns, the first 16 with f0 and the others with f1.
__device__ __forceinline__ void accumulate(const uint32_t (&d)[32], float f0, float f1, float2 (&acc)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float f = i < 8 ? f0 : f1;
        acc[i] = dev::ffma2(make_float2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), make_float2(f, f), acc[i]);
    }
}

// A warp's 32 tokens x 64 columns to memory, 16 tokens at a time through shared memory (the 16-byte piece k of token l at
// k ^ (l % 8): no bank conflicts either way), so that a store instruction covers whole lines of 128 bytes; kW columns a
// lane and store. Pieces of 32 bytes of 16 rows cost 1.8 us a tile of 256 x 256 more.
template <int kW>
__device__ __forceinline__ void store_tile(const Params& p, uint4* stage, int lane, const float2 (&acc)[2][16], float weight,
                                           uint16_t* y, int tokens, int columns) {
    struct alignas(2 * kW) Piece {
        uint16_t v[kW];
    };
    uint32_t o[32];
    if (p.bf16) {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = pack16(acc[i >> 4][i & 15].x * weight, acc[i >> 4][i & 15].y * weight, true);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = pack16(acc[i >> 4][i & 15].x * weight, acc[i >> 4][i & 15].y * weight, false);
    }
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        if ((lane >> 4) == pass)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                stage[(lane & 15) * 8 + (k ^ (lane & 7))] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        __syncwarp();
#pragma unroll 4
        for (int j = 0; j < 32 / kW; ++j) {
            const int l = (32 * j + lane) / (64 / kW), n = (32 * j + lane) % (64 / kW) * kW;
            const Piece v = *reinterpret_cast<const Piece*>(reinterpret_cast<const uint16_t*>(&stage[l * 8 + ((n >> 3) ^ (l & 7))]) + (n & 7));
            if (16 * pass + l >= tokens) continue;
            uint16_t* to = y + (16 * pass + l) * p.ldy + n;
            if (n + kW <= columns) {
                *reinterpret_cast<Piece*>(to) = v;
            } else {
#pragma unroll
                for (int i = 0; i < kW; ++i)
                    if (n + i < columns) to[i] = v.v[i];
            }
        }
        __syncwarp();
    }
}

// The residual's tile of a warp into its stage (laid out as store_tile's, all 32 tokens): asked for before the tile's blocks,
// there when they are summed. What lies outside the matrix is 0.
template <int kW>
__device__ __forceinline__ void ask_residual(const Params& p, uint4* stage, int lane, const uint16_t* residual, int tokens, int columns) {
#pragma unroll 4
    for (int j = 0; j < 64 / kW; ++j) {
        const int l = (32 * j + lane) / (64 / kW), n = (32 * j + lane) % (64 / kW) * kW;
        uint16_t* to = reinterpret_cast<uint16_t*>(&stage[l * 8 + ((n >> 3) ^ (l & 7))]) + (n & 7);
        const uint16_t* from = residual + l * p.e.ldr + n;
        if (n + kW <= columns || n >= columns || l >= tokens) {
            const bool there = l < tokens && n < columns;
            dev::cp_async_if<2 * kW>(dev::smem_u32(to), there ? static_cast<const void*>(from) : p.e.residual, there);
        } else {
#pragma unroll
            for (int i = 0; i < kW; ++i) to[i] = l < tokens && n + i < columns ? from[i] : static_cast<uint16_t>(0);
        }
    }
}

// The same for rows that start anywhere, in the L2 by then and read when they are needed: in whole pieces, shifted. With store_rows: 2082 x
// 4078 to 3719 bf16, bias, silu, residual, 53 us; residual and outputs by single elements 67.
__device__ __forceinline__ void read_residual(const Params& p, uint4* stage, int lane, const uint16_t* residual, int tokens, int columns) {
    const int k = lane & 7;
#pragma unroll 2
    for (int j = 0; j < 8; ++j) {
        const int l = 4 * j + (lane >> 3);
        const uint16_t* from = residual + l * p.e.ldr;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (l < tokens && 8 * k + 8 <= columns) {
            v = eight_at(from, 8 * k);
        } else if (l < tokens) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (8 * k + 2 * i < columns ? from[8 * k + 2 * i] : 0u) | (8 * k + 2 * i + 1 < columns ? static_cast<uint32_t>(from[8 * k + 2 * i + 1]) << 16 : 0u);
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        stage[l * 8 + (k ^ (l & 7))] = v;
    }
}

// A warp's staged tile to rows that start anywhere: 7 whole pieces a row, shifted, and 8 elements at its two ends.
__device__ __forceinline__ void store_rows(const Params& p, const uint4* stage, int lane, uint16_t* y, int tokens, int columns) {
#pragma unroll 1
    for (int j = 0; j < 7; ++j) {
        const int i = 32 * j + lane, l = i / 7, k = i % 7 + 1;
        if (l >= tokens) continue;
        uint16_t* row = y + l * p.ldy;
        const int past = static_cast<int>(elements_past(row));
        const uint4 a = stage[l * 8 + ((k - 1) ^ (l & 7))], b = stage[l * 8 + (k ^ (l & 7))];
        const uint4 v = past == 0 ? b : shifted(a, b, 8u - past);
        const int n = 8 * k - past;
        if (n + 8 <= columns) {
            *reinterpret_cast<uint4*>(row + n) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (n + c < columns) row[n + c] = static_cast<uint16_t>(w[c >> 1] >> ((c & 1) * 16));
        }
    }
    const uint16_t* elements = reinterpret_cast<const uint16_t*>(stage);
#pragma unroll 4
    for (int j = 0; j < 8; ++j) {
        const int l = 4 * j + (lane >> 3), c = lane & 7;
        if (l >= tokens) continue;
        uint16_t* row = y + l * p.ldy;
        const int past = static_cast<int>(elements_past(row)), n = c < 8 - past ? c : 56 + c;
        if (n < columns) row[n] = elements[(l * 8 + ((n >> 3) ^ (l & 7))) * 8 + (n & 7)];
    }
}

// Bias and activation on a thread's token and 64 columns, its residual from the stage, the rounding; the outputs take the
// residual's place there and go out by whole lines. (The tile is read and written by this warp alone, so the residual may be Y.)
template <int kW>
__device__ __forceinline__ void store_tile_epilogue(const Params& p, uint4* stage, int lane, float2 (&acc)[2][16], uint16_t* y,
                                                    const uint16_t* residual, int n0, int tokens, int columns) {
    struct alignas(2 * kW) Piece {
        uint16_t v[kW];
    };
    const bool bf16 = p.bf16 != 0;
    if (residual != nullptr && kW == 1) read_residual(p, stage, lane, residual, tokens, columns);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (p.e.bias != nullptr) {
            const float b = 32 * c + lane < columns ? epi::bias_at(p.e, n0 + 32 * c + lane, bf16) : 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                acc[c][i].x += __shfl_sync(0xFFFFFFFFu, b, 2 * i);
                acc[c][i].y += __shfl_sync(0xFFFFFFFFu, b, 2 * i + 1);
            }
        }
        activate_all(p.e.act, acc[c]);
    }
    if (kW > 1) dev::cp_async_wait_all();
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint4* at = &stage[lane * 8 + (k ^ (lane & 7))];
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = acc[k >> 2][4 * (k & 3) + i];
        if (residual != nullptr) {
            const uint4 r = *at;
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = epi::values16(w[i], bf16);
                f[i] = make_float2(f[i].x + a.x, f[i].y + a.y);
            }
        }
        *at = make_uint4(pack16(f[0].x, f[0].y, bf16), pack16(f[1].x, f[1].y, bf16), pack16(f[2].x, f[2].y, bf16),
                         pack16(f[3].x, f[3].y, bf16));
    }
    __syncwarp();
    if (kW == 1) {
        store_rows(p, stage, lane, y, tokens, columns);
        __syncwarp();
        return;
    }
#pragma unroll 4
    for (int j = 0; j < 64 / kW; ++j) {
        const int l = (32 * j + lane) / (64 / kW), n = (32 * j + lane) % (64 / kW) * kW;
        const Piece v = *reinterpret_cast<const Piece*>(reinterpret_cast<const uint16_t*>(&stage[l * 8 + ((n >> 3) ^ (l & 7))]) + (n & 7));
        if (l >= tokens) continue;
        uint16_t* to = y + l * p.ldy + n;
        if (n + kW <= columns) {
            *reinterpret_cast<Piece*>(to) = v;
        } else {
#pragma unroll
            for (int i = 0; i < kW; ++i)
                if (n + i < columns) to[i] = v.v[i];
        }
    }
    __syncwarp();
}

// The same for FP32 outputs (a routed product whose rows are still to be summed), all 32 tokens and 16 columns at a time
// (piece k of token l at k ^ (l / 2 % 4)), every lane staging its own token; kW 4 or 1. 8 tokens and whole lines at a
// time leave three quarters of the lanes idle at the staging: 793 against 772 us for 4096 tokens through 8 of 128
// experts of 4096 x 1024.
template <int kW>
__device__ __forceinline__ void store_tile_f32(const Params& p, uint4* stage, int lane, const float2 (&acc)[2][16], float weight,
                                               float* y, int tokens, int columns) {
    struct alignas(4 * kW) Piece {
        float v[kW];
    };
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 a = acc[pass >> 1][8 * (pass & 1) + 2 * k], b = acc[pass >> 1][8 * (pass & 1) + 2 * k + 1];
            stage[lane * 4 + (k ^ ((lane >> 1) & 3))] =
                make_uint4(__float_as_uint(a.x * weight), __float_as_uint(a.y * weight), __float_as_uint(b.x * weight), __float_as_uint(b.y * weight));
        }
        __syncwarp();
#pragma unroll 4
        for (int j = 0; j < 16 / kW; ++j) {
            const int l = (32 * j + lane) / (16 / kW), m = (32 * j + lane) % (16 / kW) * kW, n = 16 * pass + m;
            const Piece v = *reinterpret_cast<const Piece*>(reinterpret_cast<const float*>(&stage[l * 4 + ((m >> 2) ^ ((l >> 1) & 3))]) + (m & 3));
            if (l >= tokens) continue;
            float* to = y + l * p.ldy + n;
            if (n + kW <= columns) {
                *reinterpret_cast<Piece*>(to) = v;
            } else {
#pragma unroll
                for (int i = 0; i < kW; ++i)
                    if (n + i < columns) to[i] = v.v[i];
            }
        }
        __syncwarp();
    }
}

// (behind the waits of this thread: volatile)
__device__ __forceinline__ float load_shared(uint32_t address) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(address) : "memory");
    return v;
}

// Thread: token 32 (warp % 4) + lane of this CTA's 128; columns 64 h .. + 63 of the accumulator: packed rows
// 64 (h / 2) .. + 63 of tile 2 pair + h % 2, acc[c][i] rows 32c + 2i and + 1 of them. The columns' halves have
// accumulators, barriers and MMAs of their own, so one half's arithmetic runs while the other waits
// for its MMAs. A warp has one TMEM load in flight (a wait covers all of a warp's loads), so four warps
// a scheduler hide them for each other. The blocks of a unit run straight-line: a TMEM load under a
// condition makes the compiler move its 32 registers at every join. A wait that gives up is remembered,
// and the unit's outputs are not stored.
template <bool kGated, bool kEpi>
__device__ __forceinline__ void epilogue(const Params& p, Smem<kEpi>& s, uint32_t rank, int warp, int lane, uint32_t tmem,
                                         volatile int* abort_flag) {
    if (kEpi) dev::pdl_wait();   // bias and residual may come from the kernel before
    const int units = unit_count<kT>(p, s.tables);
    const int q = warp & 3, h = (warp - 4) >> 2;
    const int local = 32 * q + lane;
    const int half = h >> 1, sub = h & 1;
    const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + 64u * h;
    const uint32_t leader_free = dev::mapa(&s.acc_free[half], 0);
    const uint32_t acc_full = dev::smem_u32(&s.acc_full[half]), factor_full = dev::smem_u32(&s.factor_full[0]);
    const uint32_t factors = dev::smem_u32(&s.factor[0][0][kGated ? 0 : sub][local]);
    uint32_t slot = 0, phase = 0;     // of the next block's accumulator
    uint32_t chunk = 0, chunk_phase = 0;
    uint32_t nu = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; u < units; u += gridDim.x >> 1) {
        ok &= wait_at(factor_full + chunk * 8u, chunk_phase, abort_flag);
        const int4 info = s.unit[nu++ & 1];
        const int row0 = info.x, n = info.y, pair = info.z;
        const int tok = static_cast<int>(rank) * 128 + local;
        const int64_t row = row0 + tok;
        float weight = 1.0f;   // of this thread's token
        if (!kGated && ok && p.pair_weight != nullptr && tok < n) weight = __ldg(p.pair_weight + p.pair_of[row]);
        // this warp's tile: token of lane 0 (in the unit), first column
        const int first = static_cast<int>(rank) * 128 + 32 * q, n0 = 256 * pair + 128 * sub + 64 * half;
        if constexpr (kEpi) {
            if (p.e.residual != nullptr && ok) {
                const uint16_t* r = static_cast<const uint16_t*>(p.e.residual) + (static_cast<int64_t>(row0) + first) * p.e.ldr + n0;
                if (p.vec == 8) ask_residual<8>(p, s.out[warp - 4], lane, r, n - first, p.N - n0);
                else if (p.vec == 4) ask_residual<4>(p, s.out[warp - 4], lane, r, n - first, p.N - n0);
                else if (lane < n - first && n0 < p.N) {
                    const uint16_t* row = r + lane * p.e.ldr;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(row + (p.N - n0 < 64 ? p.N - n0 : 64) - 1));
                }
            }
        }
        float2 acc[2][16];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c][i] = make_float2(0.0f, 0.0f);
        // (little besides the loads and the arithmetic: with the scales and the rings' index arithmetic in
        // it, this loop's own instructions took most of a block's time)
#pragma unroll 1
        for (int i = 0; i < p.nb; ++i) {
            const int j = i % kChunk;
            if (j == 0) ok &= wait_at(factor_full + chunk * 8u, chunk_phase, abort_flag);
            const uint32_t f = factors + (chunk * kChunk + j) * static_cast<uint32_t>(sizeof(s.factor[0][0]));
            const float f0 = load_shared(f), f1 = kGated ? load_shared(f + sizeof(s.factor[0][0][0])) : f0;
            ok &= wait_at(acc_full + slot * 16u, phase, abort_flag);
            __syncwarp();
            dev::tc_fence_after();
            const uint32_t at = base + slot * 256u;
            uint32_t d[32];
            dev::tmem_ld32(at, d);
            dev::tmem_ld_wait32(d);
            accumulate(d, f0, f1, acc[0]);
            dev::tmem_ld32(at + 32u, d);
            dev::tmem_ld_wait32(d);
            // all of it is in registers: the accumulator is free
            dev::tc_fence_before();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive_remote(leader_free + slot * 16u);
            if (j == kChunk - 1 || i + 1 == p.nb) {
                if (lane == 0) dev::mbar_arrive(&s.factor_empty[chunk]);
                chunk ^= 1;
                chunk_phase ^= chunk ^ 1;
            }
            slot ^= 1;
            phase ^= slot ^ 1;
            accumulate(d, f0, f1, acc[1]);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);

        const bool mine = ok && tok < n;
        if constexpr (kGated) {
            // acc[c][0..7] gates and acc[c][8..15] ups of 16 hidden channels: h = silu(gate) * up, kept
            // in the gates' place
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float2& g = acc[c][i];
                    g = make_float2(silu_times(g.x, acc[c][i + 8].x), silu_times(g.y, acc[c][i + 8].y));
                    top = max_magnitude(top, max_magnitude(fabsf(g.x), fabsf(g.y)));
                }
            // the block's other channels are with the same lane of the other three column warps; a warp
            // two units ahead has seen the others arrive for the unit between, after their reads
            const int par = nu & 1;
            s.amax[par][h][local] = top;
            dev::named_bar_sync(2 + q, 128);
            const float scale = __fdiv_rn(max_magnitude(max_magnitude(s.amax[par][0][local], s.amax[par][1][local]),
                                                        max_magnitude(s.amax[par][2][local], s.amax[par][3][local])), 448.0f);
            if (mine) {
                uint8_t* out = p.H + (static_cast<int64_t>(pair) * p.rows + row) * 128;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[4] = {0u, 0u, 0u, 0u};
                    if (scale > 0.0f) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 g = acc[c][i];
                            o[i >> 1] |= e4m3x2(__fdiv_rn(g.x, scale), __fdiv_rn(g.y, scale)) << (16 * (i & 1));
                        }
                    }
                    *reinterpret_cast<uint4*>(out + (((4 * sub + 2 * half + c) ^ static_cast<int>(row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                if (h == 0) p.h_scales[pair * p.sstride + row] = scale;
            }
        } else {
            const int64_t at = (static_cast<int64_t>(row0) + first) * p.ldy + n0;
            uint16_t* y = static_cast<uint16_t*>(p.Y) + at;
            const int tokens = ok ? n - first : 0, columns = p.N - n0;
            if constexpr (kEpi) {
                const uint16_t* r = static_cast<const uint16_t*>(p.e.residual);
                if (r != nullptr) r += (static_cast<int64_t>(row0) + first) * p.e.ldr + n0;
                if (p.vec == 8) store_tile_epilogue<8>(p, s.out[warp - 4], lane, acc, y, r, n0, tokens, columns);
                else if (p.vec == 4) store_tile_epilogue<4>(p, s.out[warp - 4], lane, acc, y, r, n0, tokens, columns);
                else store_tile_epilogue<1>(p, s.out[warp - 4], lane, acc, y, r, n0, tokens, columns);
            } else if (p.f32) {
                float* yf = static_cast<float*>(p.Y) + at;
                if (p.vec == 4) store_tile_f32<4>(p, s.out[warp - 4], lane, acc, weight, yf, tokens, columns);
                else store_tile_f32<1>(p, s.out[warp - 4], lane, acc, weight, yf, tokens, columns);
            } else if (p.vec == 8) store_tile<8>(p, s.out[warp - 4], lane, acc, weight, y, tokens, columns);
            else if (p.vec == 4) store_tile<4>(p, s.out[warp - 4], lane, acc, weight, y, tokens, columns);
            else store_tile<1>(p, s.out[warp - 4], lane, acc, weight, y, tokens, columns);
        }
    }
    if (!ok && lane == 0) fail(p, abort_flag);
}

template <bool kGated, bool kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
fp8_wide_kernel(const Params p, const __grid_constant__ CUtensorMap scales) {
    extern __shared__ uint8_t smem_raw[];
    // (an offset from the array, so that the compiler still knows the accesses to be shared memory's)
    Smem<kEpi>& s = *reinterpret_cast<Smem<kEpi>*>(smem_raw + ((1024u - (dev::smem_u32(smem_raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = dev::cluster_ctarank();
    if (threadIdx.x == 0) {
        dev::tma_prefetch_map(&scales);
        for (int i = 0; i < Smem<kEpi>::kStages; ++i) {
            dev::mbar_init(&s.full[i], rank == 0 ? 2 : 1);
            dev::mbar_init(&s.empty[i], 2);
        }
        for (int i = 0; i < 2 * kAcc; ++i) {
            dev::mbar_init(&s.acc_full[i], 1);
            dev::mbar_init(&s.acc_free[i], kWideEpi);   // half the warps of both CTAs
        }
        for (int i = 0; i < kSlots; ++i) {
            dev::mbar_init(&s.sc_full[i], 1);
            dev::mbar_init(&s.sc_empty[i], 1);
            dev::mbar_init(&s.factor_full[i], 1);
            dev::mbar_init(&s.factor_empty[i], kWideEpi);
        }
        for (int i = 0; i < 2; ++i) dev::mbar_init(&s.mma_done[i], 1);
        s.abort_flag = 0;
        dev::fence_barrier_init();
    }
    if (warp == 2) dev::tmem_alloc_pair(&s.tmem_base, kTmemCols);
    if (p.start != nullptr) fill_tables<kT>(p, s.tables, warp, lane);
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // both CTAs' barriers and TMEM exist before any traffic between them
    dev::tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    volatile int* abort_flag = &s.abort_flag;

    if (warp < 4) {
        dev::setmaxnreg_dec<32>();
        if (warp == 0) {
            if (lane == 0) producer(p, &scales, s, rank, abort_flag);
        } else if (warp == 1) {
            mma_issuer(p, s, rank, 0, tmem, abort_flag);
        } else if (warp == 2) {
            scaler<kGated>(p, s, lane, abort_flag);
        } else if (rank == 0) {
            mma_issuer(p, s, rank, 1, tmem, abort_flag);
        }
        __syncwarp();
    } else {
        dev::setmaxnreg_inc<112>();   // 128 x 32 + 512 x 112 = the 640 x 96 of the launch
        epilogue<kGated, kEpi>(p, s, rank, warp, lane, tmem, abort_flag);
    }
    dev::tc_fence_before();
    __syncthreads();
    dev::cluster_sync();   // the peer's MMAs, commits and arrivals on this CTA are done
    if (warp == 2) {
        dev::tc_fence_after();
        dev::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

constexpr size_t kSmemBytes = (sizeof(Smem<false>) > sizeof(Smem<true>) ? sizeof(Smem<false>) : sizeof(Smem<true>)) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory exceeds the 227 KB a CTA may use");

}  // namespace
}  // namespace fp8

// The persistent grids never launch more pairs than can be resident; asked once per device.
int fp8_resident_pairs(const fp8_layer& L) {
    static int cached[64] = {};
    if (L.device >= 0 && L.device < 64 && cached[L.device] > 0) return cached[L.device];
    int pairs = L.num_sms / 2 > 0 ? L.num_sms / 2 : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(fp8::kWideThreads);
    cfg.dynamicSmemBytes = fp8::kSmemBytes;
    int clusters = 0;
    if (ensure_smem_limit(reinterpret_cast<const void*>(fp8::fp8_wide_kernel<false, false>), static_cast<int>(fp8::kSmemBytes)) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, fp8::fp8_wide_kernel<false, false>, &cfg) == cudaSuccess && clusters > 0 && clusters < pairs)
        pairs = clusters;
    cudaGetLastError();   // a failed query leaves no error behind
    if (L.device >= 0 && L.device < 64) cached[L.device] = pairs;
    return pairs;
}

bool encode_code_map(CUtensorMap* map, const void* codes, int64_t rows, int nb, int tokens) {
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(nb)};
    const cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(rows) * 128};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(tokens), fp8::kScChunk}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_scale_map(CUtensorMap* map, const float* scales, int64_t sstride, int nb, int tokens, int blocks) {
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(sstride), static_cast<cuuint64_t>(nb)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(sstride) * sizeof(float)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(tokens), static_cast<cuuint32_t>(blocks)}, step[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(scales), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_fp8_wide(const fp8_layer& L, const fp8::Params& p, const float* a_scales, int64_t tiles, bool pdl,
                            cudaStream_t stream) {
    CUtensorMap map;
    if (!encode_scale_map(&map, a_scales, p.sstride, L.nb, 128, fp8::kChunk)) return cudaErrorInvalidValue;
    const int64_t units = tiles * L.pairs;
    const int grid = 2 * static_cast<int>(units < fp8_resident_pairs(L) ? units : fp8_resident_pairs(L));
    auto fn = L.gated ? fp8::fp8_wide_kernel<true, false> : p.e.any() ? fp8::fp8_wide_kernel<false, true> : fp8::fp8_wide_kernel<false, false>;
    return launch_pairs(fn, grid, fp8::kWideThreads, fp8::kSmemBytes, pdl, stream, p, map);
}

}  // namespace fmpq
