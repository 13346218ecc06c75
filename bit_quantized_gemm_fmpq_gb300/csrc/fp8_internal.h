// Internals of the E4M3 linear layers (fp8_*) and the routed experts (moe_*).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

struct fp8_layer {
    int32_t K = 0, N = 0, experts = 0;
    int32_t gated = 0;      // N = 2F: F gate rows, then F up rows
    int32_t nb = 0;         // blocks of 128 input channels (the last may be partial)
    int32_t pairs = 0;      // pair tiles of 256 packed weight rows per expert
    int32_t scale_rows = 0; // rows of the weight scales per expert
    int device = -1;
    int num_sms = 0;
    int32_t* d_status = nullptr;
};

namespace fmpq {

constexpr int kFp8Block = 128;
constexpr int kTileBytes = 128 * 128;   // one operand tile: 128 rows of 128 codes
constexpr int kMaxFp8Experts = 512;

// ---------------------------------------------------------------- the packed weight layout
// A pair tile is two tiles of 128 weight rows, one for each CTA of a pair; its blocks follow one
// another: tile t of an expert holds [nb][128 rows][128 codes], the 16-byte chunk c of row r at
// position c ^ (r % 8) (the 128-byte-swizzled K-major operand tile, one bulk copy of 16 KB).
// Plain layer: row p of tile t is channel 128t + p. Gated layer: rows 32q .. 32q + 15 are gate rows
// and rows 32q + 16 .. 32q + 31 the up rows of the hidden channels 64t + 16q .. + 15, so a warp of
// the product's epilogue holds both of a channel and the two tiles of a pair cover a block of 128.
// Returns the weight row (of N) held by row `p` of tile `t`, or -1 past the last one.
__host__ __device__ inline int fp8_source_row(int t, int p, int N, int gated) {
    if (!gated) return 128 * t + p < N ? 128 * t + p : -1;
    const int F = N / 2, f = 64 * t + 16 * (p >> 5) + (p & 15);
    if (f >= F) return -1;
    return (p & 16) ? F + f : f;
}
// Row of the weight scales that weight row n belongs to.
__host__ __device__ inline int fp8_scale_row(int n, int N, int gated) {
    if (!gated) return n >> 7;
    const int F = N / 2;
    return n < F ? n >> 7 : ((F + 127) >> 7) + ((n - F) >> 7);
}

// Rows of the experts' buffers: every expert's rows start at a multiple of 8 (the phase of the
// swizzle), so each expert that has tokens may cost up to 7 rows more.
inline int64_t moe_rows_of(int64_t T, int64_t k, int64_t E) {
    const int64_t P = T * k;
    return (P + 7 * (E < P ? E : P) + 7) / 8 * 8;
}
__host__ __device__ inline int64_t scale_stride(int64_t rows) { return (rows + 3) / 4 * 4; }   // fp32 rows of 16 bytes

// The plan's parts (int32): first row and row count of each expert, the row of each (token, slot)
// pair (-1: none), the pair of each row.
struct MoePlan {
    const int32_t* start;
    const int32_t* count;
    const int32_t* row_of;
    const int32_t* pair_of;
};
inline MoePlan moe_plan_parts(const void* plan, int64_t T, int64_t k, int64_t E) {
    const int32_t* p = static_cast<const int32_t*>(plan);
    return MoePlan{p, p + E, p + 2 * E, p + 2 * E + T * k};
}

// ---------------------------------------------------------------- launchers
enum { kF16 = 0, kBF16 = 1, kF32 = 2 };

// rows/positions: nullptr writes token m to row m; otherwise token m goes to the rows
// positions[m * slots .. + slots) that are not negative.
cudaError_t launch_fp8_quantize(const void* X, int dtype, int64_t ldx, int64_t M, int K, const int32_t* positions,
                                int slots, int64_t rows, void* A, float* scales, int num_sms, bool pdl,
                                cudaStream_t stream);
cudaError_t launch_fp8_pack_weights(const fp8_layer& L, int expert, const void* W, int dtype, int64_t ldw, void* Wp,
                                    float* scales, cudaStream_t stream);
cudaError_t launch_fp8_pack_codes(const fp8_layer& L, int expert, const void* codes, int64_t ldw, void* Wp,
                                  cudaStream_t stream);
cudaError_t launch_fp8_unpack(const fp8_layer& L, int expert, const void* Wp, const float* scales, float* W,
                              cudaStream_t stream);

struct Fp8GemmArgs {
    const void* A;
    const float* a_scales;
    const void* W;
    const float* w_scales;
    int64_t rows;             // rows of A (and of Y, H)
    // experts: first row, rows and pairs of the plan; nullptr for a dense layer
    const int32_t* start;
    const int32_t* count;
    const int32_t* pair_of;
    const float* pair_weight; // scales a row's outputs (nullptr: 1)
    int64_t pairs_routed;     // T * k, an upper bound of the rows in use (dense: rows)
    void* Y;                  // plain layer: output of type dtype (FP32: experts only)
    int dtype;
    int64_t ldy;
    void* H;                  // gated layer: E4M3 codes [F/128][rows][128] and scales
    float* h_scales;
    void* workspace;
    // Launched as the programmatic dependent of this library's kernel before it: its prologue, and the
    // weights' stream, start while that one runs; only its codes and scales are waited for. Every kernel
    // launched so lets its own dependent start after its wait, so what was written two launches
    // before (the plan) is complete from the start.
    bool pdl;
};
cudaError_t launch_fp8_gemm(const fp8_layer& L, const Fp8GemmArgs& a, cudaStream_t stream);
// Workspace of a dense product of M rows (0: none needed), zero before its first use.
size_t fp8_gemm_workspace(const fp8_layer& L, int64_t M);

struct RouteArgs {
    const void* logits;
    int dtype;
    int64_t ldl, T;
    int E, k, sigmoid, groups, top_groups, group_top, renormalize;
    float scale;
    const float* bias;
    int32_t* ids;
    float* weights;
};
cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_moe_plan(const int32_t* ids, int64_t T, int k, int E, int32_t* plan, int32_t* counts,
                            cudaStream_t stream);
cudaError_t launch_moe_combine(const void* D, int d_dtype, int64_t ldd, const int32_t* row_of, int64_t T, int k, int N,
                               void* Y, int dtype, int64_t ldy, bool pdl, cudaStream_t stream);

// Launch; pdl: as the programmatic dependent of the launch before it.
template <typename... P, typename... A>
cudaError_t launch_after(void (*fn)(P...), dim3 grid, int threads, size_t smem, bool pdl, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

}  // namespace fmpq
