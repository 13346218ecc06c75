// Internals of the layers kept in 16 bits (w16_*).
#pragma once

#include "fp8_internal.h"

struct w16_layer {
    int32_t K = 0, N = 0, experts = 0;
    int32_t gated = 0;   // N = 2F: F gate rows, then F up rows
    int32_t dtype = 0;   // of weights and activations
    int32_t nb = 0;      // blocks of 64 input channels (the last may be partial)
    int32_t pairs = 0;   // pair tiles of 256 packed weight rows per expert
    int device = -1;
    int num_sms = 0;
    int32_t* d_status = nullptr;
};

namespace fmpq {

constexpr int kW16Block = 64;   // channels of a block: a packed tile of 128 rows is 16 KB (kTileBytes), as an E4M3 one is

struct W16Args {
    const void* X;              // [rows][ldx], rows on 16-byte boundaries
    int64_t ldx, rows;
    const void* W;
    const int32_t* start;       // experts: first row of each, and row counts; nullptr: one group of all rows
    const int32_t* count;       // nullptr: start has experts + 1 entries, each group ending where the next begins
    const float* row_weight;    // scales a row's outputs before the residual (nullptr: 1)
    const int32_t* pair_of;     // row r has row_weight[pair_of[r]] (nullptr: row_weight[r])
    Epilogue epilogue;          // bias [experts][N]
    void* Y;                    // of type dtype: the layer's, or FP32
    int dtype;
    int64_t ldy;
    // 0, or the failure-detection test (a plain layer without an epilogue): polls before a wait gives up, and the copy of weights that a CTA leaves out
    uint32_t polls;
    int withheld_cta, withheld_copy;
};
cudaError_t launch_w16_gemm(const w16_layer& L, const W16Args& a, cudaStream_t stream);
cudaError_t launch_w16_pack(const w16_layer& L, int expert, const void* W, int64_t ld_n, int64_t ld_k, void* Wp, cudaStream_t stream);
// X's rows to rows of `ld` elements (a multiple of 8) on 16-byte boundaries: row m to row m, or to the rows row_of[m * slots ..
// + slots) that are not negative.
cudaError_t launch_w16_rows(const void* X, int64_t ldx, int64_t rows, int K, const int32_t* row_of, int slots, void* out, int64_t ld,
                            int num_sms, cudaStream_t stream);

}  // namespace fmpq
