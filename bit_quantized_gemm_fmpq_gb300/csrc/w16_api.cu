// C ABI of the layers kept in 16 bits (declared in include/fmpq.h): argument validation, layer handles, and kernel launches
// on the caller's stream.
#include <cstdint>
#include <new>

#include "../../include/fmpq.h"
#include "api_checks.h"
#include "w16_internal.h"

namespace {

using namespace fmpq::api;

fmpq_status check_device(const w16_layer* L) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return FMPQ_ERR_CUDA;
    return dev == L->device ? FMPQ_OK : FMPQ_ERR_DEVICE;
}

// TMA reads rows that start on 16-byte boundaries; others are copied to such rows first. (One row has no stride.)
int64_t aligned_ld(const w16_layer* L) { return (L->K + 7) / 8 * 8; }
bool rows_aligned(const void* X, int64_t ldx, int64_t rows) { return aligned16(X) && (ldx % 8 == 0 || rows == 1); }

// What every product checks, but for X and the workspace.
fmpq_status product_ok(const w16_layer* L, const void* X, int64_t ldx, int64_t rows, const void* W_packed, const fmpq_epilogue* e,
                       const float* row_weight, const void* Y, int32_t dtype, int64_t ldy) {
    if (L == nullptr || X == nullptr || W_packed == nullptr || Y == nullptr || (dtype != L->dtype && dtype != FMPQ_DTYPE_F32))
        return FMPQ_ERR_INVALID_ARG;
    const int64_t N = L->gated ? L->N / 2 : L->N;
    if (rows < 1 || rows > kMaxRows || ldx < L->K || ldy < N) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(W_packed) || !element_aligned(X, L->dtype) || !element_aligned(Y, dtype) || !element_aligned(row_weight, FMPQ_DTYPE_F32))
        return FMPQ_ERR_MISALIGNED;
    return epilogue_ok(e, dtype, N);
}
fmpq_status workspace_ok(size_t need, const void* workspace, size_t workspace_bytes) {
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FMPQ_ERR_WORKSPACE;
    return need > 0 && !aligned16(workspace) ? FMPQ_ERR_MISALIGNED : FMPQ_OK;
}
fmpq::W16Args args_of(const w16_layer* L, const void* X, int64_t ldx, int64_t rows, const void* W_packed, const fmpq_epilogue* e,
                      const float* row_weight, void* Y, int32_t dtype, int64_t ldy) {
    fmpq::W16Args a{};
    a.X = X;
    a.ldx = ldx % 8 == 0 ? ldx : aligned_ld(L);   // (one row, or replaced by the workspace)
    a.rows = rows;
    a.W = W_packed;
    a.row_weight = row_weight;
    a.epilogue = epilogue_of(e);
    a.Y = Y;
    a.dtype = dtype;
    a.ldy = ldy;
    return a;
}

fmpq_status product(const w16_layer* L, const void* X, int64_t ldx, int64_t rows, const int32_t* offsets, const void* W_packed,
                    const fmpq_epilogue* e, const float* row_weight, void* Y, int32_t dtype, int64_t ldy, void* workspace,
                    size_t workspace_bytes, void* stream) {
    if (fmpq_status s = product_ok(L, X, ldx, rows, W_packed, e, row_weight, Y, dtype, ldy)) return s;
    if (!element_aligned(offsets, FMPQ_DTYPE_F32)) return FMPQ_ERR_MISALIGNED;
    const size_t need = w16_workspace_bytes(L, X, ldx, rows);
    if (fmpq_status s = workspace_ok(need, workspace, workspace_bytes)) return s;
    if (fmpq_status s = check_device(L)) return s;
    fmpq::W16Args a = args_of(L, X, ldx, rows, W_packed, e, row_weight, Y, dtype, ldy);
    a.start = offsets;
    if (need > 0) {
        a.X = workspace;
        a.ldx = aligned_ld(L);
        const cudaError_t c = fmpq::launch_w16_rows(X, ldx, rows, L->K, nullptr, 1, workspace, a.ldx, L->num_sms, st(stream));
        if (c != cudaSuccess) return launched(c);
    }
    return launched(fmpq::launch_w16_gemm(*L, a, st(stream)));
}

}  // namespace

extern "C" {

fmpq_status w16_layer_create(int32_t K, int32_t N, int32_t experts, int32_t gated, int32_t dtype, w16_layer** out) {
    if (out == nullptr) return FMPQ_ERR_INVALID_ARG;
    *out = nullptr;
    if ((gated != 0 && gated != 1) || !sixteen_bits(dtype)) return FMPQ_ERR_INVALID_ARG;
    if (K < 1 || K > W16_MAX_K || N < 1 || N > W16_MAX_N || experts < 1 || experts > fmpq::kMaxFp8Experts || (gated && N % 2 != 0))
        return FMPQ_ERR_UNSUPPORTED_SHAPE;
    int dev = -1, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10 || minor != 3)
        return FMPQ_ERR_DEVICE;   // built for sm_103a only
    w16_layer* L = new (std::nothrow) w16_layer();
    if (L == nullptr) return FMPQ_ERR_INVALID_ARG;
    L->K = K;
    L->N = N;
    L->experts = experts;
    L->gated = gated;
    L->dtype = dtype;
    L->nb = (K + fmpq::kW16Block - 1) / fmpq::kW16Block;
    L->pairs = gated ? (N / 2 + 127) / 128 : (N + 255) / 256;
    L->device = dev;
    L->num_sms = sms;
    if (cudaMalloc(&L->d_status, sizeof(int32_t)) != cudaSuccess || cudaMemset(L->d_status, 0, sizeof(int32_t)) != cudaSuccess) {
        w16_layer_destroy(L);
        return FMPQ_ERR_CUDA;
    }
    *out = L;
    return FMPQ_OK;
}

void w16_layer_destroy(w16_layer* L) {
    if (L == nullptr) return;
    int prev = -1;
    const bool switched = cudaGetDevice(&prev) == cudaSuccess && prev != L->device && L->device >= 0 &&
                          cudaSetDevice(L->device) == cudaSuccess;
    cudaDeviceSynchronize();
    cudaFree(L->d_status);
    if (switched) cudaSetDevice(prev);
    delete L;
}

fmpq_status w16_device_status(const w16_layer* L, int32_t* status_host, int32_t clear) {
    if (L == nullptr || status_host == nullptr) return FMPQ_ERR_INVALID_ARG;
    if (fmpq_status s = check_device(L)) return s;
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(status_host, L->d_status, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
        return FMPQ_ERR_CUDA;
    if (clear && cudaMemset(L->d_status, 0, sizeof(int32_t)) != cudaSuccess) return FMPQ_ERR_CUDA;
    return FMPQ_OK;
}

size_t w16_packed_w_bytes(const w16_layer* L) {
    return L ? static_cast<size_t>(L->experts) * L->pairs * 2 * L->nb * fmpq::kTileBytes : 0;
}

fmpq_status w16_pack_weights(const w16_layer* L, int32_t expert, const void* W, int64_t ld_n, int64_t ld_k, void* W_packed,
                             void* stream) {
    if (L == nullptr || W == nullptr || W_packed == nullptr || expert < 0 || expert >= L->experts) return FMPQ_ERR_INVALID_ARG;
    if (ld_n < 1 || ld_k < 1) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(W_packed) || !element_aligned(W, L->dtype)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    return launched(fmpq::launch_w16_pack(*L, expert, W, ld_n, ld_k, W_packed, st(stream)));
}

size_t w16_workspace_bytes(const w16_layer* L, const void* X, int64_t ldx, int64_t rows) {
    if (L == nullptr || rows < 1 || rows > kMaxRows || rows_aligned(X, ldx, rows)) return 0;
    return static_cast<size_t>(rows) * static_cast<size_t>(aligned_ld(L)) * 2;
}

fmpq_status w16_gemm(const w16_layer* L, const void* X, int64_t ldx, int64_t M, const void* W_packed, const fmpq_epilogue* epilogue,
                     void* Y, int32_t dtype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    if (L != nullptr && L->experts != 1) return FMPQ_ERR_INVALID_ARG;
    return product(L, X, ldx, M, nullptr, W_packed, epilogue, nullptr, Y, dtype, ldy, workspace, workspace_bytes, stream);
}

fmpq_status w16_gemm_fault_test(const w16_layer* L, const void* X, int64_t ldx, int64_t M, const void* W_packed, void* Y, int64_t ldy,
                                int32_t withhold_cta, int32_t withhold_copy, uint32_t poll_limit, void* stream) {
    if (L == nullptr || L->experts != 1 || L->gated) return FMPQ_ERR_INVALID_ARG;
    if (fmpq_status s = product_ok(L, X, ldx, M, W_packed, nullptr, nullptr, Y, L->dtype, ldy)) return s;
    if (withhold_cta < 0 || withhold_copy < 0 || poll_limit < 1024) return FMPQ_ERR_INVALID_ARG;
    if (!rows_aligned(X, ldx, M)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    fmpq::W16Args a = args_of(L, X, ldx, M, W_packed, nullptr, nullptr, Y, L->dtype, ldy);
    a.polls = poll_limit;
    a.withheld_cta = withhold_cta;
    a.withheld_copy = withhold_copy;
    return launched(fmpq::launch_w16_gemm(*L, a, st(stream)));
}

fmpq_status w16_grouped_gemm(const w16_layer* L, const void* X, int64_t ldx, int64_t rows, const int32_t* offsets, const void* W_packed,
                             const fmpq_epilogue* epilogue, const float* row_weight, void* Y, int32_t dtype, int64_t ldy,
                             void* workspace, size_t workspace_bytes, void* stream) {
    if (offsets == nullptr) return FMPQ_ERR_INVALID_ARG;
    return product(L, X, ldx, rows, offsets, W_packed, epilogue, row_weight, Y, dtype, ldy, workspace, workspace_bytes, stream);
}

size_t w16_experts_workspace_bytes(const w16_layer* L, const void* X, int64_t ldx, int64_t T, int32_t k, int32_t gather) {
    if (L == nullptr || moe_rows(T, k, L->experts) == 0) return 0;
    const int64_t rows = moe_rows(T, k, L->experts);
    if (!gather && rows_aligned(X, ldx, rows)) return 0;
    return static_cast<size_t>(rows) * static_cast<size_t>(aligned_ld(L)) * 2;
}

fmpq_status w16_experts_gemm(const w16_layer* L, const void* plan, int64_t T, int32_t k, const void* X, int64_t ldx, int32_t gather,
                             const void* W_packed, const fmpq_epilogue* epilogue, const float* weights, void* Y, int32_t dtype,
                             int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    if (L == nullptr || plan == nullptr || (gather != 0 && gather != 1)) return FMPQ_ERR_INVALID_ARG;
    const int64_t rows = moe_rows(T, k, L->experts);
    if (fmpq_status s = product_ok(L, X, ldx, rows, W_packed, epilogue, weights, Y, dtype, ldy)) return s;   // (no rows: sizes outside the plan's)
    if (!aligned16(plan)) return FMPQ_ERR_MISALIGNED;
    const size_t need = w16_experts_workspace_bytes(L, X, ldx, T, k, gather);
    if (fmpq_status s = workspace_ok(need, workspace, workspace_bytes)) return s;
    if (fmpq_status s = check_device(L)) return s;
    const fmpq::MoePlan parts = fmpq::moe_plan_parts(plan, T, k, L->experts);
    fmpq::W16Args a = args_of(L, X, ldx, rows, W_packed, epilogue, weights, Y, dtype, ldy);
    a.start = parts.start;
    a.count = parts.count;
    a.pair_of = parts.pair_of;
    if (need > 0) {
        a.X = workspace;
        a.ldx = aligned_ld(L);
        const cudaError_t c = fmpq::launch_w16_rows(X, ldx, gather ? T : rows, L->K, gather ? parts.row_of : nullptr, k, workspace, a.ldx,
                                                    L->num_sms, st(stream));
        if (c != cudaSuccess) return launched(c);
    }
    return launched(fmpq::launch_w16_gemm(*L, a, st(stream)));
}

}  // extern "C"
