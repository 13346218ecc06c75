// C ABI of the E4M3 linear layers and the routed experts (declared in include/fmpq.h): argument
// validation, layer handles, and kernel launches on the caller's stream.
#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/fmpq.h"
#include "fp8_internal.h"

namespace {

constexpr int64_t kMaxRows = INT64_C(1) << 24;
constexpr int kMaxPlanExperts = 1024;
constexpr int64_t kMaxPairs = INT64_C(1) << 22;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P>
bool all_aligned16(const P*... p) { return (aligned16(p) && ...); }

fmpq_status launched(cudaError_t e) { return e == cudaSuccess ? FMPQ_OK : FMPQ_ERR_CUDA; }

fmpq_status check_device(const fp8_layer* L) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return FMPQ_ERR_CUDA;
    return dev == L->device ? FMPQ_OK : FMPQ_ERR_DEVICE;
}
bool sixteen_bits(int32_t dtype) { return dtype == FMPQ_DTYPE_F16 || dtype == FMPQ_DTYPE_BF16; }
bool any_type(int32_t dtype) { return sixteen_bits(dtype) || dtype == FMPQ_DTYPE_F32; }
bool element_aligned(const void* p, int32_t dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == FMPQ_DTYPE_F32 ? 3u : 1u)) == 0;
}
cudaStream_t st(void* stream) { return static_cast<cudaStream_t>(stream); }

// T tokens of k slots over E experts: what the plan and the experts' calls take.
bool routing_ok(int64_t T, int32_t k, int32_t E) {
    return T >= 1 && k >= 1 && k <= 32 && E >= 1 && E <= kMaxPlanExperts && T <= kMaxPairs && T * k <= kMaxPairs;
}

}  // namespace

extern "C" {

fmpq_status fp8_layer_create(int32_t K, int32_t N, int32_t experts, int32_t gated, fp8_layer** out) {
    if (out == nullptr) return FMPQ_ERR_INVALID_ARG;
    *out = nullptr;
    if (gated != 0 && gated != 1) return FMPQ_ERR_INVALID_ARG;
    if (K < 1 || K > FP8_MAX_K || N < 1 || N > FP8_MAX_N || experts < 1 || experts > fmpq::kMaxFp8Experts || (gated && N % 2 != 0))
        return FMPQ_ERR_UNSUPPORTED_SHAPE;
    int dev = -1, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10 || minor != 3)
        return FMPQ_ERR_DEVICE;   // built for sm_103a only
    fp8_layer* L = new (std::nothrow) fp8_layer();
    if (L == nullptr) return FMPQ_ERR_INVALID_ARG;
    L->K = K;
    L->N = N;
    L->experts = experts;
    L->gated = gated;
    L->nb = (K + 127) / 128;
    const int32_t half = (N / 2 + 127) / 128;
    L->pairs = gated ? half : (N + 255) / 256;
    L->scale_rows = gated ? 2 * half : (N + 127) / 128;
    L->device = dev;
    L->num_sms = sms;
    if (cudaMalloc(&L->d_status, sizeof(int32_t)) != cudaSuccess ||
        cudaMemset(L->d_status, 0, sizeof(int32_t)) != cudaSuccess) {
        fp8_layer_destroy(L);
        return FMPQ_ERR_CUDA;
    }
    *out = L;
    return FMPQ_OK;
}

void fp8_layer_destroy(fp8_layer* L) {
    if (L == nullptr) return;
    int prev = -1;
    const bool switched = cudaGetDevice(&prev) == cudaSuccess && prev != L->device && L->device >= 0 &&
                          cudaSetDevice(L->device) == cudaSuccess;
    cudaDeviceSynchronize();
    cudaFree(L->d_status);
    if (switched) cudaSetDevice(prev);
    delete L;
}

fmpq_status fp8_device_status(const fp8_layer* L, int32_t* status_host, int32_t clear) {
    if (L == nullptr || status_host == nullptr) return FMPQ_ERR_INVALID_ARG;
    if (fmpq_status s = check_device(L)) return s;
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(status_host, L->d_status, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
        return FMPQ_ERR_CUDA;
    if (clear && cudaMemset(L->d_status, 0, sizeof(int32_t)) != cudaSuccess) return FMPQ_ERR_CUDA;
    return FMPQ_OK;
}

size_t fp8_packed_w_bytes(const fp8_layer* L) {
    return L ? static_cast<size_t>(L->experts) * L->pairs * 2 * L->nb * fmpq::kTileBytes : 0;
}
size_t fp8_weight_scale_count(const fp8_layer* L) {
    return L ? static_cast<size_t>(L->experts) * L->scale_rows * L->nb : 0;
}
size_t fp8_packed_a_bytes(const fp8_layer* L, int64_t rows) {
    return L && rows > 0 ? static_cast<size_t>(L->nb) * static_cast<size_t>(rows) * 128 : 0;
}
size_t fp8_a_scale_count(const fp8_layer* L, int64_t rows) {
    return L && rows > 0 ? static_cast<size_t>(L->nb) * static_cast<size_t>(fmpq::scale_stride(rows)) : 0;
}

fmpq_status fp8_pack_weights(const fp8_layer* L, int32_t expert, const void* W, int32_t dtype, int64_t ldw, void* W_packed,
                             void* w_scales, void* stream) {
    if (L == nullptr || W == nullptr || W_packed == nullptr || w_scales == nullptr || expert < 0 || expert >= L->experts ||
        !sixteen_bits(dtype))
        return FMPQ_ERR_INVALID_ARG;
    if (ldw < L->K) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(W_packed, w_scales) || !element_aligned(W, dtype)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    return launched(fmpq::launch_fp8_pack_weights(*L, expert, W, dtype, ldw, W_packed, static_cast<float*>(w_scales),
                                                  st(stream)));
}

fmpq_status fp8_pack_codes(const fp8_layer* L, int32_t expert, const void* codes, int64_t ldw, void* W_packed,
                           void* stream) {
    if (L == nullptr || codes == nullptr || W_packed == nullptr || expert < 0 || expert >= L->experts)
        return FMPQ_ERR_INVALID_ARG;
    if (ldw < L->K) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(W_packed)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    return launched(fmpq::launch_fp8_pack_codes(*L, expert, codes, ldw, W_packed, st(stream)));
}

fmpq_status fp8_unpack_weights(const fp8_layer* L, int32_t expert, const void* W_packed, const void* w_scales, void* W,
                               void* stream) {
    if (L == nullptr || W_packed == nullptr || w_scales == nullptr || W == nullptr || expert < 0 || expert >= L->experts)
        return FMPQ_ERR_INVALID_ARG;
    if (!all_aligned16(W_packed, w_scales, W)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    return launched(fmpq::launch_fp8_unpack(*L, expert, W_packed, static_cast<const float*>(w_scales),
                                            static_cast<float*>(W), st(stream)));
}

fmpq_status fp8_quantize(const fp8_layer* L, const void* X, int32_t dtype, int64_t ldx, int64_t M, void* A_packed,
                         void* a_scales, void* stream) {
    if (L == nullptr || X == nullptr || A_packed == nullptr || a_scales == nullptr || !sixteen_bits(dtype))
        return FMPQ_ERR_INVALID_ARG;
    if (M < 1 || M > kMaxRows || ldx < L->K) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(A_packed, a_scales) || !element_aligned(X, dtype)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    return launched(fmpq::launch_fp8_quantize(X, dtype, ldx, M, L->K, nullptr, 1, M, A_packed,
                                              static_cast<float*>(a_scales), L->num_sms, false, st(stream)));
}

size_t fp8_gemm_workspace_bytes(const fp8_layer* L, int64_t M) {
    return L && M > 0 ? fmpq::fp8_gemm_workspace(*L, M) : 0;
}

static fmpq_status gemm_after(const fp8_layer* L, const void* A_packed, const void* a_scales, const void* W_packed,
                              const void* w_scales, int64_t M, void* Y, int32_t dtype, int64_t ldy, void* workspace,
                              size_t workspace_bytes, bool pdl, void* stream);

fmpq_status fp8_gemm(const fp8_layer* L, const void* A_packed, const void* a_scales, const void* W_packed,
                     const void* w_scales, int64_t M, void* Y, int32_t dtype, int64_t ldy, void* workspace,
                     size_t workspace_bytes, void* stream) {
    return gemm_after(L, A_packed, a_scales, W_packed, w_scales, M, Y, dtype, ldy, workspace, workspace_bytes, false, stream);
}

static fmpq_status gemm_after(const fp8_layer* L, const void* A_packed, const void* a_scales, const void* W_packed,
                              const void* w_scales, int64_t M, void* Y, int32_t dtype, int64_t ldy, void* workspace,
                              size_t workspace_bytes, bool pdl, void* stream) {
    if (L == nullptr || A_packed == nullptr || a_scales == nullptr || W_packed == nullptr || w_scales == nullptr ||
        Y == nullptr || !sixteen_bits(dtype) || L->gated || L->experts != 1)
        return FMPQ_ERR_INVALID_ARG;
    if (M < 1 || M > kMaxRows || ldy < L->N) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(A_packed, a_scales, W_packed, w_scales) || !element_aligned(Y, dtype)) return FMPQ_ERR_MISALIGNED;
    const size_t need = fmpq::fp8_gemm_workspace(*L, M);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FMPQ_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    fmpq::Fp8GemmArgs a{};
    a.A = A_packed;
    a.a_scales = static_cast<const float*>(a_scales);
    a.W = W_packed;
    a.w_scales = static_cast<const float*>(w_scales);
    a.rows = M;
    a.pairs_routed = M;
    a.Y = Y;
    a.dtype = dtype;
    a.ldy = ldy;
    a.workspace = need > 0 ? workspace : nullptr;
    a.pdl = pdl;
    return launched(fmpq::launch_fp8_gemm(*L, a, st(stream)));
}

fmpq_status fp8_quantize_gemm(const fp8_layer* L, const void* X, int32_t dtype, int64_t ldx, int64_t M, void* A_packed,
                              void* a_scales, const void* W_packed, const void* w_scales, void* Y, int64_t ldy,
                              void* workspace, size_t workspace_bytes, void* stream) {
    // both calls' checks first, so that a refusal launches nothing
    if (L == nullptr || X == nullptr || A_packed == nullptr || a_scales == nullptr || W_packed == nullptr ||
        w_scales == nullptr || Y == nullptr || !sixteen_bits(dtype) || L->gated || L->experts != 1)
        return FMPQ_ERR_INVALID_ARG;
    if (M < 1 || M > kMaxRows || ldx < L->K || ldy < L->N) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(A_packed, a_scales, W_packed, w_scales) || !element_aligned(X, dtype) || !element_aligned(Y, dtype))
        return FMPQ_ERR_MISALIGNED;
    const size_t need = fmpq::fp8_gemm_workspace(*L, M);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FMPQ_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = fp8_quantize(L, X, dtype, ldx, M, A_packed, a_scales, stream)) return s;
    return gemm_after(L, A_packed, a_scales, W_packed, w_scales, M, Y, dtype, ldy, workspace, workspace_bytes, true, stream);
}

// ---------------------------------------------------------------- routing and experts

fmpq_status moe_route(const void* logits, int32_t dtype, int64_t ldl, int64_t T, int32_t E, int32_t k, int32_t score,
                      const void* bias, int32_t groups, int32_t top_groups, int32_t group_top, int32_t renormalize,
                      float scale, void* ids, void* weights, void* stream) {
    if (logits == nullptr || ids == nullptr || weights == nullptr || !any_type(dtype) ||
        (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || (group_top != 1 && group_top != 2) ||
        (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
        return FMPQ_ERR_INVALID_ARG;
    if (T < 1 || T > kMaxRows || E < 1 || E > fmpq::kMaxFp8Experts || k < 1 || k > 32 || k > E || ldl < E || groups < 1 ||
        groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups || k > top_groups * (E / groups))
        return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!element_aligned(logits, dtype) || !element_aligned(bias, FMPQ_DTYPE_F32) ||
        !element_aligned(ids, FMPQ_DTYPE_F32) || !element_aligned(weights, FMPQ_DTYPE_F32))
        return FMPQ_ERR_MISALIGNED;
    fmpq::RouteArgs a{};
    a.logits = logits;
    a.dtype = dtype;
    a.ldl = ldl;
    a.T = T;
    a.E = E;
    a.k = k;
    a.sigmoid = score == MOE_SCORE_SIGMOID;
    a.groups = groups;
    a.top_groups = top_groups;
    a.group_top = group_top;
    a.renormalize = renormalize;
    a.scale = scale;
    a.bias = static_cast<const float*>(bias);
    a.ids = static_cast<int32_t*>(ids);
    a.weights = static_cast<float*>(weights);
    return launched(fmpq::launch_moe_route(a, st(stream)));
}

int64_t moe_rows(int64_t T, int32_t k, int32_t E) { return routing_ok(T, k, E) ? fmpq::moe_rows_of(T, k, E) : 0; }

size_t moe_plan_bytes(int64_t T, int32_t k, int32_t E) {
    if (!routing_ok(T, k, E)) return 0;
    const size_t P = static_cast<size_t>(T) * k;
    // the parts of MoePlan, then the counts of each chunk of 1024 pairs
    return (2 * static_cast<size_t>(E) + P + static_cast<size_t>(fmpq::moe_rows_of(T, k, E)) +
            (P + 1023) / 1024 * static_cast<size_t>(E)) * sizeof(int32_t);
}

fmpq_status moe_plan(const void* ids, int64_t T, int32_t k, int32_t E, void* plan, void* stream) {
    if (ids == nullptr || plan == nullptr) return FMPQ_ERR_INVALID_ARG;
    if (!routing_ok(T, k, E)) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(plan) || !element_aligned(ids, FMPQ_DTYPE_F32)) return FMPQ_ERR_MISALIGNED;
    int32_t* p = static_cast<int32_t*>(plan);
    return launched(fmpq::launch_moe_plan(static_cast<const int32_t*>(ids), T, k, E, p,
                                          p + 2 * E + T * k + fmpq::moe_rows_of(T, k, E), st(stream)));
}

static fmpq_status quantize_after(const fp8_layer* L, const void* plan, int64_t T, int32_t k, const void* X, int32_t dtype,
                         int64_t ldx, void* A_packed, void* a_scales, bool pdl, void* stream) {
    if (L == nullptr || plan == nullptr || X == nullptr || A_packed == nullptr || a_scales == nullptr || !sixteen_bits(dtype))
        return FMPQ_ERR_INVALID_ARG;
    if (!routing_ok(T, k, L->experts) || ldx < L->K) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(plan, A_packed, a_scales) || !element_aligned(X, dtype)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    const fmpq::MoePlan p = fmpq::moe_plan_parts(plan, T, k, L->experts);
    return launched(fmpq::launch_fp8_quantize(X, dtype, ldx, T, L->K, p.row_of, k, fmpq::moe_rows_of(T, k, L->experts),
                                              A_packed, static_cast<float*>(a_scales), L->num_sms, pdl, st(stream)));
}
fmpq_status moe_quantize(const fp8_layer* L, const void* plan, int64_t T, int32_t k, const void* X, int32_t dtype,
                         int64_t ldx, void* A_packed, void* a_scales, void* stream) {
    return quantize_after(L, plan, T, k, X, dtype, ldx, A_packed, a_scales, false, stream);
}

static fmpq_status up_after(const fp8_layer* L, const void* plan, int64_t T, int32_t k, const void* A_packed, const void* a_scales,
                   const void* W_packed, const void* w_scales, void* H_packed, void* h_scales, bool pdl, void* stream) {
    if (L == nullptr || plan == nullptr || A_packed == nullptr || a_scales == nullptr || W_packed == nullptr ||
        w_scales == nullptr || H_packed == nullptr || h_scales == nullptr || !L->gated)
        return FMPQ_ERR_INVALID_ARG;
    if (!routing_ok(T, k, L->experts)) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(plan, A_packed, a_scales, W_packed, w_scales, H_packed, h_scales)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    const fmpq::MoePlan p = fmpq::moe_plan_parts(plan, T, k, L->experts);
    fmpq::Fp8GemmArgs a{};
    a.A = A_packed;
    a.a_scales = static_cast<const float*>(a_scales);
    a.W = W_packed;
    a.w_scales = static_cast<const float*>(w_scales);
    a.rows = fmpq::moe_rows_of(T, k, L->experts);
    a.start = p.start;
    a.count = p.count;
    a.pair_of = p.pair_of;
    a.pairs_routed = T * k;
    a.H = H_packed;
    a.h_scales = static_cast<float*>(h_scales);
    a.pdl = pdl;
    return launched(fmpq::launch_fp8_gemm(*L, a, st(stream)));
}
fmpq_status moe_up(const fp8_layer* L, const void* plan, int64_t T, int32_t k, const void* A_packed, const void* a_scales,
                   const void* W_packed, const void* w_scales, void* H_packed, void* h_scales, void* stream) {
    return up_after(L, plan, T, k, A_packed, a_scales, W_packed, w_scales, H_packed, h_scales, false, stream);
}

static fmpq_status down_after(const fp8_layer* L, const void* plan, int64_t T, int32_t k, const void* weights, const void* A_packed,
                     const void* a_scales, const void* W_packed, const void* w_scales, void* D, int32_t dtype, int64_t ldd,
                     bool pdl, void* stream) {
    if (L == nullptr || plan == nullptr || A_packed == nullptr || a_scales == nullptr || W_packed == nullptr ||
        w_scales == nullptr || D == nullptr || !any_type(dtype) || L->gated)
        return FMPQ_ERR_INVALID_ARG;
    if (!routing_ok(T, k, L->experts) || ldd < L->N) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(plan, A_packed, a_scales, W_packed, w_scales) || !element_aligned(weights, FMPQ_DTYPE_F32) ||
        !element_aligned(D, dtype))
        return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(L)) return s;
    const fmpq::MoePlan p = fmpq::moe_plan_parts(plan, T, k, L->experts);
    fmpq::Fp8GemmArgs a{};
    a.A = A_packed;
    a.a_scales = static_cast<const float*>(a_scales);
    a.W = W_packed;
    a.w_scales = static_cast<const float*>(w_scales);
    a.rows = fmpq::moe_rows_of(T, k, L->experts);
    a.start = p.start;
    a.count = p.count;
    a.pair_of = p.pair_of;
    a.pair_weight = static_cast<const float*>(weights);
    a.pairs_routed = T * k;
    a.Y = D;
    a.dtype = dtype;
    a.ldy = ldd;
    a.pdl = pdl;
    return launched(fmpq::launch_fp8_gemm(*L, a, st(stream)));
}
fmpq_status moe_down(const fp8_layer* L, const void* plan, int64_t T, int32_t k, const void* weights, const void* A_packed,
                     const void* a_scales, const void* W_packed, const void* w_scales, void* D, int32_t dtype, int64_t ldd,
                     void* stream) {
    return down_after(L, plan, T, k, weights, A_packed, a_scales, W_packed, w_scales, D, dtype, ldd, false, stream);
}

static fmpq_status combine_after(const void* D, int32_t d_dtype, int64_t ldd, const void* plan, int64_t T, int32_t k, int32_t E,
                        int32_t N, void* Y, int32_t dtype, int64_t ldy, bool pdl, void* stream) {
    if (D == nullptr || plan == nullptr || Y == nullptr || !sixteen_bits(dtype)) return FMPQ_ERR_INVALID_ARG;
    if (!routing_ok(T, k, E) || N < 1 || N > FP8_MAX_N || ldd < N || ldy < N) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(plan) || !element_aligned(D, d_dtype) || !element_aligned(Y, dtype)) return FMPQ_ERR_MISALIGNED;
    const fmpq::MoePlan p = fmpq::moe_plan_parts(plan, T, k, E);
    return launched(fmpq::launch_moe_combine(D, d_dtype, ldd, p.row_of, T, k, N, Y, dtype, ldy, pdl, st(stream)));
}
fmpq_status moe_combine(const void* D, int32_t dtype, int64_t ldd, const void* plan, int64_t T, int32_t k, int32_t E,
                        int32_t N, void* Y, int64_t ldy, void* stream) {
    return combine_after(D, dtype, ldd, plan, T, k, E, N, Y, dtype, ldy, false, stream);
}
fmpq_status moe_combine_f32(const float* D, int64_t ldd, const void* plan, int64_t T, int32_t k, int32_t E, int32_t N, void* Y,
                            int32_t dtype, int64_t ldy, void* stream) {
    return combine_after(D, FMPQ_DTYPE_F32, ldd, plan, T, k, E, N, Y, dtype, ldy, false, stream);
}

namespace {

// The parts of moe_experts' scratch buffer: byte offsets.
struct Scratch {
    size_t plan, codes, scales, h_codes, h_scales, d, end;
};
bool experts_ok(const fp8_layer* up, const fp8_layer* down) {
    return up != nullptr && down != nullptr && up->gated && !down->gated && up->experts == down->experts &&
           up->N == 2 * down->K && up->device == down->device;
}
Scratch scratch_parts(const fp8_layer* up, const fp8_layer* down, int64_t T, int32_t k) {
    const int64_t rows = fmpq::moe_rows_of(T, k, up->experts);
    auto after = [](size_t at, size_t bytes) { return (at + bytes + 255) & ~size_t(255); };
    Scratch s{};
    s.plan = 0;
    s.codes = after(s.plan, moe_plan_bytes(T, k, up->experts));
    s.scales = after(s.codes, fp8_packed_a_bytes(up, rows));
    s.h_codes = after(s.scales, fp8_a_scale_count(up, rows) * sizeof(float));
    s.h_scales = after(s.h_codes, fp8_packed_a_bytes(down, rows));
    s.d = after(s.h_scales, fp8_a_scale_count(down, rows) * sizeof(float));
    s.end = after(s.d, static_cast<size_t>(rows) * ((down->N + 7) / 8 * 8) * sizeof(float));
    return s;
}

}  // namespace

size_t moe_experts_bytes(const fp8_layer* up, const fp8_layer* down, int64_t T, int32_t k) {
    return experts_ok(up, down) && routing_ok(T, k, up->experts) ? scratch_parts(up, down, T, k).end : 0;
}

fmpq_status moe_experts(const fp8_layer* up, const fp8_layer* down, const void* X, int32_t dtype, int64_t ldx, int64_t T,
                        int32_t k, const void* ids, const void* weights, const void* W_up, const void* s_up,
                        const void* W_down, const void* s_down, void* Y, int64_t ldy, void* scratch, size_t scratch_bytes,
                        void* stream) {
    // every step's checks first, so that a refusal launches nothing
    if (!experts_ok(up, down) || X == nullptr || ids == nullptr || weights == nullptr || W_up == nullptr ||
        s_up == nullptr || W_down == nullptr || s_down == nullptr || Y == nullptr || !sixteen_bits(dtype))
        return FMPQ_ERR_INVALID_ARG;
    if (!routing_ok(T, k, up->experts) || ldx < up->K || ldy < down->N) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!all_aligned16(W_up, s_up, W_down, s_down) || !element_aligned(X, dtype) || !element_aligned(Y, dtype) ||
        !element_aligned(ids, FMPQ_DTYPE_F32) || !element_aligned(weights, FMPQ_DTYPE_F32))
        return FMPQ_ERR_MISALIGNED;
    const Scratch at = scratch_parts(up, down, T, k);
    if (scratch == nullptr || scratch_bytes < at.end) return FMPQ_ERR_WORKSPACE;
    if (!aligned16(scratch)) return FMPQ_ERR_MISALIGNED;
    if (fmpq_status s = check_device(up)) return s;
    uint8_t* b = static_cast<uint8_t*>(scratch);
    // The experts' products stay in FP32 until a token's slots are summed, so that the output is rounded once: rounded
    // one by one the error grows from 1.7e-3 to 2.4e-3 of the norm (bf16, 8 slots), and in fp16 a slot may overflow
    // where the sum does not. It costs 4 bytes an output, written and read, in place of 2.
    const int64_t ldd = (down->N + 7) / 8 * 8;   // 16-byte rows, whatever N is
    if (fmpq_status s = moe_plan(ids, T, k, up->experts, b + at.plan, stream)) return s;
    if (fmpq_status s = quantize_after(up, b + at.plan, T, k, X, dtype, ldx, b + at.codes, b + at.scales, true, stream)) return s;
    if (fmpq_status s = up_after(up, b + at.plan, T, k, b + at.codes, b + at.scales, W_up, s_up, b + at.h_codes,
                               b + at.h_scales, true, stream))
        return s;
    if (fmpq_status s = down_after(down, b + at.plan, T, k, weights, b + at.h_codes, b + at.h_scales, W_down, s_down, b + at.d,
                                 FMPQ_DTYPE_F32, ldd, true, stream))
        return s;
    return combine_after(b + at.d, FMPQ_DTYPE_F32, ldd, b + at.plan, T, k, up->experts, down->N, Y, dtype, ldy, true, stream);
}

}  // extern "C"
