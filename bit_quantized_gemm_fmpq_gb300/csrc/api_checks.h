// What the C entry points check, shared by the files that define them.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fmpq.h"
#include "epilogue.h"

namespace fmpq {
namespace api {

constexpr int64_t kMaxRows = INT64_C(1) << 24;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P>
bool all_aligned16(const P*... p) { return (aligned16(p) && ...); }

inline fmpq_status launched(cudaError_t e) { return e == cudaSuccess ? FMPQ_OK : FMPQ_ERR_CUDA; }

inline bool sixteen_bits(int32_t dtype) { return dtype == FMPQ_DTYPE_F16 || dtype == FMPQ_DTYPE_BF16; }
inline bool any_type(int32_t dtype) { return sixteen_bits(dtype) || dtype == FMPQ_DTYPE_F32; }
inline bool element_aligned(const void* p, int32_t dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == FMPQ_DTYPE_F32 ? 3u : 1u)) == 0;
}
inline cudaStream_t st(void* stream) { return static_cast<cudaStream_t>(stream); }


// A product's epilogue (NULL: none), for outputs of `dtype` and N columns.
inline fmpq_status epilogue_ok(const fmpq_epilogue* e, int32_t dtype, int64_t N) {
    if (e == nullptr) return FMPQ_OK;
    if (e->activation < FMPQ_ACT_NONE || e->activation > FMPQ_ACT_GELU_TANH ||
        (e->bias != nullptr && e->bias_dtype != FMPQ_DTYPE_F32 && e->bias_dtype != dtype))
        return FMPQ_ERR_INVALID_ARG;
    if (e->residual != nullptr && e->ldr < N) return FMPQ_ERR_UNSUPPORTED_SHAPE;
    if (!element_aligned(e->bias, e->bias_dtype) || !element_aligned(e->residual, dtype)) return FMPQ_ERR_MISALIGNED;
    return FMPQ_OK;
}
inline Epilogue epilogue_of(const fmpq_epilogue* e) {
    Epilogue r{};
    if (e == nullptr) return r;
    r.bias = e->bias;
    r.bias_f32 = e->bias_dtype == FMPQ_DTYPE_F32;
    r.residual = e->residual;
    r.ldr = e->residual != nullptr ? e->ldr : 0;
    r.act = e->activation;
    return r;
}

}  // namespace api
}  // namespace fmpq
