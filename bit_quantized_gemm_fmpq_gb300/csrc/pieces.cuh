// Eight 16-bit elements at any alignment, from the aligned pieces of 16 bytes that hold them.
#pragma once

#include <cstdint>

namespace fmpq {
namespace {

// Eight elements that begin `off` (1 to 7) elements behind a 16-byte boundary, from the two pieces of 16 bytes that hold them.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, uint32_t off) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = (off & 4) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = (off & 2) ? w[i + 1] : w[i];
    const uint32_t by = (off & 1) * 16;
    return make_uint4(__funnelshift_r(w[0], w[1], by), __funnelshift_r(w[1], w[2], by), __funnelshift_r(w[2], w[3], by),
                      __funnelshift_r(w[3], w[4], by));
}
// Of an address: the boundary before it, and the elements between.
__device__ __forceinline__ uint32_t elements_past(const void* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1; }
// The eight elements k .. k + 7 of a row that has them all. The pieces read hold one of them at least, so they lie in its allocation.
template <typename T>
__device__ __forceinline__ uint4 eight_at(const T* row, int64_t k) {
    const uint32_t off = elements_past(row + k);
    const uint4* at = reinterpret_cast<const uint4*>(row + k - off);
    return off == 0 ? at[0] : shifted(at[0], at[1], off);
}

}  // namespace
}  // namespace fmpq
