// A product's epilogue, as the launchers and kernels pass it: Y = act(sum + bias) + residual, rounded once.
#pragma once

#include <cstdint>

namespace fmpq {

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

struct Epilogue {
    const void* bias;      // [N] of FP32 or the outputs' type; nullptr: 0
    const void* residual;  // [M][ldr] of the outputs' type; nullptr: 0
    int64_t ldr;
    int bias_f32, act;
    bool any() const { return bias != nullptr || residual != nullptr || act != kActNone; }
};

}  // namespace fmpq
