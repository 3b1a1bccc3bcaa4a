// integers.cuh -- integer arithmetic of kernels.
#pragma once
#include <stdint.h>

namespace rmsnorm {

// a / b for a >= 0, b > 0; numbers of 32 bits, as most are, in a quarter of the instructions.
__device__ __forceinline__ int64_t div_nonneg(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

}  // namespace rmsnorm
