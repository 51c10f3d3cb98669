// 8-bit pieces in registers.
#pragma once

#include "groups_kernels.hpp"

namespace gemm_relu_hip {

// The first `valid` of 16 bytes, zeros after them.
__device__ __forceinline__ u32x4 keep_bytes(u32x4 v, int valid)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int left = valid - 4 * i;
        v[i] = left >= 4 ? v[i] : left > 0 ? v[i] & (0xffffffffu >> (32 - 8 * left)) : 0u;
    }
    return v;
}

}  // namespace gemm_relu_hip
