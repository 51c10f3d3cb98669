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

// dma_b128 of what is read once: it does not stay in the caches.
__device__ __forceinline__ void dma_b128_once(int32x4_t rsrc, uint32_t lds_addr, uint32_t voffset, uint32_t soffset)
{
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                 :
                 : "s"(lds_addr), "v"(voffset), "s"(rsrc), "s"(soffset)
                 : "memory", "m0");
}

}  // namespace gemm_relu_hip
