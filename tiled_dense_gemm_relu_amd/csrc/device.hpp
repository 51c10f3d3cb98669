// Host-side device check shared by the library's C entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/gemm_relu.h"

namespace gemm_relu_hip {

// Checks that the current device is a gfx950 and returns its CU count in *cus.
inline int check_device(int* cus)
{
    // Per-device cache: 0 unknown, > 0 gfx950 with that many CUs, -1 something else.
    static std::atomic<int> device_cus[64];
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GEMM_RELU_ERR_NO_DEVICE;
    if (dev < 64) {
        const int known = device_cus[dev].load(std::memory_order_relaxed);
        if (known != 0) {
            *cus = known;
            return known > 0 ? GEMM_RELU_OK : GEMM_RELU_ERR_NO_DEVICE;
        }
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMM_RELU_ERR_NO_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 && prop.multiProcessorCount > 0;
    const int value = ok ? prop.multiProcessorCount : -1;
    if (dev < 64) device_cus[dev].store(value, std::memory_order_relaxed);
    *cus = value;
    return ok ? GEMM_RELU_OK : GEMM_RELU_ERR_NO_DEVICE;
}

// Whether [a, a + a_bytes) and [b, b + b_bytes) share a byte.
inline bool overlaps(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes)
{
    if (a_bytes <= 0 || b_bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)b_bytes && b0 < a0 + (uintptr_t)a_bytes;
}

}  // namespace gemm_relu_hip
