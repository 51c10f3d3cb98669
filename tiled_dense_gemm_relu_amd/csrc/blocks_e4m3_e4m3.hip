// The kernel instances of gemm_relu_blocks for A in e4m3 and B in e4m3.
#include "blocks_instances.hpp"

namespace gemm_relu_hip {
const BlocksKernels& blocks_kernels_e4m3_e4m3()
{
    static const BlocksKernels t = make_blocks_table<kE4M3, kE4M3>();
    return t;
}
}  // namespace gemm_relu_hip
