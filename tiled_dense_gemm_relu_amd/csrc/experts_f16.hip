// The kernel instances of the expert layer for a few tokens, for the f16 dtype.
#include "experts_instances.hpp"

namespace gemm_relu_hip {
const ExpertsKernels& experts_kernels_f16()
{
    static const ExpertsKernels t = make_experts_table<kF16>();
    return t;
}
}  // namespace gemm_relu_hip
