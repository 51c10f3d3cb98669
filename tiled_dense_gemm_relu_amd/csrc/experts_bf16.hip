// The kernel instances of the expert layer for a few tokens, for the bf16 dtype.
#include "experts_instances.hpp"

namespace gemm_relu_hip {
const ExpertsKernels& experts_kernels_bf16()
{
    static const ExpertsKernels t = make_experts_table<kBF16>();
    return t;
}
}  // namespace gemm_relu_hip
