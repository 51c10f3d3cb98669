// The register-staged kernel instances of gemm_relu_groups.h for the bf16 dtype, rows of any length.
#include "groups_instances.hpp"

namespace gemm_relu_hip {
const StagedKernels& staged_kernels_bf16_odd()
{
    static const StagedKernels t = make_staged_table<kBF16, true>();
    return t;
}
}  // namespace gemm_relu_hip
