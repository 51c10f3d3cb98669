// The register-staged kernel instances of gemm_relu_groups.h for the fp16 dtype, rows of an even length.
#include "groups_instances.hpp"

namespace gemm_relu_hip {
const StagedKernels& staged_kernels_f16_even()
{
    static const StagedKernels t = make_staged_table<kF16, false>();
    return t;
}
}  // namespace gemm_relu_hip
