// The kernel instances of gemm_relu_groups.h for the bf16 dtype.
#include "groups_instances.hpp"

namespace gemm_relu_hip {
const GroupKernels& group_kernels_bf16()
{
    static const GroupKernels t = make_group_table<kBF16>();
    return t;
}
}  // namespace gemm_relu_hip
