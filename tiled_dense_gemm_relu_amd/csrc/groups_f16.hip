// The kernel instances of gemm_relu_groups.h for the f16 dtype.
#include "groups_instances.hpp"

namespace gemm_relu_hip {
const GroupKernels& group_kernels_f16()
{
    static const GroupKernels t = make_group_table<kF16>();
    return t;
}
}  // namespace gemm_relu_hip
