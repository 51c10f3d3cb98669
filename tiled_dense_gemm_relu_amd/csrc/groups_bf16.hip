// The kernel instances of gemm_relu_groups.h for one dtype.
#include "groups_kernels.hpp"

namespace gemm_relu_hip {
const GroupKernels& group_kernels_bf16()
{
    static const GroupKernels t = make_group_table<kBF16>();
    return t;
}
}  // namespace gemm_relu_hip
