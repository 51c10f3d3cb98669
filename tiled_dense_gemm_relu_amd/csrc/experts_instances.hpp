// The kernel instances of the expert layer for a few tokens, for one dtype.
#pragma once

#include "experts_kernels.hpp"

namespace gemm_relu_hip {

template <int DT, int STORE, bool ODD>
constexpr void fill_experts(const void* (&to)[2][kNumExpertBlocks])
{
    if constexpr (STORE != kStoreKN) {
        to[0][0] = (const void*)expert_products<DT, STORE, ODD, false, 1>;
        to[1][0] = (const void*)expert_products<DT, STORE, ODD, true, 1>;
    }
    to[0][1] = (const void*)expert_products<DT, STORE, ODD, false, 4>;
    to[1][1] = (const void*)expert_products<DT, STORE, ODD, true, 4>;
}

template <int DT>
ExpertsKernels make_experts_table()
{
    ExpertsKernels t{};
    fill_experts<DT, kStoreNK, false>(t.products[kStoreNK][0]);
    fill_experts<DT, kStoreNK, true>(t.products[kStoreNK][1]);
    fill_experts<DT, kStoreKN, false>(t.products[kStoreKN][0]);
    fill_experts<DT, kStoreKN, true>(t.products[kStoreKN][1]);
    fill_experts<DT, kStoreE4M3, false>(t.products[kStoreE4M3][0]);
    fill_experts<DT, kStoreE4M3, true>(t.products[kStoreE4M3][1]);
    fill_experts<DT, kStoreE5M2, false>(t.products[kStoreE5M2][0]);
    fill_experts<DT, kStoreE5M2, true>(t.products[kStoreE5M2][1]);
    return t;
}

}  // namespace gemm_relu_hip
