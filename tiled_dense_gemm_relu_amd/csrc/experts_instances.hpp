// The kernel instances of the expert layer for a few tokens, for one dtype.
#pragma once

#include "experts_kernels.hpp"

namespace gemm_relu_hip {

template <int DT, int STORE, bool ODD, int KIND = 0>
constexpr void fill_experts(const void* (&to)[2][kNumExpertKinds])
{
    to[0][KIND] = (const void*)expert_products<DT, STORE, ODD, false, KIND>;
    // (the second product of 8-bit weights has no odd rows)
    to[1][KIND] = (const void*)expert_products<DT, STORE, ODD && STORE < kStoreE4M3, true, KIND>;
    if constexpr (KIND + 1 < kNumExpertKinds) fill_experts<DT, STORE, ODD, KIND + 1>(to);
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
    t.route = (const void*)route_tokens;
    return t;
}

}  // namespace gemm_relu_hip
