// The host side of gemm_relu_blocks.h with a recorder in the place of the HIP runtime and
// of the kernels, which keeps every argument of the products.  Pointers are never followed.
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstring>
#include <vector>

#include "../tiled_dense_gemm_relu_amd/csrc/blocks_api.hip"

namespace {

using namespace gemm_relu_hip;

char g_tables[4][sizeof(BlocksKernels)], g_experts[sizeof(ExpertsKernels)], g_other;

template <class Table>
Table addresses(char* base)
{
    Table t;
    const void** p = reinterpret_cast<const void**>(&t);
    for (size_t i = 0; i < sizeof(Table) / sizeof(void*); ++i) p[i] = base + i * sizeof(void*);
    return t;
}
const BlocksKernels g_kernels[4] = {addresses<BlocksKernels>(g_tables[0]), addresses<BlocksKernels>(g_tables[1]),
                                    addresses<BlocksKernels>(g_tables[2]), addresses<BlocksKernels>(g_tables[3])};
const ExpertsKernels g_expert_kernels = addresses<ExpertsKernels>(g_experts);

// One product: formats 2 a + b, scales of B by rows, whether one of a pair, and its arguments.
struct Product {
    int64_t formats, b_rows, pair, a, sa, b, sb, c, ends, m, n, k, groups, lda, ldb, relu, bf16;
};
std::vector<Product> g_products;

void keep(int formats, int b_rows, int pair, const BlocksArgs& a)
{
    const auto at = [](const void* p) { return (int64_t) reinterpret_cast<uintptr_t>(p); };
    g_products.push_back(Product{formats, b_rows, pair, at(a.a), at(a.sa), at(a.b), at(a.sb), at(a.c), at(a.ends), a.m, a.n, a.k, a.groups,
                                 a.lda, a.ldb, a.relu, a.bf16});
}

}  // namespace

namespace gemm_relu_hip {
const BlocksKernels& blocks_kernels_e4m3_e4m3() { return g_kernels[0]; }
const BlocksKernels& blocks_kernels_e4m3_e5m2() { return g_kernels[1]; }
const BlocksKernels& blocks_kernels_e5m2_e4m3() { return g_kernels[2]; }
const BlocksKernels& blocks_kernels_e5m2_e5m2() { return g_kernels[3]; }
const ExpertsKernels& experts_kernels_f16() { return g_expert_kernels; }
const ExpertsKernels& experts_kernels_bf16() { return g_expert_kernels; }
const void* quantize_kernel(int, int, int, int) { return &g_other; }
const void* zero_fill_kernel() { return &g_other; }
}  // namespace gemm_relu_hip

extern "C" {

hipError_t hipGetDevice(int* dev)
{
    *dev = 0;
    return hipSuccess;
}

hipError_t hipGetDeviceProperties(hipDeviceProp_t* prop, int)
{
    std::memset(prop, 0, sizeof(*prop));
    std::strcpy(prop->gcnArchName, "gfx950");
    prop->multiProcessorCount = 256;
    return hipSuccess;
}

hipError_t hipLaunchKernel(const void* fn, dim3, dim3, void** args, size_t, hipStream_t)
{
    const char* f = static_cast<const char*>(fn);
    for (int t = 0; t < 4; ++t) {
        const ptrdiff_t at = f - g_tables[t];
        if (at < 0 || at >= (ptrdiff_t)sizeof(BlocksKernels)) continue;
        if (at == (ptrdiff_t)offsetof(BlocksKernels, pair)) {
            const BlocksPair& p = *static_cast<BlocksPair*>(args[0]);
            keep(t, 0, 1, p.product[0]);
            keep(t, 1, 1, p.product[1]);
        } else {
            keep(t, (int)(at / (ptrdiff_t)sizeof(void*)) % 2, 0, *static_cast<BlocksArgs*>(args[0]));
        }
    }
    return hipSuccess;
}

// The products launched since the last call (at most `room`), 17 numbers each; returns how many.
int products(int64_t* to, int room)
{
    const int n = (int)g_products.size();
    for (int i = 0; i < n && i < room; ++i) std::memcpy(to + 17 * i, &g_products[i], sizeof(Product));
    g_products.clear();
    return n;
}

}  // extern "C"
