// The host side of gemm_relu_groups.h with a recorder in the place of the HIP
// runtime and of the kernels: the entry points choose and check as ever, and what
// they would launch is kept as JSON.  Pointers are never followed.
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdio>
#include <cstring>
#include <string>

#include "../tiled_dense_gemm_relu_amd/csrc/groups_api.hip"

namespace {

using namespace gemm_relu_hip;

// Every table entry is an address of its own: which table, and its place there.
char g_group[sizeof(GroupKernels)], g_staged[sizeof(StagedKernels)], g_zero;
std::string g_log;
int g_cus = 256;

template <class Table>
Table addresses(char* base)
{
    Table t;
    const void** p = reinterpret_cast<const void**>(&t);
    for (size_t i = 0; i < sizeof(Table) / sizeof(void*); ++i) p[i] = base + i * sizeof(void*);
    return t;
}
const GroupKernels g_group_table = addresses<GroupKernels>(g_group);
const StagedKernels g_staged_table = addresses<StagedKernels>(g_staged);

void put(const char* name, long long v)
{
    char s[96];
    std::snprintf(s, sizeof(s), ", \"%s\": %lld", name, v);
    g_log += s;
}
void put(const char* name, const void* p) { put(name, (long long)reinterpret_cast<uintptr_t>(p)); }

void put(const RowsArgs& a)
{
    put("a", a.a), put("b", a.b), put("c", a.c), put("m", a.m), put("n", a.n), put("k", a.k), put("groups", a.groups);
    put("lda", a.lda), put("ldb", a.ldb), put("c_vec", a.c_vec);
}
void put(const WeightArgs& a)
{
    put("p", a.p), put("q", a.q), put("out", a.out), put("m", a.m), put("i", a.i), put("j", a.j);
    put("w_groups", a.groups), put("ldp", a.ldp), put("ldq", a.ldq);
}

}  // namespace

namespace gemm_relu_hip {
const GroupKernels& group_kernels_f16() { return g_group_table; }
const GroupKernels& group_kernels_bf16() { return g_group_table; }
const StagedKernels& staged_kernels_f16_even() { return g_staged_table; }
const StagedKernels& staged_kernels_f16_odd() { return g_staged_table; }
const StagedKernels& staged_kernels_bf16_even() { return g_staged_table; }
const StagedKernels& staged_kernels_bf16_odd() { return g_staged_table; }
const void* zero_fill_kernel() { return &g_zero; }
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
    prop->multiProcessorCount = g_cus;
    return hipSuccess;
}

hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t)
{
    const char* f = static_cast<const char*>(fn);
    const ptrdiff_t g = f - g_group, s = f - g_staged;
    g_log += g_log.empty() ? "{\"kernel\": \"" : ",\n{\"kernel\": \"";
    auto head = [&](const char* name, ptrdiff_t place) {
        g_log += name;
        g_log += "\"";
        put("place", (long long)(place / (ptrdiff_t)sizeof(void*)));
        put("x", (long long)grid.x), put("y", (long long)grid.y), put("threads", (long long)block.x), put("lds", (long long)lds);
    };
    auto within = [](ptrdiff_t at, size_t from, size_t bytes) { return at >= (ptrdiff_t)from && at < (ptrdiff_t)(from + bytes); };
#define MEMBER(table, at, member) within(at, offsetof(table, member), sizeof(table::member))
    if (fn == &g_zero) {
        head("zero", 0);
        put("c", *static_cast<void**>(args[0])), put("count", (long long)*static_cast<size_t*>(args[1]));
    } else if (MEMBER(GroupKernels, g, rows_dma)) {
        head("rows_dma", g - (ptrdiff_t)offsetof(GroupKernels, rows_dma));
        put(*static_cast<RowsArgs*>(args[0]));
        put("v", static_cast<AdapterArgs*>(args[1])->v), put("t", static_cast<AdapterArgs*>(args[1])->t);
    } else if (MEMBER(GroupKernels, g, weight_dma)) {
        head("weight_dma", g - (ptrdiff_t)offsetof(GroupKernels, weight_dma));
        put(*static_cast<WeightArgs*>(args[0]));
    } else if (MEMBER(GroupKernels, g, rows_skinny)) {
        head("rows_skinny", g - (ptrdiff_t)offsetof(GroupKernels, rows_skinny));
        put(*static_cast<RowsArgs*>(args[0]));
        put("v", static_cast<AdapterArgs*>(args[1])->v);
        put("parts", *static_cast<void**>(args[2])), put("counters", *static_cast<void**>(args[3]));
        put("mask", *static_cast<void**>(args[4]));
    } else if (MEMBER(GroupKernels, g, weight_outer)) {
        head("weight_outer", g - (ptrdiff_t)offsetof(GroupKernels, weight_outer));
        put(*static_cast<WeightArgs*>(args[0]));
        put("mask", *static_cast<void**>(args[1]));
    } else if (MEMBER(GroupKernels, g, mask)) {
        head("mask", 0);
        const MaskArgs& a = *static_cast<MaskArgs*>(args[0]);
        put("dc", a.dc), put("c", a.c), put("d", a.d), put("count", (long long)a.count);
    } else if (MEMBER(GroupKernels, g, pad)) {
        head("pad", 0);
        const PadArgs& a = *static_cast<PadArgs*>(args[0]);
        put("src", a.src), put("mask", a.mask), put("dst", a.dst), put("rows", (long long)a.rows), put("cols", a.cols);
        put("pitch", a.pitch);
    } else if (MEMBER(GroupKernels, g, shrink)) {
        head("shrink", g - (ptrdiff_t)offsetof(GroupKernels, shrink));
        const ShrinkArgs& a = *static_cast<ShrinkArgs*>(args[0]);
        put("t", a.t), put("factor", a.factor), put("row_id", a.row_id), put("part", a.part), put("counters", a.counters);
        put("m", a.m), put("k", a.k), put("rank", a.rank), put("rank_pad", a.rank_pad);
    } else if (MEMBER(StagedKernels, s, rows)) {
        head("staged_rows", s - (ptrdiff_t)offsetof(StagedKernels, rows));
        put(*static_cast<RowsArgs*>(args[0]));
    } else if (MEMBER(StagedKernels, s, grad)) {
        head("staged_grad", s - (ptrdiff_t)offsetof(StagedKernels, grad));
        put(*static_cast<RowsArgs*>(args[0])), put(*static_cast<WeightArgs*>(args[1]));
        put("mask", *static_cast<void**>(args[2])), put("blocks_rows", *static_cast<int*>(args[3]));
    } else {
        head("unknown", 0);
    }
#undef MEMBER
    g_log += "}";
    return hipSuccess;
}

int low_rank_first(int n, int N, int whole) { return low_rank_column(n, N, whole != 0); }

// The launches since the last call, as a JSON list; the next call of this frees it.
const char* launches()
{
    static std::string kept;
    kept = "[" + g_log + "]";
    g_log.clear();
    return kept.c_str();
}

}  // extern "C"
