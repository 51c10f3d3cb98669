// The host side of gemm_relu_blocks.h with a recorder in the place of the HIP
// runtime and of the kernels: the entry points choose and check as ever, and what
// they would launch is kept as JSON.  Pointers are never followed.
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdio>
#include <cstring>
#include <string>

#include "../tiled_dense_gemm_relu_amd/csrc/blocks_api.hip"

namespace {

using namespace gemm_relu_hip;

// Every table entry is an address of its own: which table, and its place there.
char g_blocks[sizeof(BlocksKernels)], g_experts[sizeof(ExpertsKernels)], g_quantize[8], g_zero;
std::string g_log;

template <class Table>
Table addresses(char* base)
{
    Table t;
    const void** p = reinterpret_cast<const void**>(&t);
    for (size_t i = 0; i < sizeof(Table) / sizeof(void*); ++i) p[i] = base + i * sizeof(void*);
    return t;
}
const BlocksKernels g_blocks_table = addresses<BlocksKernels>(g_blocks);
const ExpertsKernels g_experts_table = addresses<ExpertsKernels>(g_experts);

void put(const char* name, long long v)
{
    char s[96];
    std::snprintf(s, sizeof(s), ", \"%s\": %lld", name, v);
    g_log += s;
}
void put(const char* name, const void* p) { put(name, (long long)reinterpret_cast<uintptr_t>(p)); }

void put(const BlocksArgs& a, const std::string& n = "")
{
    const auto name = [&](const char* s) { return n + s; };
    put(name("a").c_str(), a.a), put(name("sa").c_str(), a.sa), put(name("c").c_str(), a.c), put(name("m").c_str(), a.m);
    put(name("n").c_str(), a.n), put(name("k").c_str(), a.k), put(name("groups").c_str(), a.groups);
    put(name("lda").c_str(), (long long)a.lda), put(name("once").c_str(), a.once);
}

}  // namespace

namespace gemm_relu_hip {
const BlocksKernels& blocks_kernels_e4m3_e4m3() { return g_blocks_table; }
const BlocksKernels& blocks_kernels_e4m3_e5m2() { return g_blocks_table; }
const BlocksKernels& blocks_kernels_e5m2_e4m3() { return g_blocks_table; }
const BlocksKernels& blocks_kernels_e5m2_e5m2() { return g_blocks_table; }
const ExpertsKernels& experts_kernels_f16() { return g_experts_table; }
const ExpertsKernels& experts_kernels_bf16() { return g_experts_table; }
const void* quantize_kernel(int, int, int tiles, int vec) { return g_quantize + 2 * tiles + vec; }
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
    prop->multiProcessorCount = 256;
    return hipSuccess;
}

hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t)
{
    const char* f = static_cast<const char*>(fn);
    const ptrdiff_t b = f - g_blocks, e = f - g_experts, q = f - g_quantize;
    const auto within = [](ptrdiff_t at, size_t from, size_t bytes) { return at >= (ptrdiff_t)from && at < (ptrdiff_t)(from + bytes); };
    const auto head = [&](const char* name, ptrdiff_t place) {
        g_log += g_log.empty() ? "{\"kernel\": \"" : ",\n{\"kernel\": \"";
        g_log += name;
        g_log += "\"";
        put("place", (long long)place);
        put("x", (long long)grid.x), put("y", (long long)grid.y), put("threads", (long long)block.x), put("lds", (long long)lds);
    };
    const ptrdiff_t word = sizeof(void*);
    if (fn == &g_zero) {
        head("zero", 0);
        put("c", *static_cast<void**>(args[0])), put("count", (long long)*static_cast<size_t*>(args[1]));
    } else if (within(q, 0, sizeof(g_quantize))) {
        head("quantize", q);
        const QuantizeArgs& a = *static_cast<QuantizeArgs*>(args[0]);
        put("q", a.q), put("s", a.s), put("qt", a.qt), put("st", a.st), put("rows", a.rows), put("cols", a.cols);
        put("tiles_r", a.tiles_r), put("tiles_c", a.tiles_c), put("ldq", (long long)a.ldq), put("ldqt", (long long)a.ldqt);
        put("apart", a.apart);
    } else if (within(b, offsetof(BlocksKernels, tile), sizeof(BlocksKernels::tile))) {
        const ptrdiff_t place = (b - (ptrdiff_t)offsetof(BlocksKernels, tile)) / word;
        head("tile", place / 2);
        put("b_rows", place % 2), put(*static_cast<BlocksArgs*>(args[0]));
    } else if (within(b, offsetof(BlocksKernels, stream), sizeof(BlocksKernels::stream))) {
        const ptrdiff_t place = (b - (ptrdiff_t)offsetof(BlocksKernels, stream)) / word;
        head("stream", place / 2);
        put("b_rows", place % 2), put(*static_cast<BlocksArgs*>(args[0]));
    } else if (b == (ptrdiff_t)offsetof(BlocksKernels, pair)) {
        head("pair", 0);
        const BlocksPair& p = *static_cast<BlocksPair*>(args[0]);
        put(p.product[0], "x_"), put(p.product[1], "w_"), put("blocks_x", p.blocks[0]), put("blocks_w", p.blocks[1]);
    } else if (e == (ptrdiff_t)offsetof(ExpertsKernels, route) || within(e, 0, sizeof(ExpertsKernels::products))) {
        const bool route = e == (ptrdiff_t)offsetof(ExpertsKernels, route);
        head(route ? "route" : "experts", route ? 0 : e / word);
        const ExpertsArgs& a = *static_cast<ExpertsArgs*>(args[0]);
        put("logits", a.logits), put("mid", a.mid), put("part", a.part), put("counters", a.counters), put("in", a.in), put("out", a.out);
        put("mid_row", a.mid_row), put("splits", a.splits), put("once", a.once);
    } else {
        head("unknown", 0);
    }
    g_log += "}";
    return hipSuccess;
}

// The launches since the last call, as a JSON list; the next call of this frees it.
const char* launches()
{
    static std::string kept;
    kept = "[" + g_log + "]";
    g_log.clear();
    return kept.c_str();
}

}  // extern "C"
