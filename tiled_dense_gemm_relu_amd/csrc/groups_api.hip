// C ABI of the products whose rows choose their weights (gemm_relu_groups.h):
// argument checks, kernel choice and launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_relu_groups.h"
#include "device.hpp"
#include "groups_table.hpp"
#include "kernel_table.hpp"

namespace gemm_relu_hip {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxGroups = 65535;

// Gradients of fewer operations than this take one register-staged launch.
constexpr double kSmallGrad = 4e9;
// Rows a group, on average, up to which the weights' gradients are written row by
// row (11 rows, 320 x 2248 bf16: 20 us against 29 in the register-staged launch;
// 106 rows in 3 groups, 704 x 5784, are past it: 14 us on tiles).
constexpr int64_t kOuterMost = 16;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// One matrix (or stack of matrices) argument.
struct Span {
    const void* p;
    int64_t bytes;
};

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Checks shared by all entry points: inputs and outputs present, aligned, and
// no output (or the workspace) sharing bytes with anything else.
int check_spans(const Span* in, int n_in, const Span* words, int n_words, const Span* out, int n_out)
{
    for (int i = 0; i < n_in; ++i) {
        if (in[i].bytes > 0 && !in[i].p) return GEMM_RELU_ERR_INVALID_ARG;
        if (in[i].bytes > 0 && !aligned(in[i].p, 2)) return GEMM_RELU_ERR_MISALIGNED;
    }
    for (int i = 0; i < n_words; ++i) {
        if (words[i].bytes > 0 && !words[i].p) return GEMM_RELU_ERR_INVALID_ARG;
        if (words[i].bytes > 0 && !aligned(words[i].p, 4)) return GEMM_RELU_ERR_MISALIGNED;
    }
    for (int i = 0; i < n_out; ++i) {
        if (out[i].bytes > 0 && !out[i].p) return GEMM_RELU_ERR_INVALID_ARG;
        if (out[i].bytes > 0 && !aligned(out[i].p, 2)) return GEMM_RELU_ERR_MISALIGNED;
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return GEMM_RELU_ERR_ALIAS;
        for (int j = 0; j < n_words; ++j)
            if (overlaps(out[i].p, out[i].bytes, words[j].p, words[j].bytes)) return GEMM_RELU_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return GEMM_RELU_ERR_ALIAS;
    }
    return GEMM_RELU_OK;
}

int check_shape(int64_t M, int64_t N, int64_t K, int64_t groups, int dtype, int b_layout)
{
    if (dtype != GEMM_RELU_F16 && dtype != GEMM_RELU_BF16) return GEMM_RELU_ERR_BAD_DTYPE;
    if (b_layout != GEMM_RELU_B_KN && b_layout != GEMM_RELU_B_NK) return GEMM_RELU_ERR_BAD_LAYOUT;
    if (M < 0 || N < 0 || K < 0 || groups < 1) return GEMM_RELU_ERR_INVALID_ARG;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim || groups > kMaxGroups) return GEMM_RELU_ERR_TOO_LARGE;
    return GEMM_RELU_OK;
}

int check_workspace(void* workspace, int64_t bytes, int64_t need)
{
    if (need == 0) return GEMM_RELU_OK;
    return !workspace || bytes < need || !aligned(workspace, 256) ? GEMM_RELU_ERR_WORKSPACE : GEMM_RELU_OK;
}

// How LDS DMA reads a matrix: rows of whole 16-byte pieces, rows of an even
// length at 4-byte alignment (the 128 and 64 tiles), or not at all.
enum DmaRows { kDmaNone = 0, kDmaEven = 1, kDmaWhole = 2 };
DmaRows dma_rows(const void* p, int64_t row)
{
    return row % 8 == 0 && aligned(p, 16) ? kDmaWhole : row % 2 == 0 && aligned(p, 4) ? kDmaEven : kDmaNone;
}

int store_width(const void* c, int64_t n) { return n % 8 == 0 && aligned(c, 16) ? 2 : n % 4 == 0 && aligned(c, 8) ? 1 : 0; }

const GroupKernels& kernels(int dtype) { return dtype == GEMM_RELU_F16 ? group_kernels_f16() : group_kernels_bf16(); }

// The register-staged kernels for matrices with these rows: elements that start
// inside a dword need more loads and shifts.
struct Rows {
    const void* p;
    int64_t length;
};
bool even_rows(std::initializer_list<Rows> operands)
{
    for (const Rows& r : operands)
        if (r.length % 2 != 0 || !aligned(r.p, 4)) return false;
    return true;
}
const StagedKernels& staged_kernels(int dtype, std::initializer_list<Rows> operands)
{
    const bool even = even_rows(operands);
    if (dtype == GEMM_RELU_F16) return even ? staged_kernels_f16_even() : staged_kernels_f16_odd();
    return even ? staged_kernels_bf16_even() : staged_kernels_bf16_odd();
}

// Whether one launch can have that many workgroups: their threads are counted in 32 bits.
bool launchable(int64_t blocks, int threads) { return blocks <= int64_t(UINT32_MAX) / threads; }

int enqueue(const void* fn, dim3 grid, int threads, void** args, hipStream_t stream, size_t lds = 0)
{
    const hipError_t err = hipLaunchKernel(fn, grid, dim3((unsigned)threads), args, lds, stream);
    return err == hipSuccess ? GEMM_RELU_OK : GEMM_RELU_ERR_LAUNCH;
}

int zero_fill(void* p, int64_t halves, hipStream_t stream)
{
    if (halves <= 0) return GEMM_RELU_OK;
    size_t count = (size_t)halves;
    void* args[] = {&p, &count};
    return enqueue(zero_fill_kernel(), dim3((unsigned)std::min<int64_t>(ceil_div(halves, 256), 65536)), 256, args, stream);
}

// Row tiles that `groups` groups (and the rows of none) can have among M rows:
// whole tiles, and one partial tile for each.
int64_t most_row_tiles(int64_t M, int64_t groups, int64_t rows) { return std::min(M, M / rows + groups + 1); }

bool known_config(int id) { return id >= GEMM_RELU_GROUPS_AUTO && id <= GEMM_RELU_GROUPS_STREAM; }

// Tile of an LDS-DMA product: the largest whose tiles are mostly full (`rows`:
// a group's rows on average) and numerous enough to occupy the CUs.  Measured, us:
// 8192 rows in 16 ragged groups, 4096 x 4096 bf16, 256 tile 300, 128 tile 337;
// with 2048 columns 188 and 174; 4096 rows in 32 groups, 2048 x 2048, 128 tile 50,
// 64 tile 86; 256 rows in 8 groups, 512 x 512, 9.0 and 7.5.
int dma_config(int64_t rows, int64_t tiles_256, int64_t tiles_128)
{
    if (rows >= 192 && tiles_256 >= 192) return GEMM_RELU_GROUPS_DMA_256;
    if (rows >= 96 && tiles_128 >= 128) return GEMM_RELU_GROUPS_DMA_128;
    return GEMM_RELU_GROUPS_DMA_64;
}

// Rows of a group on average, and the tiles of `tile` x `tile` that this makes.
struct GroupShape {
    int64_t used, rows;
    GroupShape(int64_t m, int64_t groups) : used(std::min(groups, m)), rows(m / used) {}
    int64_t tiles(int64_t tile, int64_t n) const { return used * ceil_div(rows, tile) * ceil_div(n, tile); }
};

// Position in kStagedTile of the tile of a register-staged product.  Measured, us,
// bf16 KN, tiles of 128 / 64.  Many rows a group and long sums are for 128: 8192 rows in
// 16 groups, 2048 x 4096 343 / 513; 4096 in 32, 2048 x 2048 143 / 173; 2048 in one 42 / 58;
// 1024 in 8, 1024 x 2048 25 / 31.  Too few tiles are not: 700 in 7, 1101 x 517 33 / 18;
// 512 in 4, 1024 x 1024 24 / 16.  Between them this rule can be wrong, where 128 makes a
// second round of a few tiles or sums are short: 4096 in 16, 1025 x 1029 59 / 52; 1536 in
// 16, 513 x 2051 43 / 29; 2000 in 8, 301 x 1501 27 / 20.  Both gradients: 2048 in one,
// 2048 x 2048 123 / 166; 8192 in 16, 2048 x 4096 1439 / 1574; 4096 in 32, 2048 x 2048 758 /
// 613 (dB has two K-steps a tile there); 800 in 8, 1024 x 1024 28 / 38, where it takes 64.
int staged_tile(int64_t rows, int64_t tiles_128) { return rows >= 96 && tiles_128 >= 128 ? 0 : 1; }

// Persistent workgroups for `tiles` units: as many as run at once (two of the
// 64 x 64 kernels on a CU).
int64_t resident(int64_t tile, int64_t tiles, int cus) { return std::min<int64_t>(tiles, tile == 64 ? 2 * cus : cus); }

// The streaming kernel's part in a product: which one (by kSkinnyBlocks), and
// into how many parts K is cut: as many as make 512 workgroups, while each of
// their 8 waves has a piece of K.  A group's rows should mostly fit a
// workgroup's, since every further workgroup reads the weights again; but small
// workgroups are more, and fill the CUs where K is not cut.  Measured, us on the
// device, bf16 KN (NK), workgroups of 16 / 32 / 64 rows:
//   1 row, 4096 x 4096             12.5 / 13.0 / 16.8   (11.3 / 11.9 / 16.5)
//   32 rows in 8 groups, 2048 x 1024   13.2 / 13.0 / 16.5   (12.1 / 13.7 / 18.9)
//   320 in 32, 1024 x 1024         20.8 / 18.9 / 28.1   (22.8 / 23.8 / 29.8)
//   160 in 8, 512 x 512             4.9 /  4.6 /  5.5   ( 5.5 /  4.9 /  5.6)
//   100 in 4, 8192 x 300           17.4 / 15.6 / 18.7   (17.4 / 16.4 / 18.6)
//   64 in one, 2048 x 512           7.8 /  8.7 / 10.9   ( 8.8 /  9.7 / 11.9)
//   64 in one, 12001 x 1304        55.5 / 45.3 / 29.2   (B^T as in a gradient, KN)
//   40 in one, 12001 x 2048        80.6 / 75.5 / 48.1   (the same)
// So 64 rows pay for long sums over wide weights and cost up to two fifths in small
// products of 20 to 64 rows a group, which this rule does not tell apart.
struct SkinnyPlan {
    int kind = -1;
    int64_t units = 0, splits = 1, bytes = 0;
    SkinnyPlan(int64_t m, int64_t n, int64_t k, int64_t groups)
    {
        if (m == 0 || n == 0 || k == 0) return;
        const GroupShape g(m, groups);
        const int64_t most = groups == 1 ? m : g.rows + g.rows / 2 + 6;     // few groups have more rows
        kind = most <= 16 ? 0 : most <= 32 ? 1 : 2;
        units = most_row_tiles(m, groups, 16 * kSkinnyBlocks[kind]) * ceil_div(n, kSkinnyCols);
        splits = std::max<int64_t>(1, std::min<int64_t>(ceil_div(k, 8 * kSkinnyK), 512 / units));
        if (splits > 1) bytes = units * splits * kSkinnyBlocks[kind] * kSkinnyThreads * 4;
    }
    bool fits() const { return launchable(units, kSkinnyThreads); }
};

// Whether to stream.  The streaming kernel starts and ends quicker than the tiles
// and cuts K where there are few units, but every 32 columns read the rows of A
// again and it reaches 3 TB/s, where the 64 x 64 tiles reach 5, or a K-step of 64
// in 0.16 us (0.35 us where rows must go through registers).  Measured, us,
// streaming against tiles, KN: 1, 8 and 16 rows x 4096 x 4096 bf16 10.9 / 16.2,
// 15.7 / 16.3, 24.5 / 16.4; 4 rows x 16384 x 4096 55 / 27; 64 rows in 8 groups
// 512 x 512 4.4 / 6.4; 16 rows x 300 x 8192 7.4 / 49.
bool streams(int64_t m, int64_t n, int64_t k, int64_t groups, bool dma)
{
    const GroupShape g(m, groups);
    if (g.rows > 64 || !SkinnyPlan(m, n, k, groups).fits()) return false;
    const double weights = 2.0 * (double)g.used * (double)n * (double)k, again = 2.0 * (double)m * (double)k * (double)ceil_div(n, kSkinnyCols);
    const double rounds = (double)ceil_div(g.tiles(64, n), 512), step = dma ? 0.16 : 0.35;
    return 3.0 + (weights + again) / 3.2e6 < 5.5 + std::max(weights / 5e6, rounds * (double)ceil_div(k, 64) * step);
}

// The streaming kernel, for A masked by `mask` if that is not NULL.  Its rows of A
// and B are as long as the product says (lda == k), never copies with a pitch.
// `parts` (may be NULL) and `counters`: space for partial sums.
int launch_stream(RowsArgs a, AdapterArgs ad, const uint16_t* mask, int dtype, int b_layout, float* parts, int* counters,
                  hipStream_t stream)
{
    SkinnyPlan plan(a.m, a.n, a.k, a.groups);
    if (!parts) plan.splits = 1;
    const bool even = even_rows({{a.a, a.lda}, {mask, a.lda}, {a.b, a.ldb}});
    void* args[] = {&a, &ad, &parts, &counters, &mask};
    return enqueue(kernels(dtype).rows_skinny[plan.kind][b_layout][!even][ad.v ? 1 : mask ? 2 : 0],
                   dim3((unsigned)plan.units, (unsigned)plan.splits), kSkinnyThreads, args, stream);
}

// Weights' gradients with few rows a group; `mask` (may be NULL) belongs to w.q if
// mask_q, else to w.p.
int launch_outer(WeightArgs w, const uint16_t* mask, bool mask_q, int dtype, hipStream_t stream)
{
    const bool whole = w.j % 8 == 0 && aligned(w.q, 16) && aligned(w.out, 16) && (!mask || aligned(mask, 16));
    const int64_t tiles = outer_tiles(w.i, w.j, whole) * w.groups;
    void* args[] = {&w, &mask};
    return enqueue(kernels(dtype).weight_outer[!mask ? 0 : mask_q ? 2 : 1][whole], dim3((unsigned)tiles), kOuterThreads, args,
                   stream);
}

// Rows of an odd length reach LDS only through registers, at about half the
// pace.  Where the product is large enough, such operands are first copied to
// rows of whole cache lines.  The estimates (us): a 128 x 128 x 64 step takes
// 5.7e-3 of the device through registers and 2.65e-3 by DMA, or, in a chain of
// steps on 64 x 64 tiles, 0.55 and 0.17; a copy moves 4.2 TB/s.  (1823 rows x
// 12800 x 2125 fp16 in 3 groups: 290 us through registers, 172 with the copies.)
int64_t pitch(int64_t row) { return round_up(row, 64); }
struct PaddedPlan {
    bool use = false;
    int64_t bytes = 0;
    // `steps`: of 128 x 128 x 64; `chain`: rounds of 64 x 64 tiles times their steps
    void weigh(double steps, double chain, int copies)
    {
        const double staged = std::max(5.7e-3 * steps, 0.55 * chain), dma = std::max(2.65e-3 * steps, 0.17 * chain);
        use = dma + 2.0 * (double)bytes / 4.2e6 + 4.0 * copies < staged;
        if (!use) bytes = 0;
    }
    int64_t add(int64_t rows, int64_t row) { return bytes += row % 2 ? round_up(2 * rows * pitch(row), 256) : 0; }
};
struct PaddedRows : PaddedPlan {
    PaddedRows(int64_t m, int64_t n, int64_t k, int64_t groups, int b_layout)
    {
        if (m == 0 || n == 0 || k == 0) return;
        const bool nk = b_layout == GEMM_RELU_B_NK;
        add(m, k);
        add(groups * (nk ? n : k), nk ? k : n);
        if (bytes == 0) return;
        const GroupShape g(m, groups);
        const double ks = (double)ceil_div(k, 64);
        weigh((double)g.tiles(128, n) * ks, (double)ceil_div(g.tiles(64, n), 512) * ks, k % 2 + (nk ? k : n) % 2);
    }
};
struct PaddedGrad : PaddedPlan {
    PaddedGrad(int64_t m, int64_t n, int64_t k, int64_t groups, int b_layout)
    {
        if (m == 0 || n == 0 || k == 0) return;
        const bool nk = b_layout == GEMM_RELU_B_NK;
        add(m, n);
        add(m, k);
        add(groups * (nk ? n : k), nk ? k : n);
        // Below kSmallGrad the register-staged launch is alone, the copies' way has five.
        // fp16, us, registers / copies with the mask (without): 1000 rows in 7 groups, 1101 x
        // 517 35 / 52 (29 / 52); 1000 in one, 1001 x 801 30 / 31 (21 / 30); 400 in 2, 1501 x
        // 1501 52 / 52 (37 / 51); 2000 in 4, 701 x 701 36 / 44 (27 / 44); 300 in 10, 1101 x
        // 1101 59 / 54 (45 / 53).  Above: 1500 in 6, 1201 x 1001 63 / 60 (49 / 60), where the
        // estimate below says registers; 2003 in 3, 2051 x 1101 126 / 87 (91 / 87).
        if (bytes == 0 || 4.0 * (double)m * (double)n * (double)k < kSmallGrad) {
            bytes = 0;
            return;
        }
        const GroupShape g(m, groups);
        const double ns = (double)ceil_div(n, 64), ms = (double)ceil_div(g.rows, 64);
        const auto weights = [&](int64_t t) { return (double)groups * (double)ceil_div(k, t) * (double)ceil_div(n, t) * ms; };
        weigh((double)g.tiles(128, k) * ns + weights(128), ((double)g.tiles(64, k) * ns + weights(64)) / 512, n % 2 + k % 2 + (nk ? k : n) % 2);
    }
};

// Copies rows of an odd length to `to`, masked if `mask` is not NULL; `p` and `row`
// become the copy's, `to` moves past it.
int launch_pad(const uint16_t*& p, int& row, const uint16_t* mask, int64_t rows, char*& to, int dtype, hipStream_t stream)
{
    PadArgs a{p, mask, reinterpret_cast<uint16_t*>(to), rows, row, (int)pitch(row)};
    void* args[] = {&a};
    const int rc = enqueue(kernels(dtype).pad, dim3((unsigned)std::min<int64_t>(ceil_div(rows, 4), 4096)), 256, args, stream);
    to += round_up(2 * rows * a.pitch, 256);
    p = a.dst;
    row = a.pitch;
    return rc;
}

// A product over row groups (M, N, K > 0).  `parts` (may be NULL) and `counters`:
// space for the streaming kernel's partial sums, or for the copies of PaddedRows.
int launch_rows(RowsArgs a, AdapterArgs ad, int dtype, int b_layout, int config, int cus, float* parts, int* counters,
                hipStream_t stream)
{
    a.c_vec = store_width(a.c, a.n);
    DmaRows dma = std::min(dma_rows(a.a, a.lda), dma_rows(a.b, a.ldb));
    const bool whole_rows = a.lda == a.k && a.ldb == (b_layout == GEMM_RELU_B_NK ? a.k : a.n);
    if (config == GEMM_RELU_GROUPS_STREAM && !SkinnyPlan(a.m, a.n, a.k, a.groups).fits()) config = GEMM_RELU_GROUPS_AUTO;
    if (whole_rows && (config == GEMM_RELU_GROUPS_STREAM ||
                       (config == GEMM_RELU_GROUPS_AUTO && streams(a.m, a.n, a.k, a.groups, dma != kDmaNone))))
        return launch_stream(a, ad, nullptr, dtype, b_layout, parts, counters, stream);
    if (dma == kDmaNone && config != GEMM_RELU_GROUPS_TILED && parts && PaddedRows(a.m, a.n, a.k, a.groups, b_layout).use) {
        char* to = reinterpret_cast<char*>(parts);
        int rc = GEMM_RELU_OK;
        if (a.lda % 2) rc = launch_pad(a.a, a.lda, nullptr, a.m, to, dtype, stream);
        if (a.ldb % 2 && rc == GEMM_RELU_OK)
            rc = launch_pad(a.b, a.ldb, nullptr, int64_t(a.groups) * (b_layout == GEMM_RELU_B_NK ? a.n : a.k), to, dtype, stream);
        if (rc != GEMM_RELU_OK) return rc;
        dma = std::min(dma_rows(a.a, a.lda), dma_rows(a.b, a.ldb));      // (of even rows one may be misaligned still)
    }
    int staged = 0;
    if (dma == kDmaNone) {
        const GroupShape g(a.m, a.groups);
        if (config != GEMM_RELU_GROUPS_TILED) staged = staged_tile(g.rows, g.tiles(128, a.n));
        config = GEMM_RELU_GROUPS_TILED;
    }
    // With adapters the 256 tile cuts its rows at the segments' ends and streams V
    // like B; the others take rows of many segments.
    const auto auto_config = [&](int64_t groups) {
        const GroupShape g(a.m, groups);
        return dma_config(g.rows, g.tiles(256, a.n), g.tiles(128, a.n));
    };
    if (config == GEMM_RELU_GROUPS_AUTO) {
        config = auto_config(ad.v ? ad.segments : a.groups);
        // 4096 rows, 4096 x 8192 bf16 KN, rank 64, 256 tiles cut at the segments' ends / 128
        // tiles of many segments, us: 2 to 8 segments 314 / 340-350, 10 339 / 338, 16 395 / 346
        // (NK, rank 16: 373 / 419), 32 544 / 371; 2048 rows in 4 205 / 180.  So 192 rows a
        // segment, the bar of dma_config, is too few for KN.  Where 256 tiles are refused, 128
        // against 64, 4096 x 4096, rank 16: 512 rows in 64 segments 57 / 49, 700 in 40 50 / 61,
        // 2048 in 256 117 / 148, 4096 in 64 171 / 246.
        if (ad.v && config != GEMM_RELU_GROUPS_DMA_256) config = std::max<int>(auto_config(1), GEMM_RELU_GROUPS_DMA_128);
    }
    if (config == GEMM_RELU_GROUPS_DMA_256 &&
        (dma < kDmaWhole || (ad.v && dma_rows(ad.v, b_layout == GEMM_RELU_B_NK ? ad.rank : a.n) < kDmaWhole)))
        config = GEMM_RELU_GROUPS_DMA_128;
    const bool first = config == GEMM_RELU_GROUPS_DMA_256 && ad.v;
    const int64_t rows = config == GEMM_RELU_GROUPS_TILED ? kStagedTile[staged] : kGroupTile[config - 1];
    const int64_t tiles = most_row_tiles(a.m, first ? ad.segments : a.groups, rows) * ceil_div(a.n, rows);
    if (tiles > INT32_MAX) return GEMM_RELU_ERR_TOO_LARGE;
    void* args[] = {&a, &ad};
    const dim3 grid((unsigned)resident(rows, tiles, cus));
    if (config == GEMM_RELU_GROUPS_TILED)
        return enqueue(staged_kernels(dtype, {{a.a, a.lda}, {a.b, a.ldb}})
                           .rows[staged][b_layout][ad.v != nullptr][a.groups > 64], grid, kStagedThreads, args, stream);
    return enqueue(kernels(dtype).rows_dma[config - 1][b_layout][dma < kDmaWhole ? 2 : a.k % 64 != 0][ad.v != nullptr], grid,
                   kGroupThreads[config - 1], args, stream);
}

// Sums over each group's rows (I, J > 0), by LDS DMA.
int launch_weights(WeightArgs a, int dtype, int config, int cus, hipStream_t stream)
{
    if (config == GEMM_RELU_GROUPS_AUTO)
        config = dma_config(a.i, a.groups * ceil_div(a.i, 256) * ceil_div(a.j, 256),
                            a.groups * ceil_div(a.i, 128) * ceil_div(a.j, 128));
    const bool whole = std::min(dma_rows(a.p, a.ldp), dma_rows(a.q, a.ldq)) == kDmaWhole;
    if (config == GEMM_RELU_GROUPS_DMA_256 && !whole) config = GEMM_RELU_GROUPS_DMA_128;
    const int64_t tile = kGroupTile[config - 1], tiles = int64_t(a.groups) * ceil_div(a.i, tile) * ceil_div(a.j, tile);
    if (tiles > INT32_MAX) return GEMM_RELU_ERR_TOO_LARGE;
    void* args[] = {&a};
    return enqueue(kernels(dtype).weight_dma[config - 1][!whole], dim3((unsigned)resident(tile, tiles, cus)), kGroupThreads[config - 1],
                   args, stream);
}

// Whether both gradients are better computed in one register-staged launch than by
// a mask and two DMA launches: few operations (the launches cost about 8 us more),
// unless their chains of K-steps are long (0.4 us a step against 0.17).
bool small_grad(int64_t m, int64_t n, int64_t k, int64_t groups)
{
    const GroupShape g(m, groups);
    const double chain = (double)ceil_div(g.tiles(64, k), 512) * (double)ceil_div(n, 64);
    return 4.0 * (double)m * (double)n * (double)k < kSmallGrad && 0.23 * chain < 8.0;
}

// Both gradients (or one: the other's output is NULL) in one register-staged
// launch.  b_layout is that of dA's product.  The workgroups are shared out by
// the two products' K-steps, a tile counting as four more for its start and end.
int launch_grad_staged(RowsArgs r, WeightArgs w, const uint16_t* mask, int dtype, int b_layout, int config, int cus,
                       hipStream_t stream)
{
    r.c_vec = store_width(r.c, r.n);
    w.c_vec = store_width(w.out, w.j);
    const GroupShape g(r.m, r.groups);
    const auto weight_tiles = [&](int64_t t) { return int64_t(w.groups) * ceil_div(w.i, t) * ceil_div(w.j, t); };
    const int staged =
        config == GEMM_RELU_GROUPS_TILED ? 0 : staged_tile(g.rows, std::min(g.tiles(128, r.n), weight_tiles(128)));
    const int64_t t = kStagedTile[staged];
    const int64_t tiles_r = r.c ? most_row_tiles(r.m, r.groups, t) * ceil_div(r.n, t) : 0, tiles_w = w.out ? weight_tiles(t) : 0;
    if (tiles_r > INT32_MAX || tiles_w > INT32_MAX) return GEMM_RELU_ERR_TOO_LARGE;
    const int64_t room = resident(t, INT32_MAX, cus);
    const double work_r = tiles_r ? (double)g.tiles(t, r.n) * (double)(ceil_div(r.k, 64) + 4) : 0;
    const double work_w = (double)tiles_w * (double)(ceil_div(g.rows, 64) + 4);
    int64_t blocks_r = tiles_r == 0 ? 0 : (int64_t)((double)room * work_r / (work_r + work_w));
    if (tiles_r > 0) blocks_r = std::min(tiles_r, std::max<int64_t>(1, blocks_r > 8 ? blocks_r / 8 * 8 : blocks_r));
    if (tiles_w > 0) blocks_r = std::min(blocks_r, room - 1);
    const int64_t blocks_w = std::min(tiles_w, room - blocks_r);
    int blocks_rows = (int)blocks_r;
    void* args[] = {&r, &w, &mask, &blocks_rows};
    const bool nk = b_layout == GEMM_RELU_B_NK;
    const Rows d{r.a, r.lda}, c{mask, r.lda}, b{r.c ? r.b : nullptr, r.ldb}, x{w.out ? (nk ? w.p : w.q) : nullptr, nk ? w.ldp : w.ldq};
    return enqueue(staged_kernels(dtype, {d, c, b, x}).grad[staged][b_layout][mask != nullptr][r.groups > 64], dim3((unsigned)(blocks_r + blocks_w)),
                   kStagedThreads, args, stream);
}

// d = dc where c > 0, else +0.0.
int launch_mask(const uint16_t* dc, const uint16_t* c, uint16_t* d, int64_t count, int dtype, hipStream_t stream)
{
    MaskArgs m{dc, c, d, count, aligned(dc, 16) && aligned(c, 16)};
    void* args[] = {&m};
    return enqueue(kernels(dtype).mask, dim3((unsigned)std::min<int64_t>(ceil_div(count, 2048), 4096)), 256, args, stream);
}

// dA alone: r.a is dC, masked by `c` (unless NULL) on the way, into `masked`.
int launch_grad_rows(RowsArgs r, const uint16_t* c, uint16_t* masked, int dtype, int b_layout, int config, int cus, hipStream_t stream)
{
    if (c) {
        const int rc = launch_mask(r.a, c, masked, int64_t(r.m) * r.k, dtype, stream);
        if (rc != GEMM_RELU_OK) return rc;
        r.a = masked;
    }
    return launch_rows(r, AdapterArgs{}, dtype, b_layout, config, cus, nullptr, nullptr, stream);
}

// Workspace of the adapters: the counters, the intermediates, each row's
// adapter, and the partial sums of a K that is cut into `splits` parts: as many
// as make 512 workgroups, while each of their 8 waves has a piece of K.
struct AdapterSpace {
    int64_t rank_pad, blocks, tiles, splits, t, factor, row_id, part, bytes;   // part: also the streaming kernel's, afterwards
};
AdapterSpace adapter_space(int64_t M, int64_t N, int64_t K, int64_t rank, int64_t segments, int b_layout)
{
    AdapterSpace s;
    s.rank_pad = round_up(rank, 64);
    // Two blocks of rows a workgroup, which read U once, where segments fill them.  First
    // product and one of 256 columns, K 4096, bf16 KN (NK), us, one block / two: rank 16:
    // 1024 rows in 4 segments 31.9 / 32.7 (32.7 / 33.0), 2048 in 8 35.6 / 34.8 (35.4 / 36.6),
    // 4096 in 6 43.0 / 40.0 (44.7 / 40.5), 8192 in 16 63.4 / 65.8 (82.2 / 85.7), 12000 in 20
    // 85.2 / 74.1 (104 / 95); rank 64: 1024 36.6 / 37.6 (39.9 / 39.2), 4096 51.1 / 46.6 (65.7 /
    // 51.9), 12000 108 / 92 (147 / 119).  32 rows a segment (4096 in 128, 1024 columns): rank
    // 64 92.6 / 95.7.
    s.blocks = M > 0 && GroupShape(M, segments).rows >= 48 && M >= 1024 ? 2 : 1;
    s.tiles = most_row_tiles(M, segments, s.blocks * kShrinkRows);
    s.splits = std::max<int64_t>(1, std::min<int64_t>(ceil_div(K, 8 * kShrinkK), s.tiles ? 512 / s.tiles : 1));
    s.t = GEMM_RELU_GROUPS_COUNTER_BYTES;
    s.factor = s.t + round_up(M * 2 * s.rank_pad * 2, 256);
    s.row_id = s.factor + round_up(M * 4, 256);
    s.part = s.row_id + round_up(M * 4, 256);
    s.bytes = s.part + std::max(s.splits > 1 ? s.tiles * s.splits * ceil_div(rank, kShrinkCols) * s.blocks * kShrinkThreads * 4 : 0,
                                std::max(SkinnyPlan(M, N, K, 1).bytes, PaddedRows(M, N, K, 1, b_layout).bytes));
    return s;
}
static_assert(512 * 4 <= GEMM_RELU_GROUPS_COUNTER_BYTES, "a counter for each row tile of a split sum");

}  // namespace
}  // namespace gemm_relu_hip

using namespace gemm_relu_hip;

extern "C" {

int64_t gemm_relu_grouped_workspace(int64_t M, int64_t N, int64_t K, int64_t groups, int dtype, int b_layout)
{
    const int rc = check_shape(M, N, K, groups, dtype, b_layout);
    if (rc != GEMM_RELU_OK) return rc;
    const int64_t bytes = std::max(SkinnyPlan(M, N, K, groups).bytes, PaddedRows(M, N, K, groups, b_layout).bytes);
    return bytes ? GEMM_RELU_GROUPS_COUNTER_BYTES + bytes : 0;
}

int gemm_relu_grouped(const void* A, const void* B, const int32_t* ends, void* C, int64_t M, int64_t N,
                      int64_t K, int64_t groups, int dtype, int b_layout, int relu, int config_id,
                      void* workspace, int64_t workspace_bytes, void* stream)
{
    const int64_t need = gemm_relu_grouped_workspace(M, N, K, groups, dtype, b_layout);
    if (need < 0) return (int)need;
    if (relu != 0 && relu != 1) return GEMM_RELU_ERR_INVALID_ARG;
    if (!known_config(config_id)) return GEMM_RELU_ERR_BAD_CONFIG;
    if (M == 0 || N == 0) return GEMM_RELU_OK;
    const Span in[] = {{A, 2 * M * K}, {B, 2 * groups * K * N}}, words[] = {{ends, 4 * groups}};
    const Span out[] = {{C, 2 * M * N}, {workspace, need}};
    int rc = check_spans(in, 2, words, 1, out, 1);
    if (rc == GEMM_RELU_OK) rc = check_workspace(workspace, workspace_bytes, need);
    if (rc == GEMM_RELU_OK) rc = check_spans(in, 2, words, 1, out, need > 0 ? 2 : 1);
    if (rc != GEMM_RELU_OK) return rc;
    int cus = 0;
    if ((rc = check_device(&cus)) != GEMM_RELU_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) return zero_fill(C, M * N, s);
    RowsArgs a{static_cast<const uint16_t*>(A), static_cast<const uint16_t*>(B), static_cast<uint16_t*>(C), ends,
               (int)M, (int)N, (int)K, (int)groups, relu, (int)K, (int)(b_layout == GEMM_RELU_B_NK ? K : N), 0};
    float* parts = need ? reinterpret_cast<float*>(static_cast<char*>(workspace) + GEMM_RELU_GROUPS_COUNTER_BYTES) : nullptr;
    return launch_rows(a, AdapterArgs{}, dtype, b_layout, config_id, cus, parts, static_cast<int*>(workspace), s);
}

int64_t gemm_relu_grouped_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t groups, int dtype,
                                             int b_layout, int relu)
{
    const int rc = check_shape(M, N, K, groups, dtype, b_layout);
    if (rc != GEMM_RELU_OK) return rc;
    if (relu != 0 && relu != 1) return GEMM_RELU_ERR_INVALID_ARG;
    // the masked gradient and partial sums of dA's product (inner dimension N), or
    // the copies of operands with odd rows, the masked gradient's among them
    const int64_t masked = relu ? round_up(2 * M * N, 256) : 0, padded = PaddedGrad(M, N, K, groups, b_layout).bytes;
    return GEMM_RELU_GROUPS_COUNTER_BYTES +
           std::max(masked + SkinnyPlan(M, K, N, groups).bytes, padded ? padded + (N % 2 ? 0 : masked) : 0);
}

int gemm_relu_grouped_backward(const void* dC, const void* C, const void* A, const void* B, const int32_t* ends,
                               void* dA, void* dB, int64_t M, int64_t N, int64_t K, int64_t groups, int dtype,
                               int b_layout, int relu, int config_id, void* workspace, int64_t workspace_bytes,
                               void* stream)
{
    const int64_t need = gemm_relu_grouped_backward_workspace(M, N, K, groups, dtype, b_layout, relu);
    if (need < 0) return (int)need;
    if (!known_config(config_id)) return GEMM_RELU_ERR_BAD_CONFIG;
    const bool want_a = dA != nullptr, want_b = dB != nullptr;
    if (!want_a && !want_b && K > 0) return GEMM_RELU_ERR_INVALID_ARG;
    if (K == 0) return GEMM_RELU_OK;                 // both gradients are empty
    const int64_t mn = M * N, mk = M * K, gkn = groups * K * N;
    const Span in[] = {{dC, 2 * mn}, {relu ? C : nullptr, relu ? 2 * mn : 0}, {want_b ? A : nullptr, want_b ? 2 * mk : 0},
                       {want_a ? B : nullptr, want_a ? 2 * gkn : 0}};
    const Span words[] = {{ends, 4 * groups}};
    const Span out[] = {{dA, want_a ? 2 * mk : 0}, {dB, want_b ? 2 * gkn : 0}, {workspace, need}};
    int rc = check_spans(in, 4, words, 1, out, 2);
    if (rc == GEMM_RELU_OK) rc = check_workspace(workspace, workspace_bytes, need);
    if (rc == GEMM_RELU_OK) rc = check_spans(in, 4, words, 1, out, 3);
    if (rc != GEMM_RELU_OK) return rc;
    int cus = 0;
    if ((rc = check_device(&cus)) != GEMM_RELU_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (mn == 0) {                                   // empty sums
        if (want_a) rc = zero_fill(dA, mk, s);
        if (want_b && rc == GEMM_RELU_OK) rc = zero_fill(dB, gkn, s);
        return rc;
    }
    const uint16_t *d = static_cast<const uint16_t*>(dC), *c = relu ? static_cast<const uint16_t*>(C) : nullptr;
    const uint16_t *x = static_cast<const uint16_t*>(A), *b = static_cast<const uint16_t*>(B);
    // dA = D (M, N) times B^T: B as stored (K, N) is the transposed weight of this product
    const bool kn = b_layout == GEMM_RELU_B_KN;
    const int64_t masked_bytes = relu ? round_up(2 * mn, 256) : 0, parts_at = GEMM_RELU_GROUPS_COUNTER_BYTES + masked_bytes;
    uint16_t* masked = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + GEMM_RELU_GROUPS_COUNTER_BYTES);
    const int layout_a = kn ? GEMM_RELU_B_NK : GEMM_RELU_B_KN;
    RowsArgs r{d, b, static_cast<uint16_t*>(dA), ends, (int)M, (int)K, (int)N, (int)groups, 0, (int)N, (int)(kn ? N : K), 0};
    WeightArgs w{kn ? x : d, kn ? d : x, static_cast<uint16_t*>(dB), ends, (int)M, (int)(kn ? K : N), (int)(kn ? N : K),
                 (int)groups, (int)(kn ? K : N), (int)(kn ? N : K), 0};
    // Few rows a group: the weights' gradients are written, the weights read, at memory's pace.
    // (Streaming is dA's: on request all of dA streams, and dB goes as by default.)
    const bool stream_only = config_id == GEMM_RELU_GROUPS_STREAM && SkinnyPlan(M, K, N, groups).fits();
    const int config = config_id == GEMM_RELU_GROUPS_STREAM ? GEMM_RELU_GROUPS_AUTO : config_id;
    const bool outer = config == GEMM_RELU_GROUPS_AUTO && GroupShape(M, groups).rows <= kOuterMost &&
                       outer_tiles(w.i, w.j, false) * groups <= INT32_MAX / kOuterThreads;   // lanes are numbered in an int
    const bool stream_a = want_a && (stream_only || (config == GEMM_RELU_GROUPS_AUTO &&
                                                     streams(M, K, N, groups, std::min(dma_rows(d, N), dma_rows(b, kn ? N : K)))));
    float* parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + parts_at);
    bool tiles_a = want_a;
    const auto stream_rows = [&] {     // dA from the matrices as they are
        tiles_a = false;
        const int streamed = launch_stream(r, AdapterArgs{}, c, dtype, layout_a, parts, static_cast<int*>(workspace), s);
        r.c = nullptr;
        return streamed;
    };
    if (stream_a && (stream_only || outer)) rc = stream_rows();
    if (outer) {
        if (tiles_a) rc = launch_grad_rows(r, c, masked, dtype, layout_a, config, cus, s);
        if (want_b && rc == GEMM_RELU_OK) rc = launch_outer(w, c, kn, dtype, s);
        return rc;
    }
    if (rc != GEMM_RELU_OK || !(tiles_a || want_b)) return rc;
    // LDS DMA needs rows of an even length and D itself in memory.  The register-
    // staged kernel needs neither, and is one launch instead of two or three.
    const bool dma = dma_rows(d, N) && (!tiles_a || dma_rows(b, kn ? N : K)) && (!want_b || dma_rows(x, K));   // kDmaNone: false
    if (!dma && config != GEMM_RELU_GROUPS_TILED && PaddedGrad(M, N, K, groups, b_layout).use) {
        char* to = static_cast<char*>(workspace) + GEMM_RELU_GROUPS_COUNTER_BYTES;
        // before the copies take its partial sums' place
        if (tiles_a && stream_a && ((rc = stream_rows()) != GEMM_RELU_OK || !want_b)) return rc;
        if (N % 2)
            rc = launch_pad(r.a, r.lda, c, M, to, dtype, s);
        else if (relu) {
            rc = launch_mask(d, c, masked, mn, dtype, s);
            r.a = masked;
            to += masked_bytes;
        }
        (kn ? w.q : w.p) = r.a;
        (kn ? w.ldq : w.ldp) = r.lda;
        if (want_b && K % 2 && rc == GEMM_RELU_OK) rc = launch_pad(kn ? w.p : w.q, kn ? w.ldp : w.ldq, nullptr, M, to, dtype, s);
        if (tiles_a && r.ldb % 2 && rc == GEMM_RELU_OK) rc = launch_pad(r.b, r.ldb, nullptr, groups * (kn ? K : N), to, dtype, s);
        const bool ready = dma_rows(r.a, r.lda) && (!tiles_a || dma_rows(r.b, r.ldb)) && (!want_b || (dma_rows(w.p, w.ldp) && dma_rows(w.q, w.ldq)));
        if (rc != GEMM_RELU_OK) return rc;
        if (!ready)                  // an even operand at an odd address
            return launch_grad_staged(r, w, nullptr, dtype, layout_a, config, cus, s);
        if (tiles_a) rc = launch_rows(r, AdapterArgs{}, dtype, layout_a, config, cus, nullptr, nullptr, s);
        w.c_vec = store_width(w.out, w.j);
        if (want_b && rc == GEMM_RELU_OK) rc = launch_weights(w, dtype, config, cus, s);
        return rc;
    }
    if (config == GEMM_RELU_GROUPS_TILED || !dma || (config == GEMM_RELU_GROUPS_AUTO && small_grad(M, N, K, groups)))
        return launch_grad_staged(r, w, c, dtype, layout_a, config, cus, s);
    if (relu) {
        rc = launch_mask(d, c, masked, mn, dtype, s);
        r.a = masked;
        (kn ? w.q : w.p) = masked;
    }
    if (tiles_a && rc == GEMM_RELU_OK) rc = launch_rows(r, AdapterArgs{}, dtype, layout_a, config, cus, nullptr, nullptr, s);
    w.c_vec = store_width(w.out, w.j);
    if (want_b && rc == GEMM_RELU_OK) rc = launch_weights(w, dtype, config, cus, s);
    return rc;
}

int64_t gemm_relu_adapters_workspace(int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters,
                                     int64_t segments, int dtype, int b_layout)
{
    const int rc = check_shape(M, N, K, segments, dtype, b_layout);
    if (rc != GEMM_RELU_OK) return rc;
    if (rank < 1 || adapters < 1) return GEMM_RELU_ERR_INVALID_ARG;
    if (rank > kMaxRank || adapters > kMaxGroups) return GEMM_RELU_ERR_TOO_LARGE;
    return adapter_space(M, N, K, rank, segments, b_layout).bytes;
}

int gemm_relu_adapters(const void* X, const void* W, const void* U, const void* V, const float* scales,
                       const int32_t* ends, const int32_t* ids, void* C, int64_t M, int64_t N, int64_t K,
                       int64_t rank, int64_t adapters, int64_t segments, int dtype, int b_layout, int relu,
                       int config_id, void* workspace, int64_t workspace_bytes, void* stream)
{
    const int64_t need = gemm_relu_adapters_workspace(M, N, K, rank, adapters, segments, dtype, b_layout);
    if (need < 0) return (int)need;
    if (relu != 0 && relu != 1) return GEMM_RELU_ERR_INVALID_ARG;
    if (!known_config(config_id)) return GEMM_RELU_ERR_BAD_CONFIG;
    if (M == 0 || N == 0) return GEMM_RELU_OK;
    const Span in[] = {{X, 2 * M * K}, {W, 2 * K * N}, {U, 2 * adapters * K * rank}, {V, 2 * adapters * rank * N}};
    const Span words[] = {{ends, 4 * segments}, {ids, 4 * segments}, {scales, 4 * adapters}};
    const Span out[] = {{C, 2 * M * N}, {workspace, need}};
    int rc = check_spans(in, 4, words, 3, out, 1);
    if (rc == GEMM_RELU_OK) rc = check_workspace(workspace, workspace_bytes, need);
    if (rc == GEMM_RELU_OK) rc = check_spans(in, 4, words, 3, out, 2);
    if (rc != GEMM_RELU_OK) return rc;
    int cus = 0;
    if ((rc = check_device(&cus)) != GEMM_RELU_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) return zero_fill(C, M * N, s);
    const AdapterSpace space = adapter_space(M, N, K, rank, segments, b_layout);
    char* const ws = static_cast<char*>(workspace);
    uint16_t* t = reinterpret_cast<uint16_t*>(ws + space.t);
    float* factor = reinterpret_cast<float*>(ws + space.factor);
    int* row_id = reinterpret_cast<int*>(ws + space.row_id);
    ShrinkArgs sh{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(U), scales, ends, ids, t, factor, row_id,
                  reinterpret_cast<float*>(ws + space.part), reinterpret_cast<int*>(ws), (int)M, (int)K, (int)segments,
                  (int)adapters, (int)rank, (int)space.rank_pad};
    void* args[] = {&sh};
    rc = enqueue(kernels(dtype).shrink[b_layout][rank > kShrinkCols][space.blocks - 1], dim3((unsigned)space.tiles, (unsigned)space.splits),
                 kShrinkThreads, args, s, (size_t)(ceil_div(rank, kShrinkCols) * space.blocks * kShrinkThreads * 4));
    if (rc != GEMM_RELU_OK) return rc;
    RowsArgs a{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(W), static_cast<uint16_t*>(C), nullptr,
               (int)M, (int)N, (int)K, 1, relu, (int)K, (int)(b_layout == GEMM_RELU_B_NK ? K : N), 0};
    const bool v_fast = b_layout == GEMM_RELU_B_NK ? rank % 8 == 0 && aligned(V, 16) : N % 4 == 0 && aligned(V, 8);
    AdapterArgs ad{static_cast<const uint16_t*>(V), t, factor, row_id, ends, ids, (int)segments, (int)adapters, (int)rank,
                   (int)space.rank_pad, v_fast};
    return launch_rows(a, ad, dtype, b_layout, config_id, cus, sh.part, sh.counters, s);
}

}  // extern "C"
