// C ABI of the 8-bit products scaled by blocks of 128 (gemm_relu_blocks.h):
// argument checks, kernel choice and launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_relu_blocks.h"
#include "blocks_table.hpp"
#include "checks.hpp"
#include "turns.hpp"

namespace gemm_relu_hip {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxPitch = int64_t(1) << 21;
constexpr int64_t kMaxGroups = 65535;

int64_t blocks_of(int64_t n) { return ceil_div(n, kBlock); }

bool known_format(int f) { return f == GEMM_RELU_E4M3 || f == GEMM_RELU_E5M2; }
bool known_form(int f) { return f == GEMM_RELU_SCALES_ROWS || f == GEMM_RELU_SCALES_TILES; }

int check_dims(std::initializer_list<int64_t> dims)
{
    for (int64_t d : dims)
        if (d < 0) return GEMM_RELU_ERR_INVALID_ARG;
    for (int64_t d : dims)
        if (d > kMaxDim) return GEMM_RELU_ERR_TOO_LARGE;
    return GEMM_RELU_OK;
}

// The pitch of an 8-bit matrix with rows of `row` bytes.
int check_pitch(int64_t ld, int64_t row)
{
    if (ld < row || ld % 16 != 0) return GEMM_RELU_ERR_MISALIGNED;
    return ld > kMaxPitch ? GEMM_RELU_ERR_TOO_LARGE : GEMM_RELU_OK;
}

// The bytes of an 8-bit matrix: its loads take whole 16-byte pieces, its stores do not.
int64_t read_bytes(int64_t rows, int64_t row, int64_t ld) { return rows && row ? (rows - 1) * ld + round_up(row, 16) : 0; }
int64_t written_bytes(int64_t rows, int64_t row, int64_t ld) { return rows && row ? (rows - 1) * ld + row : 0; }

const BlocksKernels& kernels(int format_a, int format_b)
{
    if (format_a == GEMM_RELU_E4M3) return format_b == GEMM_RELU_E4M3 ? blocks_kernels_e4m3_e4m3() : blocks_kernels_e4m3_e5m2();
    return format_b == GEMM_RELU_E4M3 ? blocks_kernels_e5m2_e4m3() : blocks_kernels_e5m2_e5m2();
}

int launch_quantize(QuantizeArgs a, int64_t count, int dtype, int format, int form, hipStream_t stream)
{
    a.tiles_r = (int)blocks_of(a.rows);
    a.tiles_c = (int)blocks_of(a.cols);
    const int vec = a.cols % 8 == 0 && aligned(a.x, 16) && (!a.mask || aligned(a.mask, 16));
    const int64_t tiles = count * a.tiles_r * a.tiles_c;
    if (!launchable(tiles, kQuantizeThreads)) return GEMM_RELU_ERR_TOO_LARGE;
    // Where tiles are few, a workgroup for each direction: both ways 1000 x 512 7.7 -> 5.9 us,
    // 2048 x 3000 (384 tiles) 11.8 -> 10.3; of 4096 x 2048 (512) 11.9 and 11.6, as tiles 11.2 and 11.8.
    a.apart = a.q && a.qt && tiles <= 384 ? (int)tiles : 0;
    void* args[] = {&a};
    return enqueue(quantize_kernel(dtype, format, form == GEMM_RELU_SCALES_TILES, vec), dim3((unsigned)(a.apart ? 2 * tiles : tiles)),
                   kQuantizeThreads, args, stream);
}

// Whether weights of so many bytes are streamed past the caches.  From memory they come
// faster so, from the cache beside it (256 MB) slower, and a model's layers take turns in
// that.  us through the caches and past them, of weights from memory / that stay in the
// cache from the call before:
//   64 MB   few rows x 8192 x 8192           18.0 16.5 / 12.7 16.9
//   96      16 rows x 12288 x 8192           21.9 20.5 / 17.2 18.9
//  128      16 rows x 16384 x 8192           26.8 23.7 / 21.6 23.2
//           64 rows x 16384 x 8192           33.9 31.8 / 25.1 32.7
//           1024 in 32 groups, 2048 x 2048   34.2 29.1 / 25.5 30.0
//  192      16 rows x 24576 x 8192           44.1 40.8 / 32.6 41.0
//           2048 in 24 groups, 4096 x 2048   69.5 47.5 / 61.2 48.8
//  234      16 rows x 30000 x 8192           49.7 45.1 / 38.2 41.2
// Weights of 64 MB lose too much where several layers' stay there together.
constexpr int64_t kStreamOnce = int64_t(96) << 20;

// Tiles of `tile` x `tile` that a product can have: whole ones, and a partial one for each group.
int64_t most_tiles(const BlocksArgs& a, int64_t tile)
{
    return std::min<int64_t>(a.m, a.m / tile + a.groups) * ceil_div(a.n, tile);
}

// Which kernel a product takes: a tile, or GEMM_RELU_BLOCKS_STREAM and which of the
// streaming kernels (by kStreamRows).
//  Streaming kernels by the workgroups they make: more rows a workgroup read the weights
// fewer times, but some 200 workgroups are needed to fill the device; 8 waves where one
// workgroup a CU is all there is, 4 where several share one.  Measured, us, kernels of
// 16 rows x 32 (8 waves) / 16 x 64 (8) / 16 x 64 (4) / 32 x 64 (8) / 32 x 64 (4) / 64 x 64 (8),
// then the 64 x 64 tile and the 128 tile:
//   1 row, 4096 x 4096             8.1 /  9.2 / 11.7 /  9.7 / 12.3 / 11.5     14.7  23.9
//   1 row, 1024 x 8192             9.4 / 11.2 / 14.2 / 12.7 / 18.2 / 15.8     22.8  40.9
//   16 rows, 16384 x 8192         34.2 / 29.2 / 32.6 / 29.7 / 33.3 / 30.3     36.1  45.6
//   32 rows, 16384 x 8192         53.8 / 48.0 / 35.0 / 30.5 / 34.7 / 31.0     36.3  46.4
//   64 rows, 16384 x 8192         90.2 / 83.8 / 68.4 / 49.5 / 40.4 / 34.6     37.3  48.7
//   64 rows, 4096 x 4096          13.4 /  9.5 / 12.2 / 11.0 / 13.3 / 14.3     15.0  25.3
//   256, 1024 x 1024               9.5 /  6.9 /  7.0 /  7.8 /  8.1 /  9.4      8.6  12.0
//   512, 1024 x 1024              15.7 / 10.7 /  8.1 /  7.9 /  8.3 /  9.5      8.7  12.2
//   512, 2048 x 2048              31.8 / 20.9 / 16.4 / 14.4 / 12.0 / 11.7     11.3  17.8
//   1024, 1024 x 1024             27.9 / 17.9 / 12.1 / 12.4 /  9.8 / 10.1      8.8  12.4
//   64 in 64 groups, 2048 x 2048  78.5 / 60.8 / 50.4 / 62.7 / 49.5 / 66.5     58.3  53.2
//   256 in 32, 1024 x 1024        19.9 / 14.4 / 11.1 / 14.4 / 11.5 / 15.3     11.7  12.3
//   512 in 8, 2048 x 2048         33.8 / 22.6 / 17.5 / 17.5 / 13.9 / 15.5     11.7  17.6
//  More than 32 rows and more than one workgroup a CU: tiles of 64, us streaming and so
// (64 rows): 65536 x 1024 30.0 / 16.8, 32768 x 2048 20.2 / 15.6, 24576 x 8192 54.6 / 50.4,
// 17000 x 1024 14.4 / 10.3; at one a CU the longer sums stream, 64 rows and 40, us streaming
// and in tiles of 64: 16384 x 4096 16.0 / 15.2, x 6144 26.1 / 27.0 and 22.9 / 26.3, x 8192 30.9 /
// 32.6 and 27.0 / 34.0, x 16384 58.8 / 61.8 and 47.7 / 61.8, 12300 x 8192 30.8 / 30.6, x 16384
// 52.3 / 58.9.  Groups of up to 32 rows likewise, 8 groups x 8192 x 512 13.5 / 11.2,
// 16 x 1024 x 2048 11.6 / 10.0, 8 x 1024 x 4096 10.8 / 14.5.
//  Groups of few rows with weights from memory: the deepest ring reads them fastest where
// its units go round three times, us streaming, tiles of 64 and of 128 (32 rows a group):
// 64 x 2048 x 4096 115 / 107 / 102, 16 x 16384 x 4096 217 / 212 / 198, 16 x 4096 x 4096
// 59.8 / 50.9 / 50.7, 32 x 2048 x 2048 30.9 / 26.8 / 30.0.
// Tiles: the largest whose tiles are mostly full and numerous enough to occupy the CUs.
//  (Most of these were measured with scales multiplied as they are.  Splitting them adds 1 to
// 10% to tiles of 64, 3 to 6% to those of 128 and 256 and 0 to 6% to streams; what a rule takes
// is the faster side still, or within 4% of it: 64 x 4096 x 4096 8.2 streaming / 15.7 / -, 512 x 1024 x 1024 5.9 / 7.6,
// 512 x 2048 x 2048 10.4 / 10.8 / 16.1, 1024 x 1024 x 1024 7.7 / 7.8 / 11.2, 512 in 8 groups
// x 2048 x 2048 12.0 / 11.0, 64 x 65536 x 1024 28.0 / 17.0.)
struct BlocksChoice {
    int config, stream = -1;
    BlocksChoice(int64_t m, int64_t n, int64_t k, int64_t groups, bool dense, bool heavy)
    {
        const int64_t used = std::min(groups, m), rows = m / used;
        const auto tiles = [&](int64_t r, int64_t c) { return used * ceil_div(rows, r) * ceil_div(n, c); };
        if (dense) {
            const int64_t by16 = tiles(16, 64), by32 = tiles(32, 64), by64 = tiles(64, 64);
            if (rows > 32 && by64 >= 192) stream = rows <= 64 && by64 <= 256 && k > 4096 ? 5 : -1;
            else if (rows > 16 && by32 >= 192) stream = by32 <= 384 ? 3 : 4;
            else stream = by16 < 192 ? 0 : by16 <= 384 ? 1 : 2;
        } else if (rows <= 32 && !heavy) {
            const int64_t most = rows + rows / 2 + 6;         // few groups have more rows
            const int64_t by16 = tiles(16, 64);
            if (most <= 16) stream = by16 < 192 ? 0 : by16 <= 384 ? 1 : by16 <= 512 ? 2 : -1;
            else if (tiles(32, 64) < 256) stream = 3;
        }
        config = stream >= 0                                                         ? GEMM_RELU_BLOCKS_STREAM
                 : rows >= 192 && tiles(256, 256) >= 192                             ? GEMM_RELU_BLOCKS_256
                 : rows >= 96 && tiles(128, 128) >= 128                              ? GEMM_RELU_BLOCKS_128
                 : !dense && heavy && tiles(128, 128) >= 768                         ? GEMM_RELU_BLOCKS_128
                                                                                     : GEMM_RELU_BLOCKS_64;
        if (stream < 0) stream = rows <= 16 ? 2 : 4;       // on request
    }
};

// A product (M, N, K > 0).
int launch_blocks(BlocksArgs a, int format_a, int format_b, int form_b, int config, int cus, hipStream_t stream)
{
    a.c_vec = a.n % 8 == 0 && aligned(a.c, 16);
    const int rows_b = form_b == GEMM_RELU_SCALES_ROWS;
    const bool heavy = (int64_t)std::min(a.groups, a.m) * a.n * a.ldb >= kStreamOnce;
    const BlocksChoice choice(a.m, a.n, a.k, a.groups, !a.ends, heavy);
    if (config == GEMM_RELU_BLOCKS_AUTO) config = choice.config;
    void* args[] = {&a};
    if (config == GEMM_RELU_BLOCKS_STREAM) {
        const int kind = choice.stream, r = 16 * kStreamRows[kind], threads = 64 * kStreamWaves[kind];
        // row tiles: whole ones, a partial one of each group, and those of no group's rows
        const int64_t tiles = a.ends ? std::min<int64_t>(a.m, a.m / r + a.groups + 1) : ceil_div(a.m, r);
        const int64_t units = tiles * ceil_div(a.n, 16 * kStreamCols[kind]);
        a.once = heavy;
        if (launchable(units, threads))
            return enqueue(kernels(format_a, format_b).stream[kind][rows_b], dim3((unsigned)units), threads, args, stream);
        config = GEMM_RELU_BLOCKS_64;
    }
    // Rows that make a tile or two a group read their weights about once (one product of 1024 rows
    // x 4096 x 4096 would take 27 instead of 25.5 us).
    a.once = heavy && (a.ends || a.m <= kBlockTile[config]) && config != GEMM_RELU_BLOCKS_256;
    const int64_t tiles = most_tiles(a, kBlockTile[config]);
    if (tiles > INT32_MAX) return GEMM_RELU_ERR_TOO_LARGE;
    const int64_t grid = std::min<int64_t>(tiles, config == GEMM_RELU_BLOCKS_64 ? 2 * cus : cus);
    return enqueue(kernels(format_a, format_b).tile[config][rows_b], dim3((unsigned)grid), kBlockThreads[config], args, stream);
}

// Both gradients' products in one launch of tiles of 64, where each alone leaves the
// device waiting: few tiles, and no long sum over few of them (which the streaming
// kernels cut over waves).  Measured, us of the backward pass with two launches and with one:
//   M x N x K     1000 x 517 x 1101    512 x 1500 x 1500   2048 x 2048 x 1024   1 x 1024 x 1024
//                 28.7 / 22.6          33.5 / 25.6         51.7 / 41.0          14.9 / 14.4
//   more tiles    512 x 2048 x 2048    28.6 / 30.4         16 x 2048 x 2048     18.9 / 20.0
//   long sums     2048 x 512 x 512     17.9 / 19.5         8192 x 512 x 512     32.6 / 48.7
bool pair_fits(const BlocksArgs (&p)[2], int cus)
{
    const int64_t tiles[2] = {most_tiles(p[0], 64), most_tiles(p[1], 64)};
    for (int i = 0; i < 2; ++i)
        if (p[i].k > 1024 && tiles[i] < cus) return false;
    return tiles[0] + tiles[1] <= 4 * cus;
}

int launch_pair(BlocksPair p, int format_a, int format_b, hipStream_t stream)
{
    for (int i = 0; i < 2; ++i) {
        p.product[i].c_vec = p.product[i].n % 8 == 0 && aligned(p.product[i].c, 16);
        p.blocks[i] = (int)round_up(most_tiles(p.product[i], 64), 8);        // (whole rounds of XCDs)
    }
    void* args[] = {&p};
    return enqueue(kernels(format_a, format_b).pair, dim3((unsigned)(p.blocks[0] + p.blocks[1])), kBlockThreads[GEMM_RELU_BLOCKS_64],
                   args, stream);
}

// Places in the backward pass's workspace.
struct BackwardSpace {
    int64_t q, s, qt, st, bytes, ldq, ldqt;
    BackwardSpace(int64_t m, int64_t n)
    {
        // long rows start at whole cache lines, so that no piece of 128 bytes lies in two
        ldq = round_up(n, n <= 1024 ? 16 : 128);
        ldqt = round_up(m, m <= 1024 ? 16 : 128);
        q = GEMM_RELU_GROUPS_COUNTER_BYTES;
        s = q + round_up(m * ldq, 256);
        qt = s + round_up(4 * m * blocks_of(n), 256);
        st = qt + round_up(n * ldqt, 256);
        bytes = st + round_up(4 * n * blocks_of(m), 256);
    }
};

// The expert layer: kinds of workgroups, parts of its second product's K, and places in
// the workspace.
//  8 waves for few units, where one workgroup a CU is all there is; 4, and 64 columns, for
// many.  Measured, us a layer with 8 waves and with 4 (tokens x top of experts, K = N x hidden;
// units of 64 columns):
//   1 x 4 of 64,  2048 x 2048     128    24.8 /  26.8        8-bit  4 x 2 of 16, 1024 x 1024   128    17.4 /  20.6
//   1 x 2 of 8,   4096 x 4096     128    33.0 /  35.8        8-bit  8 x 2 of 32, 2048 x 2048   544    46.4 /  36.8
//   4 x 2 of 16,  1024 x 1024     128    19.1 /  21.1        8-bit 24 x 4 of 64                4480   213  / 171
//   2 x 4 of 64,  2048 x 2048     256    45.4 /  38.0        (K, N)  4 x 2 of 16, 1024 x 1024  128    20.3 /  20.6
//   8 x 2 of 32,  1024 x 1024     272    33.3 /  25.8        (K, N)  8 x 2 of 32, 1024 x 1024  272    25.7 /  25.5
//  16 x 4 of 64,  2048 x 2048    2176     157 / 122          (K, N) 16 x 2 of 32, 2048 x 2048  1088   99.8 /  86.6
//  The second product's K is cut where its units leave CUs without work: 1 x 1 of 8,
// 512 x 8192, 23.5 us whole and 17.7 in 8 parts; 1 x 2 of 8, 1024 x 4096, 21.0 and 20.5.
struct ExpertsSpace {
    int kind1, kind2;      // index into kExpertBlocks
    int64_t units1, units2, splits, mid_row, mid, part, part_bytes, bytes;
    ExpertsSpace(int64_t tokens, int64_t n, int64_t hidden, int64_t experts, int64_t top, int b_layout)
    {
        const int64_t slots = tokens * top, used = std::min(experts, slots);
        const auto columns = [&](int kind) { return int64_t(16) * (b_layout == GEMM_RELU_B_KN ? 4 : kExpertBlocks[kind]); };
        const auto kind = [&](int64_t out) {
            if (ceil_div(out, 32) > kMaxColumnBlocks) return 1;
            return (used + slots / kExpertRows) * ceil_div(out, 64) <= (b_layout == GEMM_RELU_B_KN ? 384 : 160) ? 0 : 1;
        };
        // row tiles: one for each expert that has rows, and one more for every 16 of them
        const auto units = [&](int64_t out, int kind) { return (used + slots / kExpertRows) * ceil_div(out, columns(kind)); };
        kind1 = kind(hidden);
        kind2 = kind(n);
        units1 = units(hidden, kind1);
        units2 = units(n, kind2);
        const int64_t least = std::max<int64_t>(1, used * ceil_div(n, columns(kind2)));
        splits = std::max<int64_t>(1, std::min<int64_t>(256 / least, blocks_of(hidden) / kBlocksAPart));
        mid_row = round_up(hidden, 8);
        mid = GEMM_RELU_GROUPS_COUNTER_BYTES;
        part = mid + round_up(4 * slots * mid_row, 256);
        part_bytes = 4 * slots * splits * n;
        bytes = part + round_up(part_bytes, 256);
    }
    // A counter for each column block; scale blocks of K for the waves of each part.
    static constexpr int64_t kMaxColumnBlocks = GEMM_RELU_GROUPS_COUNTER_BYTES / 4, kBlocksAPart = 8;
};
static_assert(((int64_t(1) << 20) + 63) / 64 <= ExpertsSpace::kMaxColumnBlocks, "a counter for each block of 64 columns");

// Every workgroup of the first product makes the choices for itself, unless that costs it more
// than a launch: a choice takes a wave about 0.1 us, for more than 64 experts longer.  Measured,
// us a layer without and with a launch for them: 8 tokens x 4 of 64 21.9 / 23.5, 16 x 4 of 64
// 26.3 / 27.5, 8 x 4 of 256 24.8 / 25.1; 17 x 4 of 64 30.8 / 29.8, 64 x 4 of 64 50.6 / 43.0,
// 16 x 8 of 256 34.5 / 29.5, 4 x 8 of 1024 39.1 / 34.4.
bool route_apart(int64_t tokens, int64_t experts, int64_t top) { return tokens > 16 || tokens * top * ceil_div(experts, 64) > 128; }

int check_experts(int64_t tokens, int64_t n, int64_t hidden, int64_t experts, int64_t top, int b_layout)
{
    if (b_layout != GEMM_RELU_B_KN && b_layout != GEMM_RELU_B_NK) return GEMM_RELU_ERR_BAD_LAYOUT;
    const int rc = check_dims({tokens, n, hidden});
    if (rc != GEMM_RELU_OK) return rc;
    if (experts < 1 || top < 1 || top > experts) return GEMM_RELU_ERR_INVALID_ARG;
    if (tokens > kMaxTokens || experts > kMaxExperts || top > kMaxTop) return GEMM_RELU_ERR_TOO_LARGE;
    // the intermediate and the partial sums have one descriptor each
    if (4 * tokens * top * round_up(hidden, 8) > INT32_MAX) return GEMM_RELU_ERR_TOO_LARGE;
    return tokens > 0 && ExpertsSpace(tokens, n, hidden, experts, top, b_layout).part_bytes > INT32_MAX ? GEMM_RELU_ERR_TOO_LARGE : GEMM_RELU_OK;
}

}  // namespace
}  // namespace gemm_relu_hip

using namespace gemm_relu_hip;

extern "C" {

int gemm_relu_quantize_blocks(const void* X, const void* mask, void* Q, float* scales, void* QT, float* scales_t,
                              int64_t count, int64_t R, int64_t C, int64_t ldq, int64_t ldqt, int dtype, int format,
                              int form, int power_of_two, void* stream)
{
    if (dtype != GEMM_RELU_F16 && dtype != GEMM_RELU_BF16) return GEMM_RELU_ERR_BAD_DTYPE;
    if (!known_format(format)) return GEMM_RELU_ERR_BAD_DTYPE;
    if (!known_form(form)) return GEMM_RELU_ERR_BAD_LAYOUT;
    if (power_of_two != 0 && power_of_two != 1) return GEMM_RELU_ERR_INVALID_ARG;
    int rc = check_dims({count, R, C});
    if (rc != GEMM_RELU_OK) return rc;
    if (count > kMaxGroups) return GEMM_RELU_ERR_TOO_LARGE;
    if (!Q && !QT) return GEMM_RELU_ERR_INVALID_ARG;
    if (Q && (rc = check_pitch(ldq, C)) != GEMM_RELU_OK) return rc;
    if (QT && (rc = check_pitch(ldqt, R)) != GEMM_RELU_OK) return rc;
    if (count == 0 || R == 0 || C == 0) return GEMM_RELU_OK;
    const bool tiles = form == GEMM_RELU_SCALES_TILES;
    const int64_t elements = count * R * C, n_tiles = count * blocks_of(R) * blocks_of(C);
    const Span in[] = {{X, 2 * elements}, {mask, mask ? 2 * elements : 0}};
    const Span out[] = {{Q, Q ? written_bytes(count * R, C, ldq) : 0}, {QT, QT ? written_bytes(count * C, R, ldqt) : 0},
                        {scales, !Q ? 0 : 4 * (tiles ? n_tiles : count * R * blocks_of(C))},
                        {scales_t, !QT ? 0 : 4 * (tiles ? n_tiles : count * C * blocks_of(R))}};
    if ((rc = check_spans(in, 2, nullptr, 0, out, 4)) != GEMM_RELU_OK) return rc;
    if ((Q && !aligned(Q, 16)) || (QT && !aligned(QT, 16)) || (Q && !aligned(scales, 4)) || (QT && !aligned(scales_t, 4)))
        return GEMM_RELU_ERR_MISALIGNED;
    int cus = 0;
    if ((rc = check_device(&cus)) != GEMM_RELU_OK) return rc;
    QuantizeArgs a{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(mask), static_cast<uint8_t*>(Q), scales,
                   static_cast<uint8_t*>(QT), scales_t, (int)R, (int)C, 0, 0, ldq, ldqt, power_of_two, 0};
    return launch_quantize(a, count, dtype, format, form, static_cast<hipStream_t>(stream));
}

int gemm_relu_blocks(const void* A, const float* scales_a, const void* B, const float* scales_b, const int32_t* ends,
                     void* C, int64_t M, int64_t N, int64_t K, int64_t groups, int64_t lda, int64_t ldb, int format_a,
                     int format_b, int form_b, int dtype, int relu, int config_id, void* stream)
{
    if (dtype != GEMM_RELU_F16 && dtype != GEMM_RELU_BF16) return GEMM_RELU_ERR_BAD_DTYPE;
    if (!known_format(format_a) || !known_format(format_b)) return GEMM_RELU_ERR_BAD_DTYPE;
    if (!known_form(form_b)) return GEMM_RELU_ERR_BAD_LAYOUT;
    int rc = check_dims({M, N, K});
    if (rc != GEMM_RELU_OK) return rc;
    if (groups > kMaxGroups) return GEMM_RELU_ERR_TOO_LARGE;
    if (groups < 1 || (relu != 0 && relu != 1) || (!ends && groups != 1)) return GEMM_RELU_ERR_INVALID_ARG;
    if (config_id < GEMM_RELU_BLOCKS_AUTO || config_id > GEMM_RELU_BLOCKS_STREAM) return GEMM_RELU_ERR_BAD_CONFIG;
    rc = check_pitch(lda, K);
    if (rc == GEMM_RELU_OK) rc = check_pitch(ldb, K);
    if (rc != GEMM_RELU_OK) return rc;
    if (M == 0 || N == 0) return GEMM_RELU_OK;
    const int64_t kb = blocks_of(K);
    const Span in[] = {{A, read_bytes(M, K, lda)}, {B, read_bytes(groups * N, K, ldb)}};
    const Span words[] = {{scales_a, 4 * M * kb},
                          {scales_b, 4 * groups * kb * (form_b == GEMM_RELU_SCALES_ROWS ? N : blocks_of(N))},
                          {ends, ends ? 4 * groups : 0}};
    const Span out[] = {{C, 2 * M * N}};
    rc = check_spans(in, 2, words, 3, out, 1);
    if (rc == GEMM_RELU_OK && K > 0 && (!aligned(A, 16) || !aligned(B, 16))) rc = GEMM_RELU_ERR_MISALIGNED;
    if (rc != GEMM_RELU_OK) return rc;
    int cus = 0;
    if ((rc = check_device(&cus)) != GEMM_RELU_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) return zero_fill(C, M * N, s);
    BlocksArgs a{static_cast<const uint8_t*>(A), scales_a, static_cast<const uint8_t*>(B), scales_b, static_cast<uint16_t*>(C),
                 ends, (int)M, (int)N, (int)K, (int)groups, (uint32_t)lda, (uint32_t)ldb, relu, dtype == GEMM_RELU_BF16, 0, 0};
    return launch_blocks(a, format_a, format_b, form_b, config_id, cus, s);
}

int64_t gemm_relu_blocks_backward_workspace(int64_t M, int64_t N, int64_t K)
{
    const int rc = check_dims({M, N, K});
    return rc != GEMM_RELU_OK ? rc : BackwardSpace(M, N).bytes;
}

int gemm_relu_blocks_backward(const void* dC, const void* C, const void* XT, const float* scales_xt, const void* WT,
                              const float* scales_wt, void* dX, void* dW, int64_t M, int64_t N, int64_t K, int64_t ldxt,
                              int64_t ldwt, int format, int format_x, int format_w, int dtype, int relu, void* workspace,
                              int64_t workspace_bytes, void* stream)
{
    if (dtype != GEMM_RELU_F16 && dtype != GEMM_RELU_BF16) return GEMM_RELU_ERR_BAD_DTYPE;
    if (!known_format(format) || !known_format(format_x) || !known_format(format_w)) return GEMM_RELU_ERR_BAD_DTYPE;
    const int64_t need = gemm_relu_blocks_backward_workspace(M, N, K);
    if (need < 0) return (int)need;
    if (relu != 0 && relu != 1) return GEMM_RELU_ERR_INVALID_ARG;
    const bool want_x = dX != nullptr, want_w = dW != nullptr;
    if (!want_x && !want_w && K > 0) return GEMM_RELU_ERR_INVALID_ARG;
    int rc = want_w ? check_pitch(ldxt, M) : GEMM_RELU_OK;
    if (rc == GEMM_RELU_OK && want_x) rc = check_pitch(ldwt, N);
    if (rc != GEMM_RELU_OK) return rc;
    if (K == 0) return GEMM_RELU_OK;                 // both gradients are empty
    const int64_t mn = M * N;
    const Span in[] = {{dC, 2 * mn}, {relu ? C : nullptr, relu ? 2 * mn : 0}, {want_w ? XT : nullptr, want_w ? read_bytes(K, M, ldxt) : 0},
                       {want_x ? WT : nullptr, want_x ? read_bytes(K, N, ldwt) : 0}};
    const Span words[] = {{want_w ? scales_xt : nullptr, want_w ? 4 * K * blocks_of(M) : 0},
                          {want_x ? scales_wt : nullptr, want_x ? 4 * blocks_of(K) * blocks_of(N) : 0}};
    const Span out[] = {{dX, want_x ? 2 * M * K : 0}, {dW, want_w ? 2 * N * K : 0}, {workspace, need}};
    rc = check_spans(in, 4, words, 2, out, 2);
    if (rc == GEMM_RELU_OK && mn > 0 && ((want_w && !aligned(XT, 16)) || (want_x && !aligned(WT, 16)))) rc = GEMM_RELU_ERR_MISALIGNED;
    if (rc == GEMM_RELU_OK) rc = check_workspace(workspace, workspace_bytes, need);
    if (rc == GEMM_RELU_OK) rc = check_spans(in, 4, words, 2, out, 3);
    if (rc != GEMM_RELU_OK) return rc;
    int cus = 0;
    if ((rc = check_device(&cus)) != GEMM_RELU_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (mn == 0) {                                   // empty sums
        if (want_x) rc = zero_fill(dX, M * K, s);
        if (want_w && rc == GEMM_RELU_OK) rc = zero_fill(dW, N * K, s);
        return rc;
    }
    const WorkspaceTurn turn(workspace);
    const BackwardSpace space(M, N);
    char* const ws = static_cast<char*>(workspace);
    uint8_t *q = reinterpret_cast<uint8_t*>(ws + space.q), *qt = reinterpret_cast<uint8_t*>(ws + space.qt);
    float *sq = reinterpret_cast<float*>(ws + space.s), *st = reinterpret_cast<float*>(ws + space.st);
    QuantizeArgs d{static_cast<const uint16_t*>(dC), relu ? static_cast<const uint16_t*>(C) : nullptr, want_x ? q : nullptr, sq,
                   want_w ? qt : nullptr, st, (int)M, (int)N, 0, 0, space.ldq, space.ldqt, 0, 0};
    rc = launch_quantize(d, 1, dtype, format, GEMM_RELU_SCALES_ROWS, s);
    const int bf16 = dtype == GEMM_RELU_BF16;
    const BlocksPair both{{{q, sq, static_cast<const uint8_t*>(WT), scales_wt, static_cast<uint16_t*>(dX), nullptr, (int)M, (int)K, (int)N, 1,
                            (uint32_t)space.ldq, (uint32_t)ldwt, 0, bf16, 0, 0},
                           {qt, st, static_cast<const uint8_t*>(XT), scales_xt, static_cast<uint16_t*>(dW), nullptr, (int)N, (int)K, (int)M, 1,
                            (uint32_t)space.ldqt, (uint32_t)ldxt, 0, bf16, 0}},
                          {}};
    // One gradient alone takes the same tiles, so that its bits do not depend on what else is asked for.
    const bool fits = pair_fits(both.product, cus);
    if (rc == GEMM_RELU_OK && fits && want_x && want_w && format_x == format_w) return launch_pair(both, format, format_x, s);
    const int config = fits ? GEMM_RELU_BLOCKS_64 : GEMM_RELU_BLOCKS_AUTO;
    if (want_x && rc == GEMM_RELU_OK) rc = launch_blocks(both.product[0], format, format_w, GEMM_RELU_SCALES_TILES, config, cus, s);
    if (want_w && rc == GEMM_RELU_OK) rc = launch_blocks(both.product[1], format, format_x, GEMM_RELU_SCALES_ROWS, config, cus, s);
    return rc;
}

int64_t gemm_relu_experts_workspace(int64_t tokens, int64_t N, int64_t hidden, int64_t experts, int64_t top, int b_layout)
{
    const int rc = check_experts(tokens, N, hidden, experts, top, b_layout);
    return rc != GEMM_RELU_OK ? rc : ExpertsSpace(tokens, N, hidden, experts, top, b_layout).bytes;
}

int gemm_relu_experts(const void* X, const void* W1, const float* scales1, const void* W2, const float* scales2,
                      const float* logits, int32_t* ids, float* weights, void* Y, int64_t tokens, int64_t N,
                      int64_t K, int64_t hidden, int64_t experts, int64_t top, int64_t ld1, int64_t ld2, int renormalize,
                      int dtype, int format, int b_layout, void* workspace, int64_t workspace_bytes, void* stream)
{
    if (dtype != GEMM_RELU_F16 && dtype != GEMM_RELU_BF16) return GEMM_RELU_ERR_BAD_DTYPE;
    if (format != -1 && !known_format(format)) return GEMM_RELU_ERR_BAD_DTYPE;
    const int64_t need = gemm_relu_experts_workspace(tokens, N, hidden, experts, top, b_layout);
    if (need < 0) return (int)need;
    int rc = check_dims({K});
    if (rc != GEMM_RELU_OK) return rc;
    if (renormalize != 0 && renormalize != 1) return GEMM_RELU_ERR_INVALID_ARG;
    const bool bytes = format != -1, kn = b_layout == GEMM_RELU_B_KN;
    if (bytes) {
        if (kn) return GEMM_RELU_ERR_BAD_LAYOUT;
        if ((rc = check_pitch(ld1, K)) != GEMM_RELU_OK || (rc = check_pitch(ld2, hidden)) != GEMM_RELU_OK) return rc;
    }
    if (tokens == 0) return GEMM_RELU_OK;
    const int64_t slots = tokens * top;
    const Span in[] = {{X, 2 * tokens * K},
                       {W1, bytes ? read_bytes(experts * hidden, K, ld1) : 2 * experts * hidden * K},
                       {W2, bytes ? read_bytes(experts * N, hidden, ld2) : 2 * experts * N * hidden}};
    const Span words[] = {{logits, logits ? 4 * tokens * experts : 0},
                          {bytes ? scales1 : nullptr, bytes ? 4 * experts * blocks_of(hidden) * blocks_of(K) : 0},
                          {bytes ? scales2 : nullptr, bytes ? 4 * experts * blocks_of(N) * blocks_of(hidden) : 0},
                          {ids, 4 * slots},
                          {weights, 4 * slots}};
    const Span out[] = {{Y, 2 * tokens * N}, {ids, 4 * slots}, {weights, 4 * slots}, {workspace, need}};
    // (ids and weights are inputs without logits: then only Y and the workspace are written)
    const Span written[] = {out[0], out[3]};
    rc = check_spans(in, 3, words, 5, out, 1);
    if (rc == GEMM_RELU_OK && logits) rc = check_spans(in, 3, words, 3, out, 3);
    if (rc == GEMM_RELU_OK && bytes && ((in[1].bytes && !aligned(W1, 16)) || (in[2].bytes && !aligned(W2, 16)))) rc = GEMM_RELU_ERR_MISALIGNED;
    if (rc == GEMM_RELU_OK) rc = check_workspace(workspace, workspace_bytes, need);
    if (rc == GEMM_RELU_OK) rc = check_spans(in, 3, words, 5, written, 2);
    if (rc != GEMM_RELU_OK) return rc;
    int cus = 0;
    if ((rc = check_device(&cus)) != GEMM_RELU_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const WorkspaceTurn turn(workspace);
    const ExpertsSpace space(tokens, N, hidden, experts, top, b_layout);
    char* const ws = static_cast<char*>(workspace);
    const int store = bytes ? 2 + format : kn ? 1 : 0;
    const ExpertsKernels& kernels = dtype == GEMM_RELU_F16 ? experts_kernels_f16() : experts_kernels_bf16();
    const auto even = [](const void* p, int64_t row) { return row % 2 == 0 && aligned(p, 4); };
    ExpertsArgs a{};
    a.x = static_cast<const uint16_t*>(X);
    a.w = static_cast<const uint8_t*>(W1);
    a.scales = scales1;
    a.logits = logits;
    a.ids = ids;
    a.weights = weights;
    a.mid = reinterpret_cast<uint16_t*>(ws + space.mid);
    a.part = reinterpret_cast<float*>(ws + space.part);
    a.counters = reinterpret_cast<int*>(ws);
    a.y = static_cast<uint16_t*>(Y);
    a.ld = bytes ? ld1 : 2 * (kn ? hidden : K);
    a.tokens = (int)tokens;
    a.in = (int)K;
    a.out = (int)hidden;
    a.experts = (int)experts;
    a.top = (int)top;
    a.mid_row = (int)space.mid_row;
    a.renormalize = renormalize;
    a.routed = logits != nullptr;
    a.splits = 1;
    void* args[] = {&a};
    // As many workgroups as run at once.
    const auto launch = [&](int odd, int second, int kind, int64_t units) {
        const int64_t room = (kind == 0 ? 2 : 3) * cus;
        a.once = std::min(experts, slots) * (kn ? a.in : a.out) * a.ld >= kStreamOnce;
        return enqueue(kernels.products[store][odd][second][kind], dim3((unsigned)std::max<int64_t>(1, std::min(units, room))),
                       64 * kExpertWaves[kind], args, s, (size_t)route_table_bytes(slots, experts));
    };
    const bool odd1 = !even(X, K) || (!bytes && !(kn ? even(W1, hidden) : even(W1, K)));
    if (logits && route_apart(tokens, experts, top)) {
        rc = enqueue(kernels.route, dim3((unsigned)tokens), 64, args, s);
        if (rc != GEMM_RELU_OK) return rc;
        a.logits = nullptr;
    }
    rc = launch(odd1, 0, space.kind1, space.units1);
    if (rc != GEMM_RELU_OK || N == 0) return rc;
    a.x = a.mid;
    a.w = static_cast<const uint8_t*>(W2);
    a.scales = scales2;
    a.logits = nullptr;              // the first launch has written its choices
    a.ld = bytes ? ld2 : 2 * (kn ? N : hidden);
    a.in = (int)hidden;
    a.out = (int)N;
    a.splits = (int)space.splits;
    const bool odd2 = !bytes && !(kn ? even(W2, N) : even(W2, hidden));
    return launch(odd2, 1, space.kind2, space.units2 * space.splits);
}

}  // extern "C"
