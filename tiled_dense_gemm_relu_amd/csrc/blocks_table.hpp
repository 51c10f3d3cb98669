// Kernel arguments and the host-side table of kernel instances of the 8-bit
// products scaled by blocks of 128 and of the expert layer for a few tokens
// (gemm_relu_blocks.h), filled by the blocks_*.hip translation units and read by
// blocks_api.hip.
#pragma once

#include <stdint.h>

namespace gemm_relu_hip {

constexpr int kBlock = 128;

// Formats of 8-bit matrices (GEMM_RELU_E4M3, _E5M2; the matrix instructions' codes).
enum { kE4M3 = 0, kE5M2 = 1 };

// One launch quantizes both ways; q or qt may be nullptr.
struct QuantizeArgs {
    const uint16_t* x;
    const uint16_t* mask;  // nullptr: none
    uint8_t* q;
    float* s;
    uint8_t* qt;
    float* st;
    int rows, cols, tiles_r, tiles_c;
    int64_t ldq, ldqt;
    int power_of_two;
    int apart;             // > 0: so many workgroups write q, and as many after them qt
};
constexpr int kQuantizeThreads = 256;

// C = act(A @ B^T) over groups of rows; ends == nullptr: all rows are group 0.
struct BlocksArgs {
    const uint8_t* a;      // (M, lda)
    const float* sa;       // (K blocks, M)
    const uint8_t* b;      // (groups, N, ldb)
    const float* sb;       // (groups, K blocks, N) or (groups, N blocks, K blocks)
    uint16_t* c;           // (M, N)
    const int* ends;
    int m, n, k, groups;
    uint32_t lda, ldb;
    int relu, bf16;
    int c_vec;             // rows of C allow 16-byte stores
    int once;              // all tiles but 256: the weights do not stay in the caches
};

// Two products of small size in one launch of tiles of 64: workgroups of each.
struct BlocksPair {
    BlocksArgs product[2];
    int blocks[2];
};

constexpr int kNumBlockTiles = 3;
constexpr int kBlockTile[kNumBlockTiles] = {256, 128, 64};
constexpr int kBlockThreads[kNumBlockTiles] = {512, 512, 512};

// Streaming kernels: 16-row blocks and 16-column blocks of a workgroup, its waves and
// the scale blocks that each wave's ring holds.
constexpr int kNumStreams = 6;
constexpr int kStreamRows[kNumStreams] = {1, 1, 1, 2, 2, 4}, kStreamCols[kNumStreams] = {2, 4, 4, 4, 4, 4};
constexpr int kStreamWaves[kNumStreams] = {8, 8, 4, 8, 4, 8}, kStreamStages[kNumStreams] = {2, 1, 1, 1, 1, 1};

struct BlocksKernels {
    const void* tile[kNumBlockTiles][2];      // [tile][scales of B by rows]
    const void* stream[kNumStreams][2];
    const void* pair;
};
// By the formats of A and B.
const BlocksKernels& blocks_kernels_e4m3_e4m3();
const BlocksKernels& blocks_kernels_e4m3_e5m2();
const BlocksKernels& blocks_kernels_e5m2_e4m3();
const BlocksKernels& blocks_kernels_e5m2_e5m2();

// vec: x and the mask allow 16-byte loads of 8 elements.
const void* quantize_kernel(int dtype, int format, int tiles, int vec);

// One of the two products of the expert layer for a few tokens.
struct ExpertsArgs {
    const uint16_t* x;     // first: (tokens, in); second: the first's `mid`
    const uint8_t* w;      // (experts, out, ld) or (experts, in, ld) bytes
    const float* scales;   // 8-bit weights: (experts, out blocks, in blocks)
    const float* logits;   // (tokens, experts); nullptr: ids and weights are inputs
    int* ids;              // (tokens, top)
    float* weights;
    uint16_t* mid;         // (tokens top, [high, low], mid_row)
    float* part;           // second: (tokens top, splits, out)
    int* counters;         // second: one for each block of columns
    uint16_t* y;           // second: (tokens, out)
    int64_t ld;            // bytes from a row of w to the next
    int tokens, in, out, experts, top, mid_row;
    int renormalize, routed, splits;
    int once;              // with many units: the weights do not stay in the caches
};

constexpr int kMaxTokens = 64, kMaxTop = 16, kMaxExperts = 1024;
// Workgroups: columns of a unit, in blocks of 16 ((K, N) weights: 4 in both), and waves.
// For few units (one workgroup a CU), and for many.  A unit has 16 rows.
constexpr int kNumExpertKinds = 2, kExpertRows = 16;
constexpr int kExpertBlocks[kNumExpertKinds] = {2, 4}, kExpertWaves[kNumExpertKinds] = {8, 4};
constexpr int64_t route_table_bytes(int64_t slots, int64_t experts)
{
    return (slots + 1) / 2 * 4 + slots * 6 + experts * 6 + ((experts < slots ? experts : slots) + slots / 16 + 1) * 4;
}

struct ExpertsKernels {
    // [storage: NK, KN, e4m3, e5m2][odd rows][second product][kind]
    const void* products[4][2][2][kNumExpertKinds];
    const void* route;
};
const ExpertsKernels& experts_kernels_f16();
const ExpertsKernels& experts_kernels_bf16();

}  // namespace gemm_relu_hip
