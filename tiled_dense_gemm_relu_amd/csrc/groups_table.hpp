// Kernel arguments and the host-side table of kernel instances of the products
// whose rows choose their weights (gemm_relu_groups.h), filled by one
// translation unit per dtype and read by groups_api.hip.
#pragma once

#include <stdint.h>

namespace gemm_relu_hip {

// A product over groups of rows.  ends == nullptr: all rows are group 0.
struct RowsArgs {
    const uint16_t* a;     // (M, K)
    const uint16_t* b;     // (groups, K, N) or (groups, N, K)
    uint16_t* c;           // (M, N)
    const int* ends;
    int m, n, k, groups;
    int relu;
    int lda, ldb;          // row lengths of a and b
    int c_vec;             // rows of C allow 2: 16-byte, 1: 8-byte, 0: 2-byte stores
};

// The low-rank term of each row (v == nullptr: none).  Row m's adapter is
// row_id[m] (-1: none) and its intermediate t[m][lo | hi][rank_pad] times
// factor[m], see adapter_shrink.
struct AdapterArgs {
    const uint16_t* v;     // (adapters, rank, N) or (adapters, N, rank)
    const uint16_t* t;
    const float* factor;
    const int* row_id;
    const int* ends;       // segments of rows and their adapters
    const int* ids;
    int segments, adapters, rank, rank_pad;
    int v_fast;            // V's rows allow the widest loads of a lane of its own: 8 bytes (4 columns), or 16 (8 rank entries)
};

struct ShrinkArgs {
    const uint16_t* x;     // (M, K)
    const uint16_t* u;     // (adapters, K, rank) or (adapters, rank, K)
    const float* scales;
    const int* ends;
    const int* ids;
    uint16_t* t;
    float* factor;
    int* row_id;
    float* part;           // [row tile][split][32 columns][rows x 32] sums
    int* counters;         // one for each row tile
    int m, k, segments, adapters, rank, rank_pad;
};

// dB[g] = sum of p[m]^T q[m] over group g's rows: p (M, I), q (M, J), out (groups, I, J).
struct WeightArgs {
    const uint16_t* p;
    const uint16_t* q;
    uint16_t* out;
    const int* ends;
    int m, i, j, groups;
    int ldp, ldq;          // row lengths of p and q
    int c_vec;
};

// Rows of `cols` elements copied to rows of `pitch` (whole 16-byte pieces), zeros
// after them; mask != nullptr: zero where that is not above zero.
struct PadArgs {
    const uint16_t* src;
    const uint16_t* mask;
    uint16_t* dst;
    int64_t rows;
    int cols, pitch;
};

struct MaskArgs {
    const uint16_t* dc;
    const uint16_t* c;
    uint16_t* d;
    int64_t count;
    int vec;               // 16-byte aligned pointers
};

constexpr int kMaxRank = 256;
constexpr int kShrinkRows = 16, kShrinkCols = 32, kShrinkK = 128, kShrinkThreads = 512;

// Square LDS-DMA tiles, by GEMM_RELU_GROUPS_DMA_* order, and their workgroups.
constexpr int kNumGroupTiles = 3;
constexpr int kGroupTile[kNumGroupTiles] = {256, 128, 64};
constexpr int kGroupThreads[kNumGroupTiles] = {512, 512, 512};

// Square tiles staged through registers (GEMM_RELU_GROUPS_TILED), large and small.
constexpr int kNumStagedTiles = 2;
constexpr int kStagedTile[kNumStagedTiles] = {128, 64};
constexpr int kStagedThreads = 512;

// The register-staged kernels: dwords may hold two rows' elements (any row
// length and 2-byte alignment), or not (even rows, 4-byte alignment).
struct StagedKernels {
    const void* rows[kNumStagedTiles][2][2][2];   // [tile][B layout][with adapters][more than 64 groups]
    // Both gradients: [tile][B layout of dA's product][masked][more than 64 groups].
    // dA's product reads B stored (K, N) as (N, K) rows and the other way round,
    // and dB of the one is A^T D, of the other D^T A.
    const void* grad[kNumStagedTiles][2][2][2];
};

// Streaming kernels for few rows a group: 16-row blocks a workgroup takes.
constexpr int kNumSkinny = 3;
constexpr int kSkinnyBlocks[kNumSkinny] = {1, 2, 4};
// Weights' gradients with few rows a group.
constexpr int kOuterThreads = 256;
// Workgroups of an (i, j) output, 8 x 8 elements to a lane; rows that start inside a dword end one element early.
constexpr int64_t outer_tiles(int64_t i, int64_t j, bool aligned)
{
    return ((i + 7) / 8 * (j / 8 + (aligned ? 0 : 1)) + kOuterThreads - 1) / kOuterThreads;
}
// First of the 4 columns of V that a lane reads for columns n .. n + 3 of its tile, which
// may lie past the last of N: then some at the end, whose sums are not stored.  `whole`: the
// 4 are read in one piece (n % 4 == 0 and N % 4 == 0), else one at a time up to N.
constexpr int low_rank_column(int n, int N, bool whole) { return n < N ? n : whole ? N - 4 : N - 1; }
constexpr int kSkinnyCols = 32, kSkinnyK = 128, kSkinnyThreads = 512;

struct GroupKernels {
    // [tile][B layout][KTAIL][with adapters].  The 256 tile takes rows of whole
    // 16-byte pieces only (KTAIL < 2); with adapters it takes any such K and starts
    // from their terms.
    const void* rows_dma[kNumGroupTiles][2][3][2];
    const void* weight_dma[kNumGroupTiles][2];    // [tile][rows of any even length]
    const void* rows_skinny[kNumSkinny][2][2][3];   // [blocks][B layout][odd rows][plain, adapters, masked]
    const void* weight_outer[3][2];                 // [masked: no, p, q][rows of whole pieces]
    const void* mask;
    const void* pad;
    const void* shrink[2][2][2];                    // [U layout][rank > 32][32 rows]
};

const GroupKernels& group_kernels_f16();
const GroupKernels& group_kernels_bf16();
const StagedKernels& staged_kernels_f16_even();
const StagedKernels& staged_kernels_f16_odd();
const StagedKernels& staged_kernels_bf16_even();
const StagedKernels& staged_kernels_bf16_odd();

}  // namespace gemm_relu_hip
