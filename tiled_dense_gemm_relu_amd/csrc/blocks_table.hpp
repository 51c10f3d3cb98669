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

// One launch quantizes both ways what it reads once; q or qt may be nullptr.
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
    int vec;               // x and mask allow 16-byte loads of 8 elements
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
};

constexpr int kNumBlockTiles = 3;
constexpr int kBlockTile[kNumBlockTiles] = {256, 128, 64};
constexpr int kBlockThreads[kNumBlockTiles] = {512, 256, 256};

struct BlocksKernels {
    const void* tile[kNumBlockTiles][2];      // [tile][scales of B by rows]
};
// By the formats of A and B.
const BlocksKernels& blocks_kernels_e4m3_e4m3();
const BlocksKernels& blocks_kernels_e4m3_e5m2();
const BlocksKernels& blocks_kernels_e5m2_e4m3();
const BlocksKernels& blocks_kernels_e5m2_e5m2();

// [dtype][format][form == tiles]
const void* quantize_kernel(int dtype, int format, int tiles);

}  // namespace gemm_relu_hip
