// The product of 8-bit matrices scaled by blocks of 128 with few rows a group, or
// few operations at all (gemm_relu_blocks.h).
//
// Where rows are few the time is that of reading the weights, and where everything
// is small that of one trip to memory.  A workgroup takes 16 MB rows of a group and
// 16 NB columns; its waves take scale blocks of 128 k in turn and add their sums in
// LDS.  Each wave streams its blocks through a ring of its own in LDS, by DMA, so no
// barrier is met before the sums, and every wave has a block or two in flight.  (DMA
// fetches whole 128-byte lines, 8 rows an instruction; a matrix operand loaded into
// registers is 64 bytes of 16 rows.  One row x 16384 x 8192: 74 us through registers,
// 29 so, and 24.3, 5.5 TB/s, past the caches.)  64 rows: 28.3.
//
// No workgroup waits for another: cutting K over workgroups too, with sums added by
// the last to end, cost more than it gave in all sizes but the longest K over the
// fewest columns (one row x 1024 x 8192: 8.7 us against 9.4; x 4096 x 4096: 9.4 against 8.5).
#pragma once

#include "blocks_bytes.hpp"
#include "blocks_dma.hpp"

namespace gemm_relu_hip {

template <int FA, int FB, bool B_ROWS, int KIND>
__global__ __launch_bounds__(64 * kStreamWaves[KIND], 1) void blocks_stream(BlocksArgs a)
{
    constexpr int MB = kStreamRows[KIND], NB = kStreamCols[KIND], WAVES = kStreamWaves[KIND], kStreamThreads = 64 * WAVES, ROWS = 16 * MB, COLS = 16 * NB, PART = COLS * 17;
    constexpr int S = kStreamStages[KIND], X_BYTES = MB * 2048, W_BYTES = NB * 2048, STAGE = X_BYTES + W_BYTES + 512;
    constexpr int NQ = 2 * MB + 2 * NB + 2, RING = WAVES * S * STAGE;
    constexpr int OUT = (16 * COLS + kStreamThreads - 1) / kStreamThreads;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > WAVES * PART * 4 ? RING : WAVES * PART * 4];
    float* const part = reinterpret_cast<float*>(smem);       // the waves' sums, after the rings
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tid = threadIdx.x;
    const int tiles_n = (a.n + COLS - 1) / COLS;
    const int pid = (int)blockIdx.x;
    const RowTile tile = find_row_tile(a.ends, a.groups, a.m, ROWS, pid / tiles_n, lane);
    if (tile.group < 0) return;
    const int rows = tile.end - tile.begin, n0 = pid % tiles_n * COLS, cols = min(COLS, a.n - n0);
    const bool real = tile.group < a.groups;
    const int r16 = lane & 15, g = lane >> 4;
    floatx4 acc[NB][MB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    if (real) {
        const int blocks = (a.k + kBlock - 1) / kBlock, n_tiles = (a.n + kBlock - 1) / kBlock;
        const float* const sb = B_ROWS ? a.sb + (size_t)tile.group * (size_t)blocks * (size_t)a.n + (size_t)n0
                                       : a.sb + ((size_t)tile.group * (size_t)n_tiles + (size_t)(n0 / kBlock)) * (size_t)blocks;
        // Every workgroup starts at another block of its rows: with row lengths of a
        // power of two a block of all rows lies in few memory channels, and workgroups
        // in step would all wait for the same ones.
        const int turn = pid % blocks;
        // This wave's i-th block of k; the ring holds S of them.
        const int mine = blocks > wave ? (blocks - wave + WAVES - 1) / WAVES : 0;
        auto block_at = [&](int i) {
            const int p = wave + i * WAVES;
            return p + turn < blocks ? p + turn : p + turn - blocks;
        };
        uint8_t* const ring = smem + wave * (S * STAGE);
        const uint32_t ring_lds = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem) + (uint32_t)(wave * (S * STAGE));
        // A lane's 16 bytes of a DMA instruction of 8 rows, swizzled (a_swizzle): the
        // pattern repeats after two of them.
        uint32_t x_off[2], w_off[2];
        int pos[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = 8 * q + lane / 8;
            pos[q] = ((lane % 8) ^ a_swizzle<128>(row)) * 16;
            x_off[q] = (uint32_t)row * a.lda + (uint32_t)pos[q];
            w_off[q] = (uint32_t)row * a.ldb + (uint32_t)pos[q];
        }
        const uint8_t* const xp = a.a + (size_t)tile.begin * a.lda;
        const uint8_t* const wp = a.b + ((size_t)tile.group * (size_t)a.n + (size_t)n0) * a.ldb;
        auto uniform = [](const void* p, uint32_t bytes) {
            const int32x4_t r = rsrc_words(p, bytes);
            return int32x4_t{__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]),
                             __builtin_amdgcn_readfirstlane(r[2]), kBufferFlags};
        };
        auto fill = [&](int i, int slot) {
            // past this wave's last block nothing is fetched
            const bool live = i < mine;
            const int b = __builtin_amdgcn_readfirstlane(block_at(live ? i : 0)), k0 = b * kBlock, left = live ? a.k - k0 : 0;
            const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(ring_lds + (uint32_t)(slot * STAGE)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t xo = pos[h] < left ? x_off[h] : kOobOffset, wo = pos[h] < left ? w_off[h] : kOobOffset;
#pragma unroll
                for (int j = 0; j < MB; ++j)
                    dma_b128(uniform(xp + (size_t)(16 * j) * a.lda, (uint32_t)max(0, rows - 16 * j) * a.lda), to + (2 * j + h) * 1024, xo, (uint32_t)k0);
                const auto weights = [&](auto&& load) __attribute__((always_inline)) {
#pragma unroll
                    for (int i2 = 0; i2 < NB; ++i2)
                        load(uniform(wp + (size_t)(16 * i2) * a.ldb, (uint32_t)max(0, cols - 16 * i2) * a.ldb), to + X_BYTES + (2 * i2 + h) * 1024, wo, (uint32_t)k0);
                };
                if (a.once) weights(dma_b128_once);
                else weights(dma_b128);
            }
            dma_b32(uniform(a.sa + (size_t)b * (size_t)a.m + (size_t)tile.begin, (live ? (uint32_t)rows : 0u) * 4u), to + X_BYTES + W_BYTES, 4u * (uint32_t)lane, 0u);
            dma_b32(uniform(B_ROWS ? sb + (size_t)b * (size_t)a.n : sb + b, live ? B_ROWS ? (uint32_t)cols * 4u : 4u : 0u),
                    to + X_BYTES + W_BYTES + 256, B_ROWS ? 4u * (uint32_t)lane : 0u, 0u);
        };
        const int kb = kgroup16(g);
        uint32_t off[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) off[h] = (uint32_t)(r16 * 128 + 16 * ((4 * h + kb) ^ a_swizzle<128>(r16)));
#pragma unroll
        for (int s = 0; s < S; ++s) fill(s, s);
        int slot = 0;
        for (int i = 0; i < mine; ++i) {
            wait_vmcnt<(S - 1) * NQ>();
            const uint8_t* const st = ring + slot * STAGE;
            const float *const sx = reinterpret_cast<const float*>(st + X_BYTES + W_BYTES), *const sw = sx + 64;
            u32x4 x[MB][2], w[NB][2];
            SplitScale scale_x[MB];
            floatx4 scale_w[B_ROWS ? NB : 1];
            uint32_t exponent_w[B_ROWS ? NB : 1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < MB; ++j) x[j][h] = *reinterpret_cast<const u32x4*>(st + off[h] + j * 2048);
#pragma unroll
                for (int i2 = 0; i2 < NB; ++i2) w[i2][h] = *reinterpret_cast<const u32x4*>(st + X_BYTES + off[h] + i2 * 2048);
            }
#pragma unroll
            for (int j = 0; j < MB; ++j) scale_x[j] = split_scale(sx[16 * j + r16]);
            if constexpr (B_ROWS) {
#pragma unroll
                for (int i2 = 0; i2 < NB; ++i2) {
                    const floatx4 s4 = *reinterpret_cast<const floatx4*>(sw + 16 * i2 + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) scale_w[i2][e] = split_scale(s4[e]).m;
                    exponent_w[i2] = split_scale(sw[16 * i2 + r16]).e;
                }
            } else {
                const SplitScale s = split_scale(sw[0]);
                scale_w[0][0] = s.m;
                exponent_w[0] = s.e;
            }
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");     // the slot has been read
            fill(i + S, slot);
            slot = slot + 1 < S ? slot + 1 : 0;
            const int k0 = block_at(i) * kBlock;
            if (a.k - k0 < kBlock) {          // what lies behind the rows must not meet the other operand's zeros
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int valid = a.k - (k0 + 16 * (4 * h + kb));
#pragma unroll
                    for (int j = 0; j < MB; ++j) x[j][h] = keep_bytes(x[j][h], valid);
#pragma unroll
                    for (int i2 = 0; i2 < NB; ++i2) w[i2][h] = keep_bytes(w[i2][h], valid);
                }
            }
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int i2 = 0; i2 < NB; ++i2) {
                    const floatx4 t = mfma_block<FB, FA>(join(w[i2][0], w[i2][1]), join(x[j][0], x[j][1]), exponent_w[B_ROWS ? i2 : 0], 0,
                                                         scale_x[j].e, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i2][j][e] = __builtin_fmaf(t[e], scale_x[j].m * scale_w[B_ROWS ? i2 : 0][B_ROWS ? e : 0], acc[i2][j][e]);
                }
        }
        wait_vmcnt<0>();                       // nothing lands in the rings after this
    }
    __syncthreads();
    uint16_t* const c = a.c + (size_t)tile.begin * (size_t)a.n + (size_t)n0;
    auto store = [&](int row, int col, float z) {
        c[(size_t)row * (size_t)a.n + (size_t)col] = a.bf16 ? act_cast<kBF16>(z, a.relu != 0) : act_cast<kF16>(z, a.relu != 0);
    };
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        if (16 * j >= rows) break;
        if (j > 0) __syncthreads();     // the sums of the row block before are read
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[wave * PART + (16 * i + 4 * g + e) * 17 + r16] = acc[i][j][e];
        __syncthreads();
#pragma unroll
        for (int s = 0; s < OUT; ++s) {
            const int o = s * kStreamThreads + tid, row = o / COLS, col = o % COLS;
            if (o >= 16 * COLS) break;
            float z = 0.0f;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) z += part[v * PART + col * 17 + row];
            if (16 * j + row < rows && col < cols) store(16 * j + row, col, z);
        }
    }
}

}  // namespace gemm_relu_hip
