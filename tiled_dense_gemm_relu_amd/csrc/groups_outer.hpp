// The weights' gradients with few rows a group (gemm_relu_groups.h):
// out[g] = p^T q over group g's rows, written as fast as memory takes it.
//
// With a few rows a group (or none: its gradient is all zeros) the time is that
// of writing the outputs.  A lane takes 8 rows of an output and 8 columns and adds
// the group's rows one by one in fp32 (64 multiply-adds for 128 bytes of output);
// nothing is staged, so stores start at once.
#pragma once

#include "groups_kernels.hpp"

namespace gemm_relu_hip {

// MASKED: 1: p, 2: q is zero where `mask`, a matrix of its shape, is not above zero.
// A lane has 8 rows of out and 8 consecutive columns, lanes numbered through the
// strips of 8 rows.  ALIGNED: rows of out and q are whole 16-byte pieces.  Else a
// lane's columns start on a dword of their output row, so in rows that start
// inside one they are one element further back; 16-byte stores at dword alignment,
// and single elements at a row's ends.
template <int DT, int MASKED, bool ALIGNED>
__global__ __launch_bounds__(kOuterThreads) void weight_outer(WeightArgs a, const uint16_t* mask)
{
    const int strips = (a.i + 7) / 8, tiles = (int)outer_tiles(a.i, a.j, ALIGNED);
    const int g = (int)blockIdx.x / tiles, t = (int)blockIdx.x % tiles;
    const int begin = g ? min(max(a.ends[g - 1], 0), a.m) : 0, end = max(min(max(a.ends[g], 0), a.m), begin);
    const int across = a.j / 8 + (ALIGNED ? 0 : 1), at = t * kOuterThreads + (int)threadIdx.x;
    const int strip = at / across, j0 = at % across * 8;
    if (strip >= strips) return;
    const int i0 = 8 * strip, is = min(8, a.i - i0);
    // 8 elements from column x on of row m of p or q (zeros, or the next row's, past its end).
    auto load8 = [&](const uint16_t* of, int cols, int m, int x, bool masked) {
        const size_t at = (size_t)m * (size_t)cols;
        const AnyRsrc r = make_any_rsrc(of + at, (uint32_t)cols * 2u);
        const AnyChunk c = load_any(r, (uint32_t)x * 2u, true);
        if (!masked) return chunk_value(c);
        const AnyRsrc rm = make_any_rsrc(mask + at, (uint32_t)cols * 2u);
        return mask_chunk<DT>(chunk_value(c), chunk_value(load_any(rm, (uint32_t)x * 2u, true)));
    };
    auto element = [](u32x4 v, int e) { return to_float<DT>((uint16_t)(v[e / 2] >> (16 * (e & 1)))); };
    uint16_t* const out = a.out + ((size_t)g * (size_t)a.i + (size_t)i0) * (size_t)a.j;
    float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    if constexpr (ALIGNED) {
#pragma unroll 2
        for (int m = begin; m < end; ++m) {
            const size_t x = (size_t)m * (size_t)a.j + (size_t)j0;
            u32x4 w = *reinterpret_cast<const u32x4*>(a.q + x);
            if constexpr (MASKED == 2) w = mask_chunk<DT>(w, *reinterpret_cast<const u32x4*>(mask + x));
            const u32x4 p = load8(a.p, a.i, m, i0, MASKED == 1);
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i][e] += element(p, i) * element(w, e);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= is) break;
            u32x4 v;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                v[w] = (uint32_t)act_cast<DT>(acc[i][2 * w], false) | ((uint32_t)act_cast<DT>(acc[i][2 * w + 1], false) << 16);
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out + (size_t)i * (size_t)a.j + (size_t)j0));
        }
    } else {
        typedef u32x4 u32x4_dwords __attribute__((aligned(4)));
        // (8 strip rows are whole dwords: the parity of row i is the same in all strips)
        const uint32_t odd0 = (uint32_t)(reinterpret_cast<uintptr_t>(a.out + (size_t)g * (size_t)a.i * (size_t)a.j) >> 1) & 1u;
#pragma unroll 2
        for (int m = begin; m < end; ++m) {
            const u32x4 p = load8(a.p, a.i, m, i0, MASKED == 1), w = load8(a.q, a.j, m, j0, MASKED == 2);
            const size_t x = (size_t)m * (size_t)a.j + (size_t)max(j0 - 1, 0);
            float q[9];                // from the element before on (of the first column, any: it is not stored)
            q[0] = to_float<DT>(MASKED == 2 ? mask_one<DT>(a.q[x], mask[x]) : a.q[x]);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e + 1] = element(w, e);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool odd = ((odd0 ^ ((uint32_t)i & (uint32_t)a.j)) & 1u) != 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float before = q[e], here = q[e + 1];    // (values: a choice of places would put q in memory)
                    acc[i][e] += element(p, i) * (odd ? before : here);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= is) break;
            const int j = j0 - (int)((odd0 ^ ((uint32_t)i & (uint32_t)a.j)) & 1u);
            uint16_t* const row = out + (size_t)i * (size_t)a.j;
            if (j >= 0 && j + 8 <= a.j) {
                u32x4 v;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    v[w] = (uint32_t)act_cast<DT>(acc[i][2 * w], false) | ((uint32_t)act_cast<DT>(acc[i][2 * w + 1], false) << 16);
                *reinterpret_cast<u32x4_dwords*>(row + j) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j + e >= 0 && j + e < a.j) row[j + e] = act_cast<DT>(acc[i][e], false);
            }
        }
    }
}

}  // namespace gemm_relu_hip
