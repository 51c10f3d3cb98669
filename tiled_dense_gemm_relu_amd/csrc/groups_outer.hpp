// The weights' gradients with few rows a group (gemm_relu_groups.h):
// out[g] = p^T q over group g's rows, written as fast as memory takes it.
//
// With a few rows a group (or none: its gradient is all zeros) the time is that
// of writing the outputs.  A wave takes 8 rows of an output and 512 columns, 8 of
// each to a lane, and adds the group's rows one by one in fp32 (64 multiply-adds
// a lane for 128 bytes of output); nothing is staged, so stores start at once.
#pragma once

#include "groups_kernels.hpp"

namespace gemm_relu_hip {

// `masked`: 1: p, 2: q is zero where `mask`, a matrix of its shape, is not above zero.
// Workgroup: tile b % tiles of group b / tiles, kOuterRows rows x kOuterCols columns,
// 8 rows to each wave.  ALIGNED: rows of out and q are whole 16-byte pieces and a
// lane has 8 consecutive columns; else it has 4 pairs of columns, 128 apart, that
// start on dwords of its output row: in a row that starts inside one, one element
// before (and single elements at the row's ends).
template <int DT, int MASKED, bool ALIGNED>
__global__ __launch_bounds__(kOuterThreads) void weight_outer(WeightArgs a, const uint16_t* mask)
{
    constexpr int kNonTemporal = 2;   // cache policy nt
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // (pairs of a row that starts inside a dword end one element early)
    const int tiles_j = ALIGNED ? (a.j + kOuterCols - 1) / kOuterCols : a.j / kOuterCols + 1, tiles = (a.i + kOuterRows - 1) / kOuterRows * tiles_j;
    const int g = (int)blockIdx.x / tiles, t = (int)blockIdx.x % tiles;
    const int i0 = t / tiles_j * kOuterRows + wave * 8, j0 = t % tiles_j * kOuterCols;
    if (i0 >= a.i) return;
    const int begin = g ? min(max(a.ends[g - 1], 0), a.m) : 0, end = max(min(max(a.ends[g], 0), a.m), begin);
    const int is = min(8, a.i - i0);
    // An element of p or q; columns past the row's end read its last one.
    auto at_p = [&](int m, int i) {
        const size_t x = (size_t)m * (size_t)a.i + (size_t)min(i, a.i - 1);
        return to_float<DT>(MASKED == 1 ? mask_one<DT>(a.p[x], mask[x]) : a.p[x]);
    };
    auto at_q = [&](int m, int j) {
        const size_t x = (size_t)m * (size_t)a.j + (size_t)min(max(j, 0), a.j - 1);
        return to_float<DT>(MASKED == 2 ? mask_one<DT>(a.q[x], mask[x]) : a.q[x]);
    };
    uint16_t* const out = a.out + ((size_t)g * (size_t)a.i + (size_t)i0) * (size_t)a.j;
    float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    if constexpr (ALIGNED) {
        const int j = j0 + 8 * lane;
        if (j >= a.j) return;
        for (int m = begin; m < end; ++m) {
            const size_t x = (size_t)m * (size_t)a.j + (size_t)j;
            u32x4 w = *reinterpret_cast<const u32x4*>(a.q + x);
            if constexpr (MASKED == 2) w = mask_chunk<DT>(w, *reinterpret_cast<const u32x4*>(mask + x));
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = at_p(m, i0 + i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float q = to_float<DT>((uint16_t)(w[e / 2] >> (16 * (e & 1))));
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i][e] += p[i] * q;
            }
        }
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(out, (uint32_t)is * (uint32_t)a.j * 2u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u32x4 v;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                v[w] = (uint32_t)act_cast<DT>(acc[i][2 * w], false) | ((uint32_t)act_cast<DT>(acc[i][2 * w + 1], false) << 16);
            // rows past the last are out of range: dropped
            __builtin_amdgcn_raw_buffer_store_b128(v, ro, ((uint32_t)i * (uint32_t)a.j + (uint32_t)j) * 2u, 0, kNonTemporal);
        }
    } else {
        for (int m = begin; m < end; ++m) {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = at_p(m, i0 + i);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = j0 + 2 * (lane + 64 * x);
                const float before = at_q(m, j - 1), q0 = at_q(m, j), q1 = at_q(m, j + 1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool odd = (reinterpret_cast<uintptr_t>(out + (size_t)i * (size_t)a.j) & 2) != 0;
                    acc[i][2 * x] += p[i] * (odd ? before : q0);
                    acc[i][2 * x + 1] += p[i] * (odd ? q0 : q1);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= is) break;
            uint16_t* const row = out + (size_t)i * (size_t)a.j;
            const int odd = (int)((reinterpret_cast<uintptr_t>(row) >> 1) & 1);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = j0 + 2 * (lane + 64 * x) - odd;
                const uint16_t v0 = act_cast<DT>(acc[i][2 * x], false), v1 = act_cast<DT>(acc[i][2 * x + 1], false);
                if (j >= 0 && j + 1 < a.j) {
                    *reinterpret_cast<uint32_t*>(row + j) = (uint32_t)v0 | ((uint32_t)v1 << 16);
                } else {
                    if (j >= 0 && j < a.j) row[j] = v0;
                    if (j + 1 >= 0 && j + 1 < a.j) row[j + 1] = v1;
                }
            }
        }
    }
}

}  // namespace gemm_relu_hip
