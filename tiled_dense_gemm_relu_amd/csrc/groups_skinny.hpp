// Products with few rows a group (gemm_relu_groups.h): the weights stream from
// memory into registers, once.
//
// With a few rows for each group the time is that of reading the weights.  A
// workgroup takes up to 16 MB rows of a group and 32 columns; its 8 waves take
// pieces of 128 k in turn, each with the piece's loads all in flight (8 KiB of
// weights a wave), and add their sums in LDS.  Workgroups are small and many
// (several on a CU, unlike the tiles' one), so loads of one cover the start and
// end of another.
#pragma once

#include "groups_kernels.hpp"

namespace gemm_relu_hip {

// 8 consecutive elements from an even byte offset on: with ODD they may start
// inside a dword (load_any), else at dword boundaries.
template <bool ODD>
struct SkinnyChunk {
    u32x4 v;
    uint32_t next;
};
template <bool ODD>
__device__ __forceinline__ SkinnyChunk<ODD> load_skinny(const AnyRsrc& r, uint32_t off)
{
    SkinnyChunk<ODD> c;
    if constexpr (ODD) {
        const uint32_t at = (off + r.shift) & ~3u;
        c.v = __builtin_amdgcn_raw_buffer_load_b128(r.rsrc, at, 0, 0);
        c.next = __builtin_amdgcn_raw_buffer_load_b32(r.rsrc, at + 16u, 0, 0);
    } else {
        c.v = __builtin_amdgcn_raw_buffer_load_b128(r.rsrc, off, 0, 0);
        c.next = 0;
    }
    return c;
}
template <bool ODD>
__device__ __forceinline__ u32x4 skinny_value(const SkinnyChunk<ODD>& c, const AnyRsrc& r, uint32_t off)
{
    if constexpr (!ODD) return c.v;
    else return chunk_value(AnyChunk{c.v, c.next, ((off + r.shift) & 2u) * 8u});
}

// Add the low-rank terms of rows m, m + 16, ... (below m_end) at column n to z:
// (hi + lo) . V_i[:, n] times the row's factor, the rows' loads in flight together.
template <int DT, bool B_NK, int MB>
__device__ __forceinline__ void add_low_rank(float (&z)[MB], const AdapterArgs& ad, int m, int m_end, int n, int N)
{
    const size_t step = B_NK ? 1 : (size_t)N;
    const uint16_t *t[MB], *v[MB];
    float factor[MB], sum[MB];
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        const int row = min(m + 16 * j, m_end - 1), id = ad.row_id[row];
        // without an adapter: V_0, and a factor that drops it
        factor[j] = id >= 0 && m + 16 * j < m_end ? ad.factor[row] : 0.0f;
        t[j] = ad.t + (size_t)row * (size_t)(2 * ad.rank_pad);
        v[j] = ad.v + (size_t)max(id, 0) * (size_t)ad.rank * (size_t)N + (B_NK ? (size_t)n * (size_t)ad.rank : (size_t)n);
        sum[j] = 0.0f;
    }
#pragma unroll MB == 1 ? 4 : 2
    for (int r0 = 0; r0 < ad.rank; r0 += 8) {
        u32x4 hi[MB], lo[MB];
        uint16_t w[MB][8];
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            lo[j] = *reinterpret_cast<const u32x4*>(t[j] + r0);
            hi[j] = *reinterpret_cast<const u32x4*>(t[j] + ad.rank_pad + r0);
            if (B_NK && ad.v_fast) {
                const u32x4 q = *reinterpret_cast<const u32x4*>(v[j] + r0);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[j][e] = (uint16_t)(q[e / 2] >> (16 * (e & 1)));
            } else {
                // entries past the rank repeat the last one
#pragma unroll
                for (int e = 0; e < 8; ++e) w[j][e] = v[j][(size_t)min(r0 + e, ad.rank - 1) * step];
            }
        }
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = to_float<DT>((uint16_t)(hi[j][e / 2] >> (16 * (e & 1)))) +
                                to_float<DT>((uint16_t)(lo[j][e / 2] >> (16 * (e & 1))));
                sum[j] += r0 + e < ad.rank ? x * to_float<DT>(w[j][e]) : 0.0f;
            }
    }
#pragma unroll
    for (int j = 0; j < MB; ++j) z[j] = factor[j] != 0.0f ? z[j] + factor[j] * sum[j] : z[j];
}

// C = act(rows of A @ their group's B [+ their adapters' terms]).  Workgroup b of
// a part of K: column block and row tile as tile_coords orders them for the
// XCDs, columns fastest.  With few units K is cut into gridDim.y parts, combined
// as in adapter_shrink.  kSkinnyMasked: A is zero where `mask`, a matrix of its
// shape, is not above zero.
enum { kSkinnyPlain = 0, kSkinnyAdapters = 1, kSkinnyMasked = 2 };
template <int DT, bool B_NK, int MB, bool ODD, int MODE>
__global__ __launch_bounds__(kSkinnyThreads) void rows_skinny(RowsArgs a, AdapterArgs ad, float* parts, int* counters,
                                                              const uint16_t* mask)
{
    constexpr int WAVES = kSkinnyThreads / 64, STEPS = kSkinnyK / 32, ROWS = 16 * MB, ROW = kSkinnyCols * 2;
    constexpr int kDeviceScope = 16;   // cache policy sc1
    constexpr bool ADAPT = MODE == kSkinnyAdapters, MASKED = MODE == kSkinnyMasked;
    constexpr int PART = kSkinnyCols * (ROWS + 1);
    // the waves' sums, and before that their strips of B (K, N)
    __shared__ __attribute__((aligned(16))) float part[WAVES * PART > WAVES * 512 ? WAVES * PART : WAVES * 512];
    __shared__ int before;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tiles_n = (a.n + kSkinnyCols - 1) / kSkinnyCols, units = (int)gridDim.x;
    const int per_xcd = units / 8, u = (int)blockIdx.x;
    const int pid = u < per_xcd * 8 ? (u % 8) * per_xcd + u / 8 : u;
    const RowTile tile = find_row_tile(a.ends, a.groups, a.m, ROWS, pid / tiles_n, lane);
    if (tile.group < 0) return;
    const int rows = tile.end - tile.begin, n0 = pid % tiles_n * kSkinnyCols;
    const bool real = tile.group < a.groups;
    if (!real && blockIdx.y > 0) return;
    const int r16 = lane & 15, kb = kgroup16(lane >> 4);
    const size_t k_len = (size_t)a.k, n_len = (size_t)a.n;
    floatx4 acc[2][MB];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    if (real) {
        const AnyRsrc rx = make_any_rsrc(a.a + (size_t)tile.begin * k_len, (uint32_t)rows * (uint32_t)a.k * 2u);
        const AnyRsrc rm = MASKED ? make_any_rsrc(mask + (size_t)tile.begin * k_len, (uint32_t)rows * (uint32_t)a.k * 2u) : rx;
        const uint16_t* b = a.b + (size_t)tile.group * k_len * n_len;
        const AnyRsrc rb = B_NK ? make_any_rsrc(b + (size_t)n0 * k_len, (uint32_t)min(kSkinnyCols, a.n - n0) * (uint32_t)a.k * 2u)
                                : AnyRsrc{};
        uint8_t* strip = reinterpret_cast<uint8_t*>(part) + wave * 2048;
        const int pieces = (a.k + kSkinnyK - 1) / kSkinnyK, splits = (int)gridDim.y;
        // Every workgroup starts at another piece of its part: with row lengths of a
        // power of two a piece of all rows lies in one L2 channel, and workgroups in
        // step would all wait for the same one.
        const int p_begin = (int)((int64_t)pieces * blockIdx.y / splits);
        const int count = (int)((int64_t)pieces * (blockIdx.y + 1) / splits) - p_begin, turn = pid % max(count, 1);
        for (int p = wave; p < count; p += WAVES) {
            const int k0 = (p_begin + (p + turn < count ? p + turn : p + turn - count)) * kSkinnyK;
            const bool tail = k0 + kSkinnyK > a.k;
            // B stored (K, N): this piece's rows from column n0 on
            const AnyRsrc rp = B_NK ? rb
                                    : make_any_rsrc(b + (size_t)k0 * n_len + n0,
                                                    (uint32_t)(min(kSkinnyK, a.k - k0) * a.n - n0) * 2u);
            SkinnyChunk<ODD> x[STEPS][MB], w[STEPS][2], above[MASKED ? STEPS : 1][MASKED ? MB : 1];
            uint32_t x_off[MB], w_off[2];
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                const int r = 16 * j + r16;
                x_off[j] = r < rows ? ((uint32_t)r * (uint32_t)a.k + (uint32_t)(k0 + 8 * kb)) * 2u : kOobOffset;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w_off[i] = B_NK ? ((uint32_t)(16 * i + r16) * (uint32_t)a.k + (uint32_t)(k0 + 8 * kb)) * 2u
                           : n0 + 8 * (lane & 3) < a.n
                               ? ((uint32_t)(16 * i + (lane >> 2)) * (uint32_t)a.n + (uint32_t)(8 * (lane & 3))) * 2u
                               : kOobOffset;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
#pragma unroll
                for (int i = 0; i < 2; ++i) w[s][i] = load_skinny<ODD>(rp, w_off[i] + (B_NK ? 64u * s : 64u * s * (uint32_t)a.n));
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    x[s][j] = load_skinny<ODD>(rx, x_off[j] + 64u * s);
                    if constexpr (MASKED) above[s][j] = load_skinny<ODD>(rm, x_off[j] + 64u * s);
                }
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int valid = a.k - (k0 + 32 * s + 8 * kb);
                u32x4 wv[2], xv[MB];
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    xv[j] = skinny_value<ODD>(x[s][j], rx, x_off[j] + 64u * s);
                    if constexpr (MASKED) xv[j] = mask_chunk<DT>(xv[j], skinny_value<ODD>(above[s][j], rm, x_off[j] + 64u * s));
                    if (tail) xv[j] = keep_first(xv[j], valid);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    wv[i] = skinny_value<ODD>(w[s][i], rp, w_off[i] + (B_NK ? 64u * s : 64u * s * (uint32_t)a.n));
                    if constexpr (B_NK) {
                        if (tail) wv[i] = keep_first(wv[i], valid);
                    } else {
                        const int kr = 16 * i + (lane >> 2);
                        if (tail && k0 + 32 * s + kr >= a.k) wv[i] = u32x4{0u, 0u, 0u, 0u};
                        *reinterpret_cast<u32x4*>(strip + kr * ROW + 16 * ((lane & 3) ^ b_swizzle<ROW, 16>(kr))) = wv[i];
                    }
                }
                if constexpr (!B_NK) {
                    const int kr = 8 * kb + (r16 >> 2);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = 16 * i + 4 * (r16 & 3);
                        const uint8_t* q = strip + kr * ROW + 16 * ((n >> 3) ^ b_swizzle<ROW, 16>(kr)) + 8 * (r16 & 1);
                        const u32x2 lo = ds_read_tr16(q), hi = ds_read_tr16(q + 4 * ROW);
                        wv[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < MB; ++j) acc[i][j] = mfma_16x16x32<DT>(wv[i], xv[j], acc[i][j]);
            }
        }
        __syncthreads();               // the strips are read
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    part[wave * PART + (16 * i + 4 * (lane >> 4) + e) * (ROWS + 1) + 16 * j + r16] = acc[i][j][e];
    }
    __syncthreads();
    // 512 threads: 16 rows x 32 columns of each block of rows
    const int row = threadIdx.x >> 5, col = threadIdx.x & 31;
    float z[MB];
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        z[j] = 0.0f;
        if (real) {
#pragma unroll
            for (int w = 0; w < WAVES; ++w) z[j] += part[w * PART + col * (ROWS + 1) + 16 * j + row];
        }
    }
    if (gridDim.y > 1 && real) {
        const uint32_t splits = gridDim.y, bytes = MB * kSkinnyThreads * 4u;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(parts + (size_t)u * (size_t)splits * (bytes / 4), splits * bytes);
#pragma unroll
        for (int j = 0; j < MB; ++j)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, z[j]), rs,
                                                  blockIdx.y * bytes + (uint32_t)(j * kSkinnyThreads + threadIdx.x) * 4u, 0,
                                                  kDeviceScope);
        wait_vmcnt<0>();               // this wave's sums have reached device scope
        __syncthreads();
        if (threadIdx.x == 0)
            before = __hip_atomic_fetch_add(counters + u, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (before != (int)splits - 1) return;
        asm volatile("" ::: "memory");   // the loads below stay after the count that allowed them
#pragma unroll
        for (int j = 0; j < MB; ++j) z[j] = 0.0f;
        for (uint32_t s0 = 0; s0 < splits; s0 += 4) {
            float o[4][MB];
#pragma unroll
            for (int s = 0; s < 4; ++s)   // parts past the last are out of range: zero
#pragma unroll
                for (int j = 0; j < MB; ++j)
                    o[s][j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                            rs, (s0 + s) * bytes + (uint32_t)(j * kSkinnyThreads + threadIdx.x) * 4u,
                                                            0, kDeviceScope));
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int j = 0; j < MB; ++j) z[j] += o[s][j];
        }
        if (threadIdx.x == 0) __hip_atomic_store(counters + u, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (n0 + col >= a.n || row >= rows) return;
    if constexpr (ADAPT) add_low_rank<DT, B_NK, MB>(z, ad, tile.begin + row, tile.end, n0 + col, a.n);
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        if (16 * j + row >= rows) continue;
        const int m = tile.begin + 16 * j + row;
        a.c[(size_t)m * n_len + (size_t)(n0 + col)] = act_cast<DT>(z[j], a.relu != 0);
    }
}

}  // namespace gemm_relu_hip
