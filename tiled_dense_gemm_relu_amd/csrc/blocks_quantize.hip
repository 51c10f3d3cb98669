// The quantizer of gemm_relu_blocks.h: 8-bit values and fp32 scales of a 16-bit
// matrix, by blocks of 128 along rows, along columns (transposed), or by tiles.
//
// It is bound by memory: 2 bytes an element in (4 with a mask), 1 out for each
// direction.  A workgroup takes a tile of 128 x 128 into registers once and
// writes both directions from there: a thread holds 8 x 8 elements, so the
// conversion of two rows' elements of a column fills two bytes of the transposed
// row, and the transposed tile passes through LDS as 8-byte pieces.
#include "groups_kernels.hpp"
#include "blocks_table.hpp"

namespace gemm_relu_hip {
namespace {


template <int FORMAT>
constexpr float kLargest = FORMAT == kE4M3 ? 448.0f : 57344.0f;
constexpr float kSmallestMagnitude = 0x1p-80f;

struct Scale {
    float s, inverse;
};

// The scale of a block whose largest finite magnitude has the bits `amax` (of a 16-bit float).
template <int DT, int FORMAT>
__device__ __forceinline__ Scale make_scale(uint32_t amax, int power_of_two)
{
    float s = fmaxf(to_float<DT>((uint16_t)amax), kSmallestMagnitude) / kLargest<FORMAT>;
    if (power_of_two) {      // (never subnormal: at least 2^-80 / 2^16)
        const uint32_t bits = __builtin_bit_cast(uint32_t, s);
        s = __builtin_bit_cast(float, (bits + 0x7fffffu) & 0xff800000u);
    }
    return Scale{s, 1.0f / s};
}

// x / s, correctly rounded: the product with the rounded reciprocal is off by at
// most two units in the last place, and one step with its exact remainder
// corrects that.  (x has 8 or 11 bits, and so has the magnitude that s was made
// of: every pair of them has been compared with the exact quotient.)  Infinities
// and NaN are left as they are (their remainder is not a number).
__device__ __forceinline__ float divide(float x, Scale c)
{
    const float t = x * c.inverse;
    const float q = __builtin_fmaf(__builtin_fmaf(-t, c.s, x), c.inverse, t);
    return __builtin_fabsf(x) < __builtin_inff() ? q : x;
}

// Two 8-bit values in the low or high half of `old`.
template <int FORMAT, bool HIGH>
__device__ __forceinline__ uint32_t to_8bit(float x, float y, uint32_t old)
{
    if constexpr (FORMAT == kE4M3)
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, y, (int)old, HIGH);
    else
        return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(x, y, (int)old, HIGH);
}

// The magnitude's bits of a 16-bit float, 0 where it is infinite or NaN.
template <int DT>
__device__ __forceinline__ uint32_t finite_magnitude(uint16_t h)
{
    constexpr uint32_t inf = DT == kF16 ? 0x7c00u : 0x7f80u;
    const uint32_t m = h & 0x7fffu;
    return m < inf ? m : 0u;
}

// Rows of a transposed tile in LDS, 8-byte pieces.
constexpr int kTransposedRow = 136;

template <int DT, int FORMAT, bool TILES>
__global__ __launch_bounds__(kQuantizeThreads) void quantize_blocks(QuantizeArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t turned[kBlock * kTransposedRow];
    __shared__ uint32_t column_amax[4][kBlock];
    __shared__ Scale column_scale[kBlock];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cc = tid & 15, rr = tid >> 4;
    const int64_t tiles = (int64_t)a.tiles_r * a.tiles_c, matrix = (int64_t)blockIdx.x / tiles;
    const int tile = (int)((int64_t)blockIdx.x - matrix * tiles), tr = tile / a.tiles_c, tc = tile % a.tiles_c;
    const int row = tr * kBlock + 8 * rr, col = tc * kBlock + 8 * cc;      // this thread's 8 x 8 elements
    const uint16_t* const x = a.x + (size_t)matrix * (size_t)a.rows * (size_t)a.cols;
    const uint16_t* const mask = a.mask ? a.mask + (size_t)matrix * (size_t)a.rows * (size_t)a.cols : nullptr;

    u32x4 v[8];
    if (a.vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const size_t at = (size_t)(row + i) * (size_t)a.cols + (size_t)col;
            const bool inside = row + i < a.rows && col < a.cols;
            v[i] = inside ? *reinterpret_cast<const u32x4*>(x + at) : u32x4{0u, 0u, 0u, 0u};
            if (mask && inside) v[i] = mask_chunk<DT>(v[i], *reinterpret_cast<const u32x4*>(mask + at));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t pair = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = col + 2 * w + h;
                    const size_t at = (size_t)(row + i) * (size_t)a.cols + (size_t)c;
                    if (row + i < a.rows && c < a.cols) {
                        const uint16_t e = mask ? mask_one<DT>(x[at], mask[at]) : x[at];
                        pair |= (uint32_t)e << (16 * h);
                    }
                }
                v[i][w] = pair;
            }
    }
    auto element = [&](int i, int j) { return (uint16_t)(v[i][j >> 1] >> (16 * (j & 1))); };

    uint32_t row_amax[8];
    if (TILES || a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, finite_magnitude<DT>(element(i, j)));
#pragma unroll
            for (int d = 1; d < 16; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
            row_amax[i] = m;
        }
    }
    Scale whole;      // TILES: the tile's
    if constexpr (TILES) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, row_amax[i]);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (lane == 0) column_amax[wave][0] = m;
        __syncthreads();
        m = max(max(column_amax[0][0], column_amax[1][0]), max(column_amax[2][0], column_amax[3][0]));
        whole = make_scale<DT, FORMAT>(m, a.power_of_two);
        if (tid == 0) {
            if (a.q) a.s[matrix * tiles + (int64_t)tr * a.tiles_c + tc] = whole.s;
            if (a.qt) a.st[matrix * tiles + (int64_t)tc * a.tiles_r + tr] = whole.s;
        }
    }
    if (a.q) {
        uint8_t* const q = a.q + (size_t)matrix * (size_t)a.rows * (size_t)a.ldq;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (row + i >= a.rows) continue;      // (the 16 threads of a row agree)
            Scale c = whole;
            if constexpr (!TILES) {
                c = make_scale<DT, FORMAT>(row_amax[i], a.power_of_two);
                if (cc == i) a.s[(matrix * a.tiles_c + tc) * (int64_t)a.rows + row + i] = c.s;
            }
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                w[p] = to_8bit<FORMAT, false>(divide(to_float<DT>(element(i, 4 * p)), c), divide(to_float<DT>(element(i, 4 * p + 1)), c), 0);
                w[p] = to_8bit<FORMAT, true>(divide(to_float<DT>(element(i, 4 * p + 2)), c), divide(to_float<DT>(element(i, 4 * p + 3)), c), w[p]);
            }
            uint8_t* const to = q + (size_t)(row + i) * (size_t)a.ldq + (size_t)col;
            if (col + 8 <= a.cols) {
                *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < a.cols) to[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
    if (!a.qt) return;
    if constexpr (!TILES) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, finite_magnitude<DT>(element(i, j)));
            m = max(m, (uint32_t)__shfl_xor((int)m, 16));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32));
            if (lane < 16) column_amax[wave][8 * cc + j] = m;
        }
        __syncthreads();
        if (tid < kBlock) {
            const uint32_t m = max(max(column_amax[0][tid], column_amax[1][tid]), max(column_amax[2][tid], column_amax[3][tid]));
            const Scale c = make_scale<DT, FORMAT>(m, a.power_of_two);
            column_scale[tid] = c;
            if (tc * kBlock + tid < a.cols)
                a.st[(matrix * a.tiles_r + tr) * (int64_t)a.cols + tc * kBlock + tid] = c.s;
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Scale c = whole;
        if constexpr (!TILES) c = column_scale[8 * cc + j];
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            w[p] = to_8bit<FORMAT, false>(divide(to_float<DT>(element(4 * p, j)), c), divide(to_float<DT>(element(4 * p + 1, j)), c), 0);
            w[p] = to_8bit<FORMAT, true>(divide(to_float<DT>(element(4 * p + 2, j)), c), divide(to_float<DT>(element(4 * p + 3, j)), c), w[p]);
        }
        *reinterpret_cast<u32x2*>(turned + (8 * cc + j) * kTransposedRow + 8 * rr) = u32x2{w[0], w[1]};
    }
    __syncthreads();
    uint8_t* const qt = a.qt + (size_t)matrix * (size_t)a.cols * (size_t)a.ldqt;
    const int r = tr * kBlock + 16 * (tid & 7);                            // 16 rows of X, 8 threads a column
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = 32 * s + (tid >> 3);
        if (tc * kBlock + c >= a.cols || r >= a.rows) continue;
        const uint8_t* const from = turned + c * kTransposedRow + 16 * (tid & 7);
        uint8_t* const to = qt + (size_t)(tc * kBlock + c) * (size_t)a.ldqt + (size_t)r;
        const u32x2 lo = *reinterpret_cast<const u32x2*>(from), hi = *reinterpret_cast<const u32x2*>(from + 8);
        if (r + 16 <= a.rows) {
            *reinterpret_cast<u32x4*>(to) = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            for (int i = 0; i < a.rows - r; ++i) to[i] = from[i];
        }
    }
}

}  // namespace

const void* quantize_kernel(int dtype, int format, int tiles)
{
    static const void* const t[2][2][2] = {
        {{(const void*)quantize_blocks<kF16, kE4M3, false>, (const void*)quantize_blocks<kF16, kE4M3, true>},
         {(const void*)quantize_blocks<kF16, kE5M2, false>, (const void*)quantize_blocks<kF16, kE5M2, true>}},
        {{(const void*)quantize_blocks<kBF16, kE4M3, false>, (const void*)quantize_blocks<kBF16, kE4M3, true>},
         {(const void*)quantize_blocks<kBF16, kE5M2, false>, (const void*)quantize_blocks<kBF16, kE5M2, true>}}};
    return t[dtype][format][tiles];
}

}  // namespace gemm_relu_hip
