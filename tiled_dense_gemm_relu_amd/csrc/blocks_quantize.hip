// The quantizer of gemm_relu_blocks.h: 8-bit values and fp32 scales of a 16-bit
// matrix, by blocks of 128 along rows, along columns (transposed), or by tiles.
//
// It is bound by memory: 2 bytes an element in (4 with a mask), 1 out for each
// direction.  A workgroup takes a tile of 128 x 128 into registers once and
// writes both directions from there: a thread holds 8 x 8 elements, so the
// conversion of two rows' elements of a column fills two bytes of the transposed
// row, and the transposed tile passes through LDS as 8-byte pieces.  Loads that do not
// stay in the caches leave them to what is written, which the product reads next
// (8192 x 4096 with a mask, both ways, over four matrices in turn: 46-47 -> 43 us, 192 MiB,
// and a layer's forward and backward pass around it 477 -> 460; stores that do not stay: 44,
// but 499 for the layer).
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
// of: every pair of them has been compared with the exact quotient.)  The remainder is
// taken with its sign turned: that of a zero is then +0, which leaves a quotient of -0
// as it is.  With CHECK infinities and NaN are left as they are (their remainder is not
// a number).
template <bool CHECK>
__device__ __forceinline__ float divide(float x, Scale c)
{
    const float t = x * c.inverse;
    const float q = __builtin_fmaf(-__builtin_fmaf(t, c.s, -x), c.inverse, t);
    return !CHECK || __builtin_fabsf(x) < __builtin_inff() ? q : x;
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

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
// The largest within 16 lanes, in all of them.
__device__ __forceinline__ uint32_t row_max_pairs(uint32_t v)
{
    v = max_pairs(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));   // row_ror 1, 2, 4, 8
    v = max_pairs(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
    v = max_pairs(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
    return max_pairs(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));
}
// The largest over the wave's 4 rows of 16 lanes, in all of them.
__device__ __forceinline__ uint32_t column_max_pairs(uint32_t v)
{
    v = max_pairs(v, (uint32_t)__shfl_xor((int)v, 16));
    return max_pairs(v, (uint32_t)__shfl_xor((int)v, 32));
}

// The magnitudes of a pair of 16-bit floats, 0 where infinite or NaN.
template <int DT>
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t pair)
{
    constexpr uint32_t inf = DT == kF16 ? 0x7c00u : 0x7f80u;
    const uint32_t m = pair & 0x7fff7fffu;
    return ((m & 0xffffu) < inf ? m & 0xffffu : 0u) | ((m >> 16) < inf ? m & 0xffff0000u : 0u);
}

// Rows of a transposed tile in LDS, 8-byte pieces.
constexpr int kTransposedRow = 136;

struct Shared {
    __attribute__((aligned(16))) uint8_t turned[kBlock * kTransposedRow];
    uint32_t column_amax[4][kBlock / 2];      // pairs
    Scale row_scale[kBlock], column_scale[kBlock];
};

// What a thread does with its 8 x 8 elements (v[row]: 4 pairs) at (row, col).
//  CHECK: some of the tile's are infinite or NaN.
template <int DT, int FORMAT, bool TILES, bool CHECK>
__device__ __forceinline__ void quantize_tile(const QuantizeArgs& a, const u32x4 (&v)[8], Shared& sh, int64_t matrix, int tr, int tc)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cc = tid & 15, rr = tid >> 4;
    const int row = tr * kBlock + 8 * rr, col = tc * kBlock + 8 * cc;
    auto element = [&](int i, int j) { return to_float<DT>((uint16_t)(v[i][j >> 1] >> (16 * (j & 1)))); };
    auto magnitudes = [&](int i, int w) { return CHECK ? finite_magnitudes<DT>(v[i][w]) : v[i][w] & 0x7fff7fffu; };

    // pairs of columns: the largest of this thread's rows
    uint32_t down[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        down[w] = magnitudes(0, w);
#pragma unroll
        for (int i = 1; i < 8; ++i) down[w] = max_pairs(down[w], magnitudes(i, w));
    }
    Scale whole;      // TILES: the tile's
    if constexpr (TILES) {
        uint32_t m = max_pairs(max_pairs(down[0], down[1]), max_pairs(down[2], down[3]));
        m = column_max_pairs(row_max_pairs(m));
        if (lane == 0) sh.column_amax[wave][0] = max(m & 0xffffu, m >> 16);
        __syncthreads();
        m = max(max(sh.column_amax[0][0], sh.column_amax[1][0]), max(sh.column_amax[2][0], sh.column_amax[3][0]));
        whole = make_scale<DT, FORMAT>(m, a.power_of_two);
        if (tid == 0) {
            const int64_t tiles = (int64_t)a.tiles_r * a.tiles_c;
            if (a.q) a.s[matrix * tiles + (int64_t)tr * a.tiles_c + tc] = whole.s;
            if (a.qt) a.st[matrix * tiles + (int64_t)tc * a.tiles_r + tr] = whole.s;
        }
    }
    if (a.q) {
        if constexpr (!TILES) {
            // Two rows' largest in a register, then one row's scale a lane, by way of LDS
            // to the 16 lanes of the row (all in one wave, whose LDS accesses are in order).
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                uint32_t m[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m[h] = max_pairs(max_pairs(magnitudes(i + h, 0), magnitudes(i + h, 1)), max_pairs(magnitudes(i + h, 2), magnitudes(i + h, 3)));
                    m[h] = max(m[h] & 0xffffu, m[h] >> 16);
                }
                const uint32_t both = row_max_pairs(m[0] | (m[1] << 16));
                if ((cc & 7) >> 1 == i >> 1) mine = (cc & 1) ? both >> 16 : both & 0xffffu;
            }
            if (cc < 8) {
                const Scale c = make_scale<DT, FORMAT>(mine, a.power_of_two);
                sh.row_scale[8 * rr + cc] = c;
                if (row + cc < a.rows) a.s[(matrix * a.tiles_c + tc) * (int64_t)a.rows + row + cc] = c.s;
            }
            __builtin_amdgcn_wave_barrier();
        }
        uint8_t* const q = a.q + (size_t)matrix * (size_t)a.rows * (size_t)a.ldq;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            Scale c = whole;
            if constexpr (!TILES) c = sh.row_scale[8 * rr + i];
            uint32_t w[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                w[p] = to_8bit<FORMAT, false>(divide<CHECK>(element(i, 4 * p), c), divide<CHECK>(element(i, 4 * p + 1), c), 0);
                w[p] = to_8bit<FORMAT, true>(divide<CHECK>(element(i, 4 * p + 2), c), divide<CHECK>(element(i, 4 * p + 3), c), w[p]);
            }
            if (row + i >= a.rows) continue;
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
        for (int w = 0; w < 4; ++w) {
            const uint32_t m = column_max_pairs(down[w]);
            if (lane < 16) sh.column_amax[wave][4 * cc + w] = m;
        }
        __syncthreads();
        if (tid < kBlock) {
            const uint32_t m = max_pairs(max_pairs(sh.column_amax[0][tid >> 1], sh.column_amax[1][tid >> 1]),
                                         max_pairs(sh.column_amax[2][tid >> 1], sh.column_amax[3][tid >> 1]));
            const Scale c = make_scale<DT, FORMAT>((tid & 1) ? m >> 16 : m & 0xffffu, a.power_of_two);
            sh.column_scale[tid] = c;
            if (tc * kBlock + tid < a.cols) a.st[(matrix * a.tiles_r + tr) * (int64_t)a.cols + tc * kBlock + tid] = c.s;
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Scale c = whole;
        if constexpr (!TILES) c = sh.column_scale[8 * cc + j];
        uint32_t w[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            w[p] = to_8bit<FORMAT, false>(divide<CHECK>(element(4 * p, j), c), divide<CHECK>(element(4 * p + 1, j), c), 0);
            w[p] = to_8bit<FORMAT, true>(divide<CHECK>(element(4 * p + 2, j), c), divide<CHECK>(element(4 * p + 3, j), c), w[p]);
        }
        *reinterpret_cast<u32x2*>(sh.turned + (8 * cc + j) * kTransposedRow + 8 * rr) = u32x2{w[0], w[1]};
    }
    __syncthreads();
    uint8_t* const qt = a.qt + (size_t)matrix * (size_t)a.cols * (size_t)a.ldqt;
    const int r = tr * kBlock + 16 * (tid & 7);                            // 16 rows of X, 8 threads a column
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = 32 * s + (tid >> 3);
        if (tc * kBlock + c >= a.cols || r >= a.rows) continue;
        const uint8_t* const from = sh.turned + c * kTransposedRow + 16 * (tid & 7);
        uint8_t* const to = qt + (size_t)(tc * kBlock + c) * (size_t)a.ldqt + (size_t)r;
        const u32x2 lo = *reinterpret_cast<const u32x2*>(from), hi = *reinterpret_cast<const u32x2*>(from + 8);
        if (r + 16 <= a.rows) {
            *reinterpret_cast<u32x4*>(to) = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            for (int i = 0; i < a.rows - r; ++i) to[i] = from[i];
        }
    }
}

// VEC: x and the mask allow 16-byte loads of 8 elements.
template <int DT, int FORMAT, bool TILES, bool VEC>
__global__ __launch_bounds__(kQuantizeThreads, 4) void quantize_blocks(QuantizeArgs a)
{
    int64_t block = blockIdx.x;
    if (a.apart > 0) {
        if (block < a.apart) a.qt = nullptr;
        else a.q = nullptr;
        block = block < a.apart ? block : block - a.apart;
    }
    __shared__ Shared sh;
    const int tid = threadIdx.x, cc = tid & 15, rr = tid >> 4;
    const int64_t tiles = (int64_t)a.tiles_r * a.tiles_c, matrix = block / tiles;
    const int tile = (int)(block - matrix * tiles), tr = tile / a.tiles_c, tc = tile % a.tiles_c;
    // This thread's 8 x 8 elements.  The tile's rows begin inside 2^28 bytes of each other.
    const int row = 8 * rr, col = 8 * cc, rows = min(kBlock, a.rows - tr * kBlock), cols = min(kBlock, a.cols - tc * kBlock);
    const size_t origin = ((size_t)matrix * (size_t)a.rows + (size_t)tr * kBlock) * (size_t)a.cols + (size_t)tc * kBlock;
    const uint32_t bytes = ((uint32_t)(rows - 1) * (uint32_t)a.cols + (uint32_t)cols) * 2u;
    const uint16_t* const mask = a.mask ? a.mask + origin : a.x + origin;
    u32x4 v[8];
    if constexpr (VEC) {
        constexpr int kNonTemporal = 2;   // cache policy nt
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + origin, bytes), rm = make_rsrc(mask, bytes);
        u32x4 m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = row + i < rows && col < cols ? ((uint32_t)(row + i) * (uint32_t)a.cols + (uint32_t)col) * 2u : kOobOffset;
            v[i] = __builtin_amdgcn_raw_buffer_load_b128(rx, at, 0, kNonTemporal);
            if (a.mask) m[i] = __builtin_amdgcn_raw_buffer_load_b128(rm, at, 0, kNonTemporal);
        }
        if (a.mask) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mask_chunk<DT>(v[i], m[i]);
        }
    } else {
        // rows of any length: dwords, shifted into place, zeros behind the row
        const AnyRsrc rx = make_any_rsrc(a.x + origin, bytes), rm = make_any_rsrc(mask, bytes);
        AnyChunk x[8], m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = ((uint32_t)(row + i) * (uint32_t)a.cols + (uint32_t)col) * 2u;
            const bool inside = row + i < rows && col < cols;
            x[i] = load_any(rx, at, inside);
            if (a.mask) m[i] = load_any(rm, at, inside);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u32x4 e = chunk_value(x[i]);
            if (a.mask) e = mask_chunk<DT>(e, chunk_value(m[i]));
            v[i] = keep_first(e, row + i < rows ? cols - col : 0);
        }
    }
    // Whether all of the tile's elements are finite, which saves their being asked for.
    constexpr uint32_t inf = DT == kF16 ? 0x7c00u : 0x7f80u;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) most = max_pairs(most, v[i][w] & 0x7fff7fffu);
    const bool finite = (most & 0xffffu) < inf && (most >> 16) < inf;
    if (__syncthreads_and(finite)) quantize_tile<DT, FORMAT, TILES, false>(a, v, sh, matrix, tr, tc);
    else quantize_tile<DT, FORMAT, TILES, true>(a, v, sh, matrix, tr, tc);
}

template <int DT, int FORMAT>
const void* pick(int tiles, int vec)
{
    if (tiles) return vec ? (const void*)quantize_blocks<DT, FORMAT, true, true> : (const void*)quantize_blocks<DT, FORMAT, true, false>;
    return vec ? (const void*)quantize_blocks<DT, FORMAT, false, true> : (const void*)quantize_blocks<DT, FORMAT, false, false>;
}

}  // namespace

const void* quantize_kernel(int dtype, int format, int tiles, int vec)
{
    if (dtype == kF16) return format == kE4M3 ? pick<kF16, kE4M3>(tiles, vec) : pick<kF16, kE5M2>(tiles, vec);
    return format == kE4M3 ? pick<kBF16, kE4M3>(tiles, vec) : pick<kBF16, kE5M2>(tiles, vec);
}

}  // namespace gemm_relu_hip
