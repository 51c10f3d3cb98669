// gfx950 kernels of the products whose rows choose their weights
// (gemm_relu_groups.h): products grouped by expert, their gradients, and
// low-rank adapters beside a shared projection.
//
// The groups' ends are in device memory and the host never learns them.  A
// kernel finds its part of the work itself: lane l of a wave takes group l, a
// scan over the wave turns the groups' row counts into running tile counts,
// and a ballot finds the group that holds a given tile (find_row_tile).
//
// All kernels compute blocks of C^T with 16x16x32 MFMAs (the MFMA "A" operand
// is the weights' side), so lane l of a block holds 4 consecutive columns of
// row l % 16: see store_cols.
#pragma once

#include <type_traits>

#include "gemm_relu_kernels.hpp"
#include "groups_table.hpp"

namespace gemm_relu_hip {

// ---------------------------------------------------------------- row table

// Rows begin .. end - 1 of the matrices, a tile of group `group`; group ==
// groups: rows of no group.  group < 0: there is no such tile.
struct RowTile {
    int group, begin, end;
};

// Inclusive scans of non-negative values over the wave's 64 lanes, by DPP moves:
// within rows of 16 lanes (row_shr 1, 2, 4, 8), then from lane 15 of rows 0 and 2
// to the row after them, and from lane 31 to rows 2 and 3.  Lanes without a
// source get 0.
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op)
{
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
    return op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
}
__device__ __forceinline__ int wave_scan_max(int v)
{
    return wave_scan(v, [](int a, int b) { return max(a, b); });
}
__device__ __forceinline__ int wave_scan_sum(int v)
{
    return wave_scan(v, [](int a, int b) { return a + b; });
}

// The rows of lane l's group g0 + l, for 64 groups from g0 on; `start` is where
// group g0 begins.  Group `groups` is made of the rows past the last end, later
// ones are empty.  The running maximum keeps groups apart whatever `ends` holds.
struct GroupRows {
    int begin, end;
};
__device__ __forceinline__ GroupRows load_group_rows(const int* __restrict__ ends, int groups, int M, int g0,
                                                     int start, int lane)
{
    const int g = g0 + lane;
    int e = M;
    if (g < groups) e = ends ? min(max(ends[g], 0), M) : M;
    e = max(wave_scan_max(e), start);
    return GroupRows{__builtin_amdgcn_update_dpp(start, e, 0x138, 0xf, 0xf, false), e};   // the lane before's end
}

// Tile number `unit` when every group's rows are cut into tiles of `rows` rows.
__device__ inline RowTile find_row_tile(const int* __restrict__ ends, int groups, int M, int rows, int unit, int lane)
{
    int tiles_before = 0, start = 0;
    for (int g0 = 0; g0 <= groups; g0 += 64) {
        const GroupRows r = load_group_rows(ends, groups, M, g0, start, lane);
        const int tiles = (r.end - r.begin + rows - 1) / rows;
        const int incl = tiles_before + wave_scan_sum(tiles);
        const uint64_t mask = __ballot(unit < incl);
        if (mask) {
            const int l = __builtin_ctzll(mask);
            const int begin = __builtin_amdgcn_readlane(r.begin, l) +
                              (unit - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(tiles, l))) * rows;
            return RowTile{g0 + l, begin, min(begin + rows, __builtin_amdgcn_readlane(r.end, l))};
        }
        tiles_before = __builtin_amdgcn_readlane(incl, 63);
        start = __builtin_amdgcn_readlane(r.end, 63);
    }
    return RowTile{-1, 0, 0};
}

// ---------------------------------------------------------------- epilogue

// An fp32 sum in C's dtype (round to nearest even), after ReLU if asked for.
template <int DT>
__device__ __forceinline__ uint16_t act_cast(float x, bool relu)
{
    if (relu) x = x > 0.0f ? x : 0.0f;
    if constexpr (DT == kF16)
        return __builtin_bit_cast(uint16_t, (_Float16)x);
    else
        return __builtin_bit_cast(uint16_t, (__bf16)x);
}

template <int DT>
__device__ __forceinline__ float to_float(uint16_t h)
{
    if constexpr (DT == kF16)
        return (float)__builtin_bit_cast(_Float16, h);
    else
        return __builtin_bit_cast(float, (uint32_t)h << 16);
}

// Store one 16x16 block of C^T: lane l holds row m = (block's first row) + l % 16
// and columns n .. n + 3.  Rows from m_end and columns from n_end on are dropped;
// n_end % 4 == 0 and rows of C are 8-byte aligned.
template <int DT>
__device__ __forceinline__ void store_cols(uint16_t* __restrict__ C, floatx4 acc, int m, int n, int m_end, int n_end,
                                           bool relu)
{
    if (m >= m_end || n >= n_end) return;
    const uint16_t h0 = act_cast<DT>(acc[0], relu), h1 = act_cast<DT>(acc[1], relu);
    const uint16_t h2 = act_cast<DT>(acc[2], relu), h3 = act_cast<DT>(acc[3], relu);
    *reinterpret_cast<u32x2*>(C + (size_t)m * (size_t)n_end + n) =
        u32x2{(uint32_t)h0 | ((uint32_t)h1 << 16), (uint32_t)h2 | ((uint32_t)h3 << 16)};
}

// ---------------------------------------------------------------- rows of any alignment

// A buffer over `bytes` bytes from p (2-byte aligned) on, from the 4-byte
// boundary at or before p: `shift` (0 or 2) goes into every offset.  The last
// dword counts as inside if any byte of it is, which touches no other dword.
struct AnyRsrc {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t shift;
};
__device__ __forceinline__ AnyRsrc make_any_rsrc(const uint16_t* p, uint32_t bytes)
{
    const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(p) & 2u;
    return AnyRsrc{make_rsrc(reinterpret_cast<const uint8_t*>(p) - shift, bytes ? (bytes + shift + 3u) & ~3u : 0u), shift};
}

// 8 consecutive elements at an even byte offset, on their way: the 16 bytes
// from the dword boundary on, and the dword after them, which only elements
// that start inside a dword need.  chunk_value shifts them into place.
struct AnyChunk {
    u32x4 v;
    uint32_t next, bits;
};
__device__ __forceinline__ AnyChunk load_any(const AnyRsrc& r, uint32_t off, bool valid)
{
    const uint32_t o = off + r.shift, at = valid ? o & ~3u : kOobOffset;
    return AnyChunk{__builtin_amdgcn_raw_buffer_load_b128(r.rsrc, at, 0, 0),
                    __builtin_amdgcn_raw_buffer_load_b32(r.rsrc, (o & 2u) ? at + 16u : kOobOffset, 0, 0), (o & 2u) * 8u};
}
__device__ __forceinline__ u32x4 chunk_value(const AnyChunk& c)
{
    return u32x4{__builtin_amdgcn_alignbit(c.v[1], c.v[0], c.bits), __builtin_amdgcn_alignbit(c.v[2], c.v[1], c.bits),
                 __builtin_amdgcn_alignbit(c.v[3], c.v[2], c.bits), __builtin_amdgcn_alignbit(c.next, c.v[3], c.bits)};
}

// The first `valid` of 8 elements, zeros after them.
__device__ __forceinline__ u32x4 keep_first(u32x4 v, int valid)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = valid >= 2 * i + 2 ? v[i] : valid == 2 * i + 1 ? v[i] & 0xffffu : 0u;
    return v;
}

// 2 W consecutive elements from p (2-byte aligned) on, of which the first
// `valid` (at least 1) exist: dword loads of dwords that hold one of them.
template <int W>
__device__ __forceinline__ void load_dwords_any(const uint16_t* p, int valid, uint32_t (&out)[W])
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const int odd = (int)(a >> 1) & 1, last = (odd + valid - 1) >> 1;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a & ~(uintptr_t)3);
    uint32_t d[W + 1];
#pragma unroll
    for (int i = 0; i <= W; ++i) d[i] = q[min(i, last)];
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = __builtin_amdgcn_alignbit(d[i + 1], d[i], 16 * odd);
}

// ---------------------------------------------------------------- ReLU's gradient

// d = dc where c > 0, else +0.0 (c's sign decides: 16-bit floats above zero are
// the patterns 0x0001 .. infinity; NaN counts as not above zero).
template <int DT>
__device__ __forceinline__ uint16_t mask_one(uint16_t dc, uint16_t c)
{
    constexpr uint16_t inf = DT == kF16 ? 0x7c00 : 0x7f80;
    return (uint16_t)(c - 1) < inf ? dc : (uint16_t)0;
}

template <int DT>
__device__ __forceinline__ u32x4 mask_chunk(u32x4 dc, u32x4 c)
{
#pragma unroll
    for (int w = 0; w < 4; ++w)
        dc[w] = (uint32_t)mask_one<DT>((uint16_t)dc[w], (uint16_t)c[w]) |
                ((uint32_t)mask_one<DT>((uint16_t)(dc[w] >> 16), (uint16_t)(c[w] >> 16)) << 16);
    return dc;
}

template <int DT>
__global__ __launch_bounds__(256) void relu_mask(MaskArgs a)
{
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t chunks = a.vec ? a.count / 8 : 0;
    for (int64_t q = first; q < chunks; q += stride) {
        reinterpret_cast<u32x4*>(a.d)[q] =
            mask_chunk<DT>(reinterpret_cast<const u32x4*>(a.dc)[q], reinterpret_cast<const u32x4*>(a.c)[q]);
    }
    for (int64_t q = chunks * 8 + first; q < a.count; q += stride) a.d[q] = mask_one<DT>(a.dc[q], a.c[q]);
}

// A wave takes a row at a time, its lanes 8 elements each.
template <int DT>
__global__ __launch_bounds__(256) void pad_rows(PadArgs a)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < a.rows; row += (int64_t)gridDim.x * 4) {
        const size_t at = (size_t)row * (size_t)a.cols;
        const AnyRsrc rs = make_any_rsrc(a.src + at, (uint32_t)a.cols * 2u);
        const AnyRsrc rm = a.mask ? make_any_rsrc(a.mask + at, (uint32_t)a.cols * 2u) : rs;
        for (int e = 8 * lane; e < a.pitch; e += 512) {
            u32x4 v = chunk_value(load_any(rs, (uint32_t)e * 2u, true));
            if (a.mask) v = mask_chunk<DT>(v, chunk_value(load_any(rm, (uint32_t)e * 2u, true)));
            *reinterpret_cast<u32x4*>(a.dst + (size_t)row * (size_t)a.pitch + e) = keep_first(v, a.cols - e);
        }
    }
}

// ---------------------------------------------------------------- adapters

// Bytes of LDS that add_adapters stages V in, per wave: 32 k of its columns.
template <int FN>
constexpr int kAdapterStrip = 32 * FN * 16 * 2;

// The products of an intermediate's low parts with V, before those of its high parts
// are added: infinities and NaN of V become finite, so that a low part of zero or of
// the other sign does not turn the term into NaN.  Where V is infinite or NaN the
// high part's product is too, and decides.
__device__ __forceinline__ floatx4 finite_low(floatx4 p)
{
    float most = __FLT_MAX__;
    asm("" : "+s"(most));            // one scalar register and its negative, not a literal and a vector register
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_fmed3f(p[e], -most, most);
    return p;
}

// Add the low-rank terms of rows m_base .. (those below m_end) to the first FX
// of FN x FM blocks of C^T, block (i, j): rows m_base + 16j .. +15, columns n_base + 16i .. +15.
//  A row's term is (its intermediate, hi + lo times a power of two) @ (its
// adapter's V).  Rows of a 16-row block may use several adapters:
// for each of them the block's product is computed in registers of its own, and
// a lane takes it over only if its row uses that adapter: rows never see
// another request's weights, not even as 0 * infinity.  (The sums of a block
// are added to acc once, outside all loops: loops that carry acc through them
// made the compiler keep it twice, and spill.)
//  A block whose rows use more than two adapters (single tokens of many
// requests) would read a V for each, one after the other.  Its lanes compute
// their own row's 4 columns instead, by fp32 multiply-adds over the rank, with
// all loads of 8 rank entries in flight together.
template <int DT, bool B_NK, int FX, int FN, int FM>
__device__ __forceinline__ void add_adapters(floatx4 (&acc)[FN][FM], const AdapterArgs& ad, int m_base, int m_end,
                                             int n_base, int N, int lane, uint8_t* strip)
{
    constexpr int ROW = FN * 32;                       // bytes of a strip's row of k
    asm volatile("" : "+v"(lane));   // what follows from it is computed here, not kept through the caller's loop
    const int r16 = lane & 15, kg = lane >> 4, kb = kgroup16(kg);
    const uint32_t t_row = (uint32_t)ad.rank_pad * 4u;
    const __amdgpu_buffer_rsrc_t rt = make_rsrc(ad.t, (uint32_t)m_end * t_row);
#pragma unroll
    for (int j = 0; j < FX; ++j) {
        floatx4 sum[FN];
#pragma unroll
        for (int i = 0; i < FN; ++i) sum[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t m = (uint32_t)(m_base + 16 * j + r16);
        const int id = (int)m < m_end ? ad.row_id[m] : -1;
        const float f = id >= 0 ? ad.factor[m] : 0.0f;
        const uint32_t all = (uint32_t)__ballot(id >= 0) & 0xffffu;    // rows with an adapter
        uint32_t more = all;
        for (int k = 0; k < 2 && more; ++k)
            more &= ~(uint32_t)__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctz(more)));
        uint32_t rest = more ? 0u : all;
        while (rest) {
            const int cur = __builtin_amdgcn_readlane(id, __builtin_ctz(rest));
            rest &= ~(uint32_t)__ballot(id == cur);
            const bool in = id == cur;
            const AnyRsrc rv = make_any_rsrc(
                ad.v + (size_t)cur * (size_t)ad.rank * (size_t)N + (B_NK ? (size_t)n_base * (size_t)ad.rank : 0),
                (uint32_t)(B_NK ? max(0, min(16 * FN, N - n_base)) : N) * (uint32_t)ad.rank * 2u);
            for (int k0 = 0; k0 < ad.rank; k0 += 32) {
                const uint32_t at = in ? m * t_row + (uint32_t)(k0 + 8 * kb) * 2u : kOobOffset;
                const u32x4 t_lo = __builtin_amdgcn_raw_buffer_load_b128(rt, at, 0, 0);
                const u32x4 t_hi = __builtin_amdgcn_raw_buffer_load_b128(rt, at, ad.rank_pad * 2, 0);
                u32x4 v[FN];
                if constexpr (B_NK) {
                    const int k = k0 + 8 * kb;
                    AnyChunk c[FN];
#pragma unroll
                    for (int i = 0; i < FN; ++i)
                        c[i] = load_any(rv, ((uint32_t)(16 * i + r16) * (uint32_t)ad.rank + (uint32_t)k) * 2u, k < ad.rank);
#pragma unroll
                    for (int i = 0; i < FN; ++i) v[i] = keep_first(chunk_value(c[i]), ad.rank - k);
                } else {
                    constexpr int PIECES = ROW / 16, PER_LANE = 32 * PIECES / 64;
                    AnyChunk c[PER_LANE];
#pragma unroll
                    for (int q = 0; q < PER_LANE; ++q) {
                        const int p = lane + 64 * q, k = p / PIECES, n = n_base + 8 * (p % PIECES);
                        c[q] = load_any(rv, ((uint32_t)(k0 + k) * (uint32_t)N + (uint32_t)n) * 2u, k0 + k < ad.rank && n < N);
                    }
#pragma unroll
                    for (int q = 0; q < PER_LANE; ++q) {
                        const int p = lane + 64 * q, k = p / PIECES;
                        *reinterpret_cast<u32x4*>(strip + k * ROW + 16 * ((p % PIECES) ^ b_swizzle<ROW, 16>(k))) = chunk_value(c[q]);
                    }
                    const int krow = 8 * kb + (r16 >> 2);
#pragma unroll
                    for (int i = 0; i < FN; ++i) {
                        const int n = 16 * i + 4 * (r16 & 3);
                        const uint8_t* p = strip + krow * ROW + 16 * ((n >> 3) ^ b_swizzle<ROW, 16>(krow)) + 8 * (r16 & 1);
                        const u32x2 lo = ds_read_tr16(p), hi = ds_read_tr16(p + 4 * ROW);
                        v[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
                    }
                }
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    floatx4 p = mfma_16x16x32<DT>(v[i], t_lo, floatx4{0.0f, 0.0f, 0.0f, 0.0f});
                    p = mfma_16x16x32<DT>(v[i], t_hi, finite_low(p));
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[i][e] = in ? sum[i][e] + f * p[e] : sum[i][e];
                }
            }
        }
        if (more && id >= 0) {
            auto half = [](uint32_t d, int e) { return to_float<DT>((uint16_t)(d >> (16 * (e & 1)))); };
            const uint16_t* vp = ad.v + (size_t)id * (size_t)ad.rank * (size_t)N;
            constexpr int SIDE = FN < 2 ? FN : 2;       // 16-column blocks whose loads are in flight together
#pragma unroll 1
            for (int r0 = 0; r0 < ad.rank; r0 += 8) {
                const int valid = min(8, ad.rank - r0);
                const uint32_t at = m * t_row + (uint32_t)r0 * 2u;
                const u32x4 t_lo = __builtin_amdgcn_raw_buffer_load_b128(rt, at, 0, 0);
                const u32x4 t_hi = __builtin_amdgcn_raw_buffer_load_b128(rt, at, ad.rank_pad * 2, 0);
#pragma unroll
                for (int i0 = 0; i0 < FN; i0 += SIDE) {
                    uint32_t w[SIDE][8][2];             // [k] pairs of columns, or [4 pairs of k, 2 columns at a time]
#pragma unroll
                    for (int i = 0; i < SIDE; ++i) {
                        const int n = low_rank_column(n_base + 16 * (i0 + i) + 4 * kg, N, !B_NK && ad.v_fast), cols = min(4, N - n);
                        if constexpr (B_NK) {
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const uint16_t* p = vp + (size_t)(n + min(x, cols - 1)) * (size_t)ad.rank + r0;
                                uint32_t q[4];
                                if (ad.v_fast) {
                                    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
                                    q[0] = v[0], q[1] = v[1], q[2] = v[2], q[3] = v[3];
                                } else {
                                    load_dwords_any<4>(p, valid, q);
                                }
#pragma unroll
                                for (int h = 0; h < 4; ++h) w[i][2 * x + (h >> 1)][h & 1] = q[h];
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint16_t* p = vp + (size_t)(r0 + min(e, valid - 1)) * (size_t)N + n;
                                if (ad.v_fast) {
                                    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
                                    w[i][e][0] = v[0], w[i][e][1] = v[1];
                                } else {
                                    load_dwords_any<2>(p, cols, w[i][e]);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float z = e < valid ? f * (half(t_hi[e / 2], e) + half(t_lo[e / 2], e)) : 0.0f;
#pragma unroll
                        for (int i = 0; i < SIDE; ++i)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float v = B_NK ? half(w[i][2 * x + (e >> 2)][(e >> 1) & 1], e) : half(w[i][e][x / 2], x);
                                sum[i0 + i][x] += e < valid ? z * v : 0.0f;
                            }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < FN; ++i) acc[i][j] += sum[i];
    }
}

// The intermediates of the low-rank terms.  For row m of a segment with adapter
// i, z = scales[i] * (X[m] @ U_i) is summed in fp32 and stored as
//     z = factor[m] * (t[m][lo][..] + t[m][hi][..]),  zeros from rank to rank_pad,
// factor a power of two of the row's largest |z|, hi the nearest 16-bit value
// to z / factor (at most 1 in size) and lo that to what is left.  row_id[m] is
// the row's adapter, -1 for none.  Two 16-bit parts, since the second product's
// matrix instructions take 16-bit operands: off by at most 2^-16 of z in bf16, 2^-22
// of z and 2^-25 of factor in fp16, where the output's own rounding is 2^-8 or 2^-11
// (a third part would hold fp32's 24 bits, for half as many low-rank products again).
//  One workgroup per 16 MB rows of a segment and part of K, CHUNKS times 32
// columns of rank at a time: its 8 waves take pieces of 128 k in turn, each with all its loads in
// flight at once, and their sums are added in wave order in LDS.  With few rows
// K is cut into `splits` parts, whose sums go through device memory
// (device-scope accesses: the parts run on different XCDs); the part that
// counts itself last adds them in part order and finishes.  Nothing waits for
// another workgroup.
template <int DT, bool U_NK, int CHUNKS, int MB>
__global__ __launch_bounds__(kShrinkThreads) void adapter_shrink(ShrinkArgs a)
{
    constexpr int WAVES = kShrinkThreads / 64, STEPS = kShrinkK / 32, ROW = kShrinkCols * 2;
    constexpr int kDeviceScope = 16;   // cache policy sc1
    constexpr int ROWS = MB * kShrinkRows, SUMS = MB * kShrinkThreads;
    __shared__ float part[WAVES][kShrinkCols][ROWS + 1];
    extern __shared__ float sums[];    // [32 columns][SUMS]: each thread's own
    __shared__ __attribute__((aligned(16))) uint8_t strips[U_NK ? 16 : WAVES * 32 * ROW];
    __shared__ int before;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const RowTile tile = find_row_tile(a.ends, a.segments, a.m, ROWS, blockIdx.x, lane);
    if (tile.group < 0) return;
    const int rows = tile.end - tile.begin;
    int id = tile.group < a.segments ? a.ids[tile.group] : -1;
    if (id >= a.adapters || id < 0) id = -1;
    if (blockIdx.y == 0 && (int)threadIdx.x < rows) a.row_id[tile.begin + threadIdx.x] = id;
    if (id < 0) return;
    const int r16 = lane & 15, kb = kgroup16(lane >> 4);
    const size_t k_len = (size_t)a.k, rank = (size_t)a.rank;
    const int chunks = (a.rank + kShrinkCols - 1) / kShrinkCols;
    // 512 threads: 16 rows x 32 columns of each block of rows; a row's 32 columns are one half of a wave
    const int row = threadIdx.x >> 5, col = threadIdx.x & 31;
    auto sum_at = [&](int c, int j) { return c * SUMS + j * kShrinkThreads + (int)threadIdx.x; };

    const AnyRsrc rx = make_any_rsrc(a.x + (size_t)tile.begin * k_len, (uint32_t)rows * (uint32_t)a.k * 2u);
    uint8_t* strip = strips + (U_NK ? 0 : wave * 32 * ROW);
    const int pieces = (a.k + kShrinkK - 1) / kShrinkK, splits = (int)gridDim.y;
    const int p_begin = (int)((int64_t)pieces * blockIdx.y / splits) + wave;
    const int p_end = (int)((int64_t)pieces * (blockIdx.y + 1) / splits);
    for (int c0 = 0; c0 < chunks; c0 += CHUNKS) {
        const int r_base = c0 * kShrinkCols;
        // U stored (rank, K): rows r_base .. of U^T
        const AnyRsrc ru = make_any_rsrc(a.u + (size_t)id * k_len * rank + (U_NK ? (size_t)r_base * k_len : 0),
                                         (uint32_t)(U_NK ? min(CHUNKS * kShrinkCols, a.rank - r_base) : a.rank) * (uint32_t)a.k * 2u);
        floatx4 acc[CHUNKS][2][MB];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int j = 0; j < MB; ++j) acc[c][0][j] = acc[c][1][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int p = p_begin; p < p_end; p += WAVES) {
            const int k0 = p * kShrinkK;
            AnyChunk x[STEPS][MB], u[STEPS][CHUNKS][2];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int k = k0 + 32 * s + 8 * kb;
#pragma unroll
                for (int j = 0; j < MB; ++j)
                    x[s][j] = load_any(rx, ((uint32_t)(16 * j + r16) * (uint32_t)a.k + (uint32_t)k) * 2u, k < a.k);
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (U_NK) {
                            const int r = c * kShrinkCols + 16 * i + r16;
                            u[s][c][i] = load_any(ru, ((uint32_t)r * (uint32_t)a.k + (uint32_t)k) * 2u, k < a.k && r_base + r < a.rank);
                        } else {
                            const int kr = k0 + 32 * s + 16 * i + (lane >> 2), r = r_base + c * kShrinkCols + 8 * (lane & 3);
                            u[s][c][i] = load_any(ru, ((uint32_t)kr * (uint32_t)a.rank + (uint32_t)r) * 2u, kr < a.k && r < a.rank);
                        }
                    }
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int valid = a.k - (k0 + 32 * s + 8 * kb);
                u32x4 xv[MB];
#pragma unroll
                for (int j = 0; j < MB; ++j) xv[j] = keep_first(chunk_value(x[s][j]), valid);
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c) {
                    u32x4 uv[2];
                    if constexpr (U_NK) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) uv[i] = keep_first(chunk_value(u[s][c][i]), valid);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int kr = 16 * i + (lane >> 2);
                            *reinterpret_cast<u32x4*>(strip + kr * ROW + 16 * ((lane & 3) ^ b_swizzle<ROW, 16>(kr))) = chunk_value(u[s][c][i]);
                        }
                        const int kr = 8 * kb + (r16 >> 2);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = 16 * i + 4 * (r16 & 3);
                            const uint8_t* q = strip + kr * ROW + 16 * ((r >> 3) ^ b_swizzle<ROW, 16>(kr)) + 8 * (r16 & 1);
                            const u32x2 lo = ds_read_tr16(q), hi = ds_read_tr16(q + 4 * ROW);
                            uv[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < MB; ++j) acc[c][i][j] = mfma_16x16x32<DT>(uv[i], xv[j], acc[c][i][j]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            if (c0 + c >= chunks) break;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < MB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) part[wave][16 * i + 4 * (lane >> 4) + e][16 * j + r16] = acc[c][i][j][e];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                float z = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) z += part[w][col][16 * j + row];
                sums[sum_at(c0 + c, j)] = z;
            }
            __syncthreads();
        }
    }
    if (splits > 1) {
        // part s of this row tile, 32 columns c: SUMS floats at (s * chunks + c) * SUMS
        const uint32_t bytes = (uint32_t)chunks * SUMS * 4u;
        const __amdgpu_buffer_rsrc_t rs =
            make_rsrc(a.part + (size_t)blockIdx.x * (size_t)splits * (bytes / 4), (uint32_t)splits * bytes);
        for (int c = 0; c < chunks; ++c)
#pragma unroll
            for (int j = 0; j < MB; ++j)
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, sums[sum_at(c, j)]), rs,
                                                      blockIdx.y * bytes + (uint32_t)sum_at(c, j) * 4u, 0, kDeviceScope);
        wait_vmcnt<0>();               // this wave's sums have reached device scope
        __syncthreads();
        if (threadIdx.x == 0)
            before = __hip_atomic_fetch_add(a.counters + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (before != splits - 1) return;
        asm volatile("" ::: "memory");   // the loads below stay after the count that allowed them
        for (int c = 0; c < chunks; ++c)
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                float z = 0.0f;
                for (int s0 = 0; s0 < splits; s0 += 4) {
                    float o[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s)   // parts past the last are out of range: zero
                        o[s] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                             rs, (uint32_t)(s0 + s) * bytes + (uint32_t)sum_at(c, j) * 4u, 0, kDeviceScope));
#pragma unroll
                    for (int s = 0; s < 4; ++s) z += o[s];
                }
                sums[sum_at(c, j)] = z;
            }
        if (threadIdx.x == 0) __hip_atomic_store(a.counters + blockIdx.x, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const float scale = a.scales[id];
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        float top = 0.0f;
        for (int c = 0; c < chunks; ++c) {
            // columns past rank are zero, whatever X holds (0 * infinity is not)
            const float z = c * kShrinkCols + col < a.rank ? sums[sum_at(c, j)] * scale : 0.0f;
            sums[sum_at(c, j)] = z;
            top = fmaxf(top, fabsf(z) < __builtin_inff() ? fabsf(z) : 0.0f);
        }
#pragma unroll
        for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
        // 2^e > top, the largest finite entry: the scaled values are below 1.  Zeros
        // keep factor 1; e stays where 2^-e is a normal number.
        int e = 0;
        if (top > 0.0f) {
            (void)frexpf(top, &e);
            e = min(max(e, -125), 125);
        }
        if (16 * j + row >= rows) continue;
        const size_t m = (size_t)(tile.begin + 16 * j + row);
        uint16_t* t = a.t + m * (size_t)(2 * a.rank_pad) + col;
        for (int c = 0; c < a.rank_pad / kShrinkCols; ++c, t += kShrinkCols) {
            const float scaled = c < chunks ? ldexpf(sums[sum_at(c, j)], -e) : 0.0f;
            const uint16_t hi = act_cast<DT>(scaled, false);
            const float rest = scaled - to_float<DT>(hi);
            t[a.rank_pad] = hi;
            // an infinite hi leaves inf - inf: such an entry has no second part
            t[0] = fabsf(scaled) < __builtin_inff() ? act_cast<DT>(rest, false) : (uint16_t)0;
        }
        if (col == 0) a.factor[m] = ldexpf(1.0f, e);
    }
}

}  // namespace gemm_relu_hip
