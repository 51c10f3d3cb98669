// The product of 8-bit matrices scaled by blocks of 128 (gemm_relu_blocks.h), on
// tiles whose operands stream into LDS by DMA.
//
// One v_mfma_f32_16x16x128_f8f6f4 sums a whole scale block of 128 k for 16 x 16
// outputs, at twice the 16-bit rate.  Its result goes, times the block's two
// scales, into fp32 sums in registers: 4 multiply-adds a lane beside 32 cycles of
// the matrix unit, which run on the vector unit meanwhile.
//
// A stage is 128 k of the tile's rows of A and B, 128 bytes a row, swizzled and
// read as the 16-bit kernels' (a_swizzle<128>), and the scales of those rows and
// columns as floats: with scales by tiles every lane of the scales' DMA fetches
// its column's tile, so both forms look alike in LDS.  They are split into factors and
// exponents (split_scale): by the wave that brought them, in LDS, for all; in the 64
// tile by each compute wave, in registers, as there the waves that load have no time to
// spare.  us in LDS and in registers: tiles of 64, 64 x 4096 x 4096 17.0 / 15.8, 512 x 2048 x
// 2048 11.8 / 10.8; of 128, 32 groups of 128 rows x 2048 x 2048 39.2 / 39.2, with scales of B
// by rows 65 / 82.
//
// The 256 tile at 8192^3 on normal data: 483-496 us, 2.22-2.27 PFLOP/s, where a library
// product with one scale a matrix takes 410-419.  With scales multiplied as they are, which
// loses what lies outside a float's range, it takes 472-478 on the same card; without the
// additions 428 then, without DMA 392; loads by all waves with one barrier a step, and matrix instructions
// interleaved with additions, are what it got there by.  The smaller tiles have waves
// that only load: 64 groups of 64 rows x 2048 x 4096 112-116 us, 4.8 TB/s (109 with scales
// multiplied as they are).
#pragma once

#include "blocks_bytes.hpp"
#include "groups_dma.hpp"
#include "blocks_table.hpp"

namespace gemm_relu_hip {

typedef int int32x8_t __attribute__((ext_vector_type(8)));

// A scale as m 2^(e - 127), exactly: e, for the matrix instruction, has what the scale's
// exponent is beyond -40 .. 40, so the product of two m is a normal float (if neither scale
// is zero, infinite or NaN, as which m is the same).  A block's sum, 2^-32 to 2^39, and its
// partial sums stay normal when they are multiplied by the two powers of two, wherever the
// scales' own product is normal: the bits are then those of sums multiplied afterwards.
struct SplitScale {
    float m;
    uint32_t e;
};
__device__ __forceinline__ SplitScale split_scale(float s)
{
    const int exponent = min((int)((__builtin_bit_cast(uint32_t, s) >> 23) & 0xffu), 254) - 127;
    const int moved = exponent - min(max(exponent, -40), 40);
    return SplitScale{__builtin_ldexpf(s, -moved), (uint32_t)(moved + 127)};
}

// 16 x 16 fp32 sums over 128 k, times two powers of two: `w` of format FW, `x` of format
// FX.  A lane holds 32 bytes of one row of each; which k those are only has to agree
// between them.  The exponents of a lane's rows are byte `bw` of `ew` and byte `bx` of `ex`
// (constants once loops are unrolled).  The product of two scales alone could be subnormal,
// zero or infinite where the result is not.  (This costs 8192^3 3%, the 128 tile with scales
// of B by rows 14%; a second body of the loop for steps whose scales need it, 30%, by its
// registers.)
template <int FW, int FX>
__device__ __forceinline__ floatx4 mfma_block(int32x8_t w, int32x8_t x, uint32_t ew, int bw, uint32_t ex, int bx)
{
    const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#define GEMM_RELU_BYTES(W, X) \
    case 4 * W + X: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, FW, FX, W, (int)ew, X, (int)ex);
    switch (4 * bw + bx) {
        GEMM_RELU_BYTES(0, 0) GEMM_RELU_BYTES(0, 1) GEMM_RELU_BYTES(0, 2) GEMM_RELU_BYTES(0, 3)
        GEMM_RELU_BYTES(1, 0) GEMM_RELU_BYTES(1, 1) GEMM_RELU_BYTES(1, 2) GEMM_RELU_BYTES(1, 3)
        GEMM_RELU_BYTES(2, 0) GEMM_RELU_BYTES(2, 1) GEMM_RELU_BYTES(2, 2) GEMM_RELU_BYTES(2, 3)
        GEMM_RELU_BYTES(3, 0) GEMM_RELU_BYTES(3, 1) GEMM_RELU_BYTES(3, 2) GEMM_RELU_BYTES(3, 3)
    }
#undef GEMM_RELU_BYTES
    __builtin_unreachable();
}

// A lane's 32 bytes of a matrix operand.
__device__ __forceinline__ int32x8_t join(u32x4 lo, u32x4 hi)
{
    return int32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

template <int BM_, int BN_, int STAGES_, int WAVES_M_, int WAVES_N_, int PRODUCERS_>
struct BlockConfig {
    static constexpr int BM = BM_, BN = BN_, BK = 128, STAGES = STAGES_, GROUP_M = 4;
    // WAVES compute waves; PRODUCERS > 0 adds waves that only load, else every
    // compute wave loads its share.
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WAVES = WAVES_M * WAVES_N, PRODUCERS = PRODUCERS_;
    static constexpr int DMA_WAVES = PRODUCERS > 0 ? PRODUCERS : WAVES, THREADS = 64 * (WAVES + PRODUCERS);
    static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N, FM = WTM / 16, FN = WTN / 16;
    static constexpr int A_STAGE = BM * BK, B_STAGE = BN * BK, B_REGION = STAGES * A_STAGE;
    static constexpr int S_STAGE = (BM + BN) * 4, S_REGION = STAGES * (A_STAGE + B_STAGE);
    // SPLIT: scales are split in LDS.  Their exponents are a byte each: of a wave's rows
    // 16 j + r for each r those of all j (FM bytes), after the rows the columns' likewise (FN).
    static constexpr bool SPLIT = BM > 64;
    static constexpr int E_STAGE = SPLIT ? BM + BN : 0, E_REGION = S_REGION + STAGES * S_STAGE;
    // A wave's strip: 16 rows of its columns of C on their way to memory.
    static constexpr int STRIP = 16 * WTN * 2, STRIPS = E_REGION + STAGES * E_STAGE;
    static constexpr int LDS_BYTES = STRIPS + WAVES * STRIP;
    static constexpr int QA = A_STAGE / 1024 / DMA_WAVES, QB = B_STAGE / 1024 / DMA_WAVES, NQ = QA + QB + 1;
    static constexpr int SCALE_PIECES = (BM + BN) / 64;
    static_assert(QA * DMA_WAVES * 1024 == A_STAGE && QB * DMA_WAVES * 1024 == B_STAGE, "whole DMA instructions");
    static_assert(QA % 2 == 0 && QB % 2 == 0, "the swizzle repeats every two instructions");
    static_assert(SCALE_PIECES <= DMA_WAVES && DMA_WAVES % SCALE_PIECES == 0, "one DMA of scales a wave");
    static_assert(!SPLIT || SCALE_PIECES == DMA_WAVES, "a piece that is rewritten is brought once");
    static_assert((STAGES & (STAGES - 1)) == 0 && LDS_BYTES <= 160 * 1024 && STAGES * NQ < 64, "ring");
    static_assert((WTN == 64 || WTN == 32) && 128 % WTN == 0, "a wave's columns lie in one tile of scales");
};

// Store FN x FM blocks of C^T (store_cols) through the wave's strip, 16 rows at a
// time: whole 16-byte pieces (c_vec), or dwords that lie on their boundaries and
// single elements at a row piece's ends.
template <int DT, int FN, int FM>
__device__ __forceinline__ void store_strips(uint16_t* __restrict__ C, const floatx4 (&acc)[FN][FM], uint8_t* strip,
                                             int lane, int m_base, int n_base, int m_end, int N, bool relu, int c_vec)
{
    constexpr int kNonTemporal = 2;   // cache policy nt
    constexpr int ROW = FN * 32, CHUNKS = ROW / 16;
    asm volatile("" : "+v"(lane));    // what follows from it is computed here, not kept through the caller's loop
    const int r16 = lane & 15, g = lane >> 4;
    auto at = [](int row, int chunk) { return row * ROW + ((chunk ^ ((row >> 1) & (CHUNKS - 1))) << 4); };
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int m = m_base + 16 * j, rows = max(0, min(16, m_end - m));
        if (rows == 0) break;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const floatx4& v = acc[i][j];
            *reinterpret_cast<u32x2*>(strip + at(r16, 2 * i + (g >> 1)) + 8 * (g & 1)) =
                u32x2{(uint32_t)act_cast<DT>(v[0], relu) | ((uint32_t)act_cast<DT>(v[1], relu) << 16),
                      (uint32_t)act_cast<DT>(v[2], relu) | ((uint32_t)act_cast<DT>(v[3], relu) << 16)};
        }
        if (c_vec) {
            const __amdgpu_buffer_rsrc_t rc = make_rsrc(C + (size_t)m * (size_t)N, (uint32_t)rows * (uint32_t)N * 2u);
#pragma unroll
            for (int s = 0; s < CHUNKS / 4; ++s) {
                const int r = s * (64 / CHUNKS) + lane / CHUNKS, c = lane % CHUNKS, n = n_base + 8 * c;
                const u32x4 v = *reinterpret_cast<const u32x4*>(strip + at(r, c));
                const uint32_t off = n < N ? ((uint32_t)r * (uint32_t)N + (uint32_t)n) * 2u : kOobOffset;
                __builtin_amdgcn_raw_buffer_store_b128(v, rc, off, 0, kNonTemporal);
            }
        } else {
            constexpr int LANES = FN * 8, STEP = 64 / LANES;          // dwords of a strip's row; rows a store
            const int cols = min(16 * FN, N - n_base), place = lane % LANES;
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += STEP) {
                const int r = r0 + lane / LANES;
                uint16_t* const p = C + (size_t)(m + r) * (size_t)N + n_base;
                const int odd = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1, e = 2 * place + odd;
                auto element = [&](int x) { return *reinterpret_cast<const uint16_t*>(strip + at(r, (x >> 3) & (CHUNKS - 1)) + 2 * (x & 7)); };
                const uint32_t lo = element(e), hi = element(e + 1), first = element(0);
                if (r < rows) {
                    if (e + 1 < cols) *reinterpret_cast<uint32_t*>(p + e) = lo | (hi << 16);
                    else if (e < cols) p[e] = (uint16_t)lo;
                    if (odd && place == 0 && cols > 0) p[0] = (uint16_t)first;
                }
            }
        }
    }
}

// Asks the scheduler for N times a matrix instruction and a block's additions: a wave
// that issues two matrix instructions in a row waits for the first with its additions.
template <int N>
__device__ __forceinline__ void interleave()
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);      // matrix
        __builtin_amdgcn_sched_group_barrier(0x2, 5, 0);      // vector
    }
}

// The product's tiles: groups one after the other, a group's tiles in panels of
// GROUP_M row tiles, column by column (tile_coords), the whole list dealt out in
// equal parts to the XCDs, so that tiles which share operands share an L2.  (Dealing
// whole columns of tiles, as RowUnits does, leaves an XCD with half as many again
// where there are few: 1000 x 1104 x 517, 18 columns of 16 tiles, 13.8 us against 11.4.)  Lane l keeps
// what belongs to group l; with more than 64 groups a lookup scans `ends` again.
template <class Cfg>
struct BlockUnits {
    const int* ends;
    int groups, M, tiles_n, lane, rows, first, listed;
    UnitOrder order;
    struct Lane {
        int begin, end, incl;      // the group's rows, units up to it
    } kept;                        // the first 64 groups

    __device__ __forceinline__ Lane scan(int g0, int& start, int& before) const
    {
        const GroupRows r = load_group_rows(ends, groups, M, g0, start, lane);
        const int tiles = g0 + lane < groups ? (r.end - r.begin + Cfg::BM - 1) / Cfg::BM : 0;
        const Lane k{r.begin, r.end, before + wave_scan_sum(tiles) * tiles_n};
        before = __builtin_amdgcn_readlane(k.incl, 63);
        start = __builtin_amdgcn_readlane(r.end, min(groups - 1 - g0, 63));
        return k;
    }
    __device__ __forceinline__ void init(const int* ends_, int groups_, int m, int n, int lane_, int block, int blocks)
    {
        ends = ends_;
        groups = groups_;
        M = m;
        tiles_n = (n + Cfg::BN - 1) / Cfg::BN;
        lane = lane_;
        order.init(block, blocks);
        int start = 0, total = 0;
        kept = scan(0, start, total);
        for (int g0 = 64; g0 < groups; g0 += 64) scan(g0, start, total);
        rows = start;
        first = (int)order.part(total, order.xcd);
        listed = (int)order.part(total, order.xcd + 1) - first;
    }
    __device__ __forceinline__ int count() const { return order.units(listed); }
    __device__ __forceinline__ DmaUnit unit(int i) const
    {
        const int at = first + order.position(i);
        int g0 = 0, start = 0, before = 0;
        Lane k = kept;
        if (groups > 64) {
            k = scan(0, start, before);
            while (at >= before) {
                g0 += 64;
                k = scan(g0, start, before);
            }
        }
        const int l = __builtin_ctzll(__ballot(at < k.incl));
        const int b = __builtin_amdgcn_readlane(k.begin, l), e = __builtin_amdgcn_readlane(k.end, l);
        const int tiles = (e - b + Cfg::BM - 1) / Cfg::BM, past = __builtin_amdgcn_readlane(k.incl, l) - at;
        int tm, tn;
        tile_coords(tiles * tiles_n - past, tiles, tiles_n, Cfg::GROUP_M, tm, tn, false);
        const int m0 = b + tm * Cfg::BM;
        return DmaUnit{m0, min(m0 + Cfg::BM, e), tn * Cfg::BN, g0 + l, 0, 0, -1};
    }
};

// What workgroup `block` of the `blocks` that share a product does.
template <class Cfg, int FA, int FB, bool B_ROWS>
__device__ __forceinline__ void blocks_tiles(const BlocksArgs& a, int block, int blocks, uint8_t* smem)
{
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, S = Cfg::STAGES, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int QA = Cfg::QA, QB = Cfg::QB, NQ = Cfg::NQ;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
    constexpr bool WS = Cfg::PRODUCERS > 0;
    const int dwave = WS ? wave - Cfg::WAVES : wave;      // among the waves that load
    const int k_blocks = (a.k + BK - 1) / BK, n_tiles = (a.n + kBlock - 1) / kBlock;
    BlockUnits<Cfg> units;
    units.init(a.ends, a.groups, a.m, a.n, lane, block, blocks);
    if (units.rows < a.m) {
        RowsArgs r{};
        r.m = a.m;
        r.n = a.n;
        r.c = a.c;
        zero_rows(r, units.rows, block, blocks);
    }
    const int n_units = __builtin_amdgcn_readfirstlane(units.count());
    if (n_units <= 0) return;
    auto unit_at = [&](int i) {
        const DmaUnit u = units.unit(i);
        return DmaUnit{__builtin_amdgcn_readfirstlane(u.m0), __builtin_amdgcn_readfirstlane(u.m_end),
                       __builtin_amdgcn_readfirstlane(u.n0), __builtin_amdgcn_readfirstlane(u.group), 0, a.k, -1};
    };
    const uint32_t lds_base = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem);

    // Where a lane's 16 bytes of a DMA instruction come from: row of the piece and
    // first k; two instructions (16 rows) on, the swizzle repeats.
    uint32_t a_voff[2], b_voff[2];
    int pos[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = 8 * q + lane / 8;
        pos[q] = ((lane % 8) ^ a_swizzle<128>(row)) * 16;
        a_voff[q] = (uint32_t)row * a.lda + (uint32_t)pos[q];
        b_voff[q] = (uint32_t)row * a.ldb + (uint32_t)pos[q];
    }
    // The scales' DMA: 64 floats of the tile's rows or columns a wave.
    const int piece = dwave & (Cfg::SCALE_PIECES - 1);
    const bool scales_of_a = piece < BM / 64;
    const uint32_t scales_lds = lds_base + Cfg::S_REGION + 256u * (uint32_t)piece;

    // The load side; past the last unit everything is out of range and fetches nothing.
    int f_unit = 0, f_k = 0, f_left = 0, f_turn = 0, f_rows = 0, f_cols = 0;
    const uint8_t *f_a = a.a, *f_b = a.b;
    const float* f_s = a.sa;          // this wave's scales of block 0
    uint32_t f_soff = 0, f_sbytes = 0, f_sstep = 0;
    auto fill_setup = [&]() {
        const int live = f_unit < n_units ? 1 : 0;
        const DmaUnit u = unit_at(live ? f_unit : n_units - 1);
        // Weights from memory: every column of tiles starts at another block of its rows (as in
        // blocks_stream.hpp), and has passed the caches once its rows' tiles have read it.  64
        // groups of 64 rows x 2048 x 4096: 123 -> 117 us past the caches, 103 so.
        if constexpr (WS) f_turn = a.once && k_blocks >= 2 * S ? (u.n0 / BN + 3 * u.group) % k_blocks * BK : 0;
        f_k = f_turn;
        f_left = k_blocks;
        f_rows = live * (u.m_end - u.m0);
        f_cols = live * min(BN, a.n - u.n0);
        f_a = a.a + (size_t)u.m0 * a.lda;
        f_b = a.b + ((size_t)u.group * (size_t)a.n + (size_t)u.n0) * a.ldb;
        int l = lane;
        asm volatile("" : "+v"(l));
        if (scales_of_a) {
            f_s = a.sa + u.m0 + 64 * piece;
            f_sbytes = 4u * (uint32_t)max(0, min(64, f_rows - 64 * piece));
            f_sstep = (uint32_t)a.m;
            f_soff = 4u * (uint32_t)l;
        } else {
            const int c = 64 * (piece - BM / 64);                    // first column, from n0 on
            if constexpr (B_ROWS) {
                f_s = a.sb + (size_t)u.group * (size_t)k_blocks * (size_t)a.n + (size_t)(u.n0 + c);
                f_sbytes = 4u * (uint32_t)max(0, min(64, f_cols - c));
                f_sstep = (uint32_t)a.n;
                f_soff = 4u * (uint32_t)l;
            } else {
                const int tile = (u.n0 + c) / kBlock;                // (64 columns lie in one tile)
                f_s = a.sb + ((size_t)u.group * (size_t)n_tiles + (size_t)min(tile, n_tiles - 1)) * (size_t)k_blocks;
                f_sbytes = 4u * (uint32_t)live;
                f_sstep = 1u;
                f_soff = 0u;
            }
        }
    };
    auto rows_from = [](const uint8_t* p, int rows, int skip, uint32_t ld) {
        const int32x4_t r = rsrc_words(p + (size_t)skip * ld, (uint32_t)max(0, rows - skip) * ld);
        return int32x4_t{__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]),
                         __builtin_amdgcn_readfirstlane(r[2]), kBufferFlags};
    };
    auto dma = [&](int slot, int q) {
        const int left = a.k - f_k;
        if (q < QA) {
            dma_b128(rows_from(f_a, f_rows, (dwave * QA + (q & ~1)) * 8, a.lda), lds_base + slot * Cfg::A_STAGE + (dwave * QA + q) * 1024,
                     pos[q & 1] >= left ? kOobOffset : a_voff[q & 1], (uint32_t)f_k);
        } else if (q < QA + QB) {
            const int p = q - QA;
            const auto load = [&](auto&& dma) __attribute__((always_inline)) {
                dma(rows_from(f_b, f_cols, (dwave * QB + (p & ~1)) * 8, a.ldb),
                    lds_base + Cfg::B_REGION + slot * Cfg::B_STAGE + (dwave * QB + p) * 1024,
                    pos[p & 1] >= left ? kOobOffset : b_voff[p & 1], (uint32_t)f_k);
            };
            if (WS && a.once) load(dma_b128_once);
            else load(dma_b128);
        } else {
            const int32x4_t r = rsrc_words(f_s + (size_t)(f_k / BK) * f_sstep, f_sbytes);
            dma_b32(int32x4_t{__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]),
                              __builtin_amdgcn_readfirstlane(r[2]), kBufferFlags},
                    scales_lds + slot * Cfg::S_STAGE, f_soff, 0u);
        }
    };
    auto fill_advance = [&]() {
        if (f_unit >= n_units) return;
        f_k = f_k + BK < a.k ? f_k + BK : 0;
        if (--f_left == 0) {
            ++f_unit;
            fill_setup();
        }
    };
    // This wave's pieces that straddle the end of the rows, of a stage that has
    // landed: what lies behind a row must not meet the other operand's zeros.
    auto cut_off = [&](int slot, int left) {
        if (left >= BK || left % 16 == 0) return;
        auto cut = [&](uint8_t* at, int first) {
            if (first < left && left < first + 16) {
                u32x4* const p = reinterpret_cast<u32x4*>(at + lane * 16);
                *p = keep_bytes(*p, left - first);
            }
        };
#pragma unroll
        for (int q = 0; q < QA; ++q) cut(smem + slot * Cfg::A_STAGE + (dwave * QA + q) * 1024, pos[q & 1]);
#pragma unroll
        for (int q = 0; q < QB; ++q) cut(smem + Cfg::B_REGION + slot * Cfg::B_STAGE + (dwave * QB + q) * 1024, pos[q & 1]);
    };

    // This wave's piece of the scales, of a stage that has landed: what is left of them in
    // their place, and their exponents.
    const auto exponent_at = [](int i) {
        constexpr int FM = Cfg::FM, FN = Cfg::FN;
        const int r = i < BM ? i : i - BM, n = i < BM ? FM : FN;
        return i - r + r / (16 * n) * (16 * n) + (r % 16) * n + r / 16 % n;
    };
    const int piece_at = 64 * piece + lane, exponent_to = exponent_at(piece_at);
    auto read_piece = [&](int slot) { return *reinterpret_cast<const float*>(smem + Cfg::S_REGION + slot * Cfg::S_STAGE + 4 * piece_at); };
    auto split_piece = [&](int slot, float s) {
        const SplitScale v = split_scale(s);
        *reinterpret_cast<float*>(smem + Cfg::S_REGION + slot * Cfg::S_STAGE + 4 * piece_at) = v.m;
        smem[Cfg::E_REGION + slot * Cfg::E_STAGE + exponent_to] = (uint8_t)v.e;
    };

    // Fragment reads (groups_dma.hpp): 16-byte chunks kb and 4 + kb of a row.
    const int kb = kgroup16(lane >> 4), g4 = lane >> 4, j16 = lane & 15;
    uint32_t a_off[2], b_off[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int ra = wm * Cfg::WTM + j16, rb = wn * Cfg::WTN + j16;
        a_off[h] = (uint32_t)(ra * BK + 16 * ((4 * h + kb) ^ a_swizzle<128>(ra)));
        b_off[h] = (uint32_t)(Cfg::B_REGION + rb * BK + 16 * ((4 * h + kb) ^ a_swizzle<128>(rb)));
    }
    auto fragment = [&](const uint8_t* stage, const uint32_t (&off)[2], int block) {
        return join(*reinterpret_cast<const u32x4*>(stage + off[0] + block * 16 * BK),
                    *reinterpret_cast<const u32x4*>(stage + off[1] + block * 16 * BK));
    };

    const int steps = n_units * k_blocks;
    if constexpr (WS) {
        // Step g's stage is filled while the step S - 1 before it is computed, and has
        // landed for every wave at barrier g.
        if (wave >= Cfg::WAVES) {
            fill_setup();
#pragma unroll 1
            for (int s = 0; s < S - 1; ++s) {
#pragma unroll
                for (int q = 0; q < NQ; ++q) dma(s, q);
                fill_advance();
            }
            int k = f_turn, left = k_blocks;                 // of the stage that lands
            for (int g = 0; g < steps; ++g) {
                wait_vmcnt<(S - 2) * NQ>();
                if constexpr (Cfg::SPLIT) split_piece(g & (S - 1), read_piece(g & (S - 1)));
                cut_off(g & (S - 1), a.k - k);
                k = k + BK < a.k ? k + BK : 0;
                lds_barrier();
#pragma unroll
                for (int q = 0; q < NQ; ++q) dma((g + S - 1) & (S - 1), q);
                fill_advance();
                if (--left == 0) {     // (the loads are less than a unit ahead, or turn is 0 for all)
                    k = f_turn;
                    left = k_blocks;
                }
            }
            wait_vmcnt<0>();           // no LDS DMA may outlive the workgroup
            lds_barrier();
            return;
        }
    } else {
        fill_setup();
#pragma unroll 1
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) dma(s, q);
            fill_advance();
        }
    }

    floatx4 acc[FN][FM];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    // Adds block (i, j)'s product.  (The empty assembly keeps the additions where they
    // are; the compiler would move all of them, and the products they wait for, behind
    // the step's last branch.)
    auto add = [&](int i, int j, const floatx4& t, float scale_x, const floatx4& scale_w) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(t[e], scale_x * scale_w[B_ROWS ? e : 0], acc[i][j][e]);
        asm volatile("" : "+v"(acc[i][j]));
    };
    auto read_scale_w = [&](const float* sc, int i) {
        if constexpr (B_ROWS) return *reinterpret_cast<const floatx4*>(sc + BM + wn * Cfg::WTN + 16 * i + 4 * g4);
        const float s = sc[BM + wn * Cfg::WTN];
        return floatx4{s, s, s, s};
    };
    auto store = [&](const DmaUnit& c) {
        const int m_base = c.m0 + wm * Cfg::WTM, n_base = c.n0 + wn * Cfg::WTN;
        uint8_t* const strip = smem + Cfg::STRIPS + wave * Cfg::STRIP;
        if (a.bf16) store_strips<kBF16>(a.c, acc, strip, lane, m_base, n_base, c.m_end, a.n, a.relu != 0, a.c_vec);
        else store_strips<kF16>(a.c, acc, strip, lane, m_base, n_base, c.m_end, a.n, a.relu != 0, a.c_vec);
    };
    auto scales = [&](int slot) { return reinterpret_cast<const float*>(smem + Cfg::S_REGION + slot * Cfg::S_STAGE); };
    constexpr int LAG = FM * FN < 8 || B_ROWS ? 2 : 3, NSW = B_ROWS ? FN : 1;       // blocks whose product is on its way
    clear();

    if constexpr (WS) {
        // A step's fragments are read while the step before is multiplied.
        struct Fragments {
            int32x8_t w[FN], x[FM];
            float scale_x[FM];
            floatx4 scale_w[NSW];
            uint32_t exponent_w[NSW], exponent_x[FM];      // (SPLIT: packed, in the first)
            float scale_own[NSW];                          // not SPLIT: that of the operand's row in this lane
        } f[2];
        auto read = [&](Fragments& to, int slot) __attribute__((always_inline)) {
            const float* sc = scales(slot);
#pragma unroll
            for (int i = 0; i < FN; ++i) to.w[i] = fragment(smem + slot * Cfg::B_STAGE, b_off, i);
#pragma unroll
            for (int j = 0; j < FM; ++j) to.x[j] = fragment(smem + slot * Cfg::A_STAGE, a_off, j);
#pragma unroll
            for (int j = 0; j < FM; ++j) to.scale_x[j] = sc[wm * Cfg::WTM + 16 * j + j16];
#pragma unroll
            for (int i = 0; i < NSW; ++i) to.scale_w[i] = read_scale_w(sc, i);
            if constexpr (Cfg::SPLIT) {
                static_assert(!Cfg::SPLIT || (FM == 4 && FN == 4), "bytes of exponents a lane");
                const uint8_t* const e = smem + Cfg::E_REGION + slot * Cfg::E_STAGE;
                to.exponent_x[0] = *reinterpret_cast<const uint32_t*>(e + wm * Cfg::WTM + j16 * FM);
                to.exponent_w[0] = *reinterpret_cast<const uint32_t*>(e + BM + wn * Cfg::WTN + j16 * FN);
            } else {
#pragma unroll
                for (int i = 0; i < NSW; ++i) to.scale_own[i] = B_ROWS ? sc[BM + wn * Cfg::WTN + 16 * i + j16] : to.scale_w[i][0];
            }
        };
        int c_unit = 0, left = k_blocks, g = 0;
        lds_barrier();
        read(f[0], 0);
        // Whether there is a step after this one.
        auto step = [&](Fragments& now, Fragments& next) __attribute__((always_inline)) {
            ++g;
            lds_barrier();                                  // step g has landed, or the last one is done
            if (g < steps) read(next, g & (S - 1));
            if constexpr (!Cfg::SPLIT) {
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const SplitScale s = split_scale(now.scale_x[j]);
                    now.scale_x[j] = s.m;
                    now.exponent_x[j] = s.e;
                }
#pragma unroll
                for (int i = 0; i < NSW; ++i) {
                    now.exponent_w[i] = split_scale(now.scale_own[i]).e;
#pragma unroll
                    for (int e = 0; e < (B_ROWS ? 4 : 1); ++e) now.scale_w[i][e] = split_scale(now.scale_w[i][e]).m;
                }
            }
            floatx4 t[LAG + 1];
#pragma unroll
            for (int u = 0; u < FM * FN + LAG; ++u) {
                if (u < FM * FN) {
                    const int i = u % FN, j = u / FN;
                    if constexpr (Cfg::SPLIT) t[u % (LAG + 1)] = mfma_block<FB, FA>(now.w[i], now.x[j], now.exponent_w[0], i, now.exponent_x[0], j);
                    else t[u % (LAG + 1)] = mfma_block<FB, FA>(now.w[i], now.x[j], now.exponent_w[B_ROWS ? i : 0], 0, now.exponent_x[j], 0);
                }
                if (u >= LAG) {
                    const int d = u - LAG, i = d % FN, j = d / FN;
                    add(i, j, t[d % (LAG + 1)], now.scale_x[j], now.scale_w[B_ROWS ? i : 0]);
                }
            }
            if (--left == 0) {
                store(unit_at(c_unit++));
                clear();
                left = k_blocks;
            }
            return g < steps;
        };
        while (step(f[0], f[1]) && step(f[1], f[0])) {
        }
    } else {
        // One set of fragments: the columns' are kept for a step, the rows' are read two
        // blocks ahead.  Before the last two row blocks everything of the slot has been
        // read: after the barrier there it is filled again, and the next step's first
        // fragments take the place of those that are done.
        static_assert(FM % 2 == 0 && FM >= 4, "row blocks");
        int32x8_t w[FN], x[3];
        float scale_x[FM];
        floatx4 scale_w[NSW];
        wait_vmcnt<(S - 1) * NQ>();
        split_piece(0, read_piece(0));
        cut_off(0, a.k);
        lds_barrier();
        auto read_x = [&](int to, int slot, int j) __attribute__((always_inline)) {
            x[to] = fragment(smem + slot * Cfg::A_STAGE, a_off, j);
        };
#pragma unroll
        for (int i = 0; i < FN; ++i) w[i] = fragment(smem, b_off, i);
        read_x(2, 0, 0);
        int slot = 0, c_unit = 0, k = 0;
        for (int g = 0; g < steps; ++g) {
            const float* sc = scales(slot);
#pragma unroll
            for (int j = 0; j < FM; ++j) scale_x[j] = sc[wm * Cfg::WTM + 16 * j + j16];
#pragma unroll
            for (int i = 0; i < NSW; ++i) scale_w[i] = read_scale_w(sc, i);
            // exponents of this lane's rows and columns, packed
            const uint8_t* const ep = smem + Cfg::E_REGION + slot * Cfg::E_STAGE;
            const u32x2 ex = *reinterpret_cast<const u32x2*>(ep + wm * Cfg::WTM + j16 * FM);
            const uint32_t ew = *reinterpret_cast<const uint32_t*>(ep + BM + wn * Cfg::WTN + j16 * FN);
            static_assert(FM == 8 && FN == 4, "bytes of exponents a lane");
            const auto product = [&](int i, int j) __attribute__((always_inline)) {
                return mfma_block<FB, FA>(w[i], x[j % 3], ew, i, ex[j / 4], j % 4);
            };
            x[0] = x[2];
            read_x(1, slot, 1);
            floatx4 t[LAG + 1];
            auto finish = [&](int u) __attribute__((always_inline)) {      // the addition for product u
                const bool late = u >= (FM - 2) * FN;
                const int v = u - (FM - 2) * FN, i = late ? v / 2 : u % FN, j = late ? FM - 2 + (v & 1) : u / FN;
                add(i, j, t[u % (LAG + 1)], scale_x[j], scale_w[B_ROWS ? i : 0]);
            };
            int u = 0;
            const int next = (slot + 1) & (S - 1);
            float landed = 0.0f;
#pragma unroll
            for (int j = 0; j < FM - 2; ++j) {
                if (j == FM - 3) {            // the next stage's scales, on their way while this is multiplied
                    wait_vmcnt<(S - 2) * NQ>();
                    landed = read_piece(next);
                }
                read_x((j + 2) % 3, slot, j + 2);
#pragma unroll
                for (int i = 0; i < FN; ++i, ++u) {
                    t[u % (LAG + 1)] = product(i, j);
                    if (u >= LAG) finish(u - LAG);
                }
                interleave<FN>();
                __builtin_amdgcn_sched_barrier(0);
            }
            const int k_next = k + BK < a.k ? k + BK : 0;
            split_piece(next, landed);
            cut_off(next, a.k - k_next);
            lds_barrier();
            // buffers (FM - 2) % 3 and (FM - 1) % 3 are in use; the third is 2 for FM = 8
            static_assert((FM - 2) % 3 == 0, "the next step's first fragment goes to x[2]");
            read_x(2, next, 0);
#pragma unroll
            for (int i = 0; i < FN; ++i) {
#pragma unroll
                for (int j = FM - 2; j < FM; ++j, ++u) {
                    t[u % (LAG + 1)] = product(i, j);
                    finish(u - LAG);
                }
                interleave<2>();
                w[i] = fragment(smem + next * Cfg::B_STAGE, b_off, i);
#pragma unroll
                for (int q = i * NQ / FN; q < (i + 1) * NQ / FN; ++q) dma(slot, q);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int d = FM * FN - LAG; d < FM * FN; ++d) finish(d);
            fill_advance();
            slot = next;
            k = k_next;
            if (k == 0) {
                store(unit_at(c_unit++));
                clear();
            }
        }
        wait_vmcnt<0>();   // no LDS DMA may outlive the workgroup
    }
}

template <class Cfg, int FA, int FB, bool B_ROWS>
__global__ __launch_bounds__(Cfg::THREADS, 1) void blocks_dma(BlocksArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Cfg::LDS_BYTES];
    blocks_tiles<Cfg, FA, FB, B_ROWS>(a, blockIdx.x, gridDim.x, smem);
}

// Two products in one launch, the second with scales of B by rows.
template <class Cfg, int FA, int FB>
__global__ __launch_bounds__(Cfg::THREADS, 1) void blocks_pair(BlocksPair p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Cfg::LDS_BYTES];
    const int block = blockIdx.x;
    if (block < p.blocks[0]) blocks_tiles<Cfg, FA, FB, false>(p.product[0], block, p.blocks[0], smem);
    else blocks_tiles<Cfg, FA, FB, true>(p.product[1], block - p.blocks[0], p.blocks[1], smem);
}

}  // namespace gemm_relu_hip
