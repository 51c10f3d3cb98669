// The LDS-DMA kernels of gemm_relu_groups.h: gemm_relu_dma's ring of stages,
// its swizzles and its schedule, with tiles that belong to row groups.
//
// One loop serves both products (DmaProduct): C = A @ B over groups of rows of
// C, and dB = A^T @ D over groups of the summed rows.  They differ in how the
// operands lie in memory and in what a work unit is:
//  * An operand is k-contiguous (A; B stored (N, K)) or k-major (B stored
//    (K, N); both operands of dB).  A k-contiguous stage is rows of BK k, read
//    with ds_read_b128; a k-major stage is BK rows as they are in memory, read
//    K-packed with the transposing ds_read_b64_tr_b16.
//  * A unit is an output tile with its range of k.  Units that share operands
//    are neighbours (tile_coords), and each workgroup (one per CU) streams the
//    K-steps of all its units through one ring.
#pragma once

#include "groups_kernels.hpp"

namespace gemm_relu_hip {

template <int BM_, int BN_, int STAGES_, int WAVES_M_, int WAVES_N_, bool A_KMAJOR_, bool B_KMAJOR_, int PRODUCERS_>
struct GroupDmaConfig {
    static constexpr int BM = BM_, BN = BN_, BK = 64, STAGES = STAGES_, GROUP_M = 4;
    // WAVES compute waves; PRODUCERS > 0 adds waves that only load, else every
    // compute wave loads its share and slots are refilled early (gemm_relu_dma).
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WAVES = WAVES_M * WAVES_N;
    static constexpr int PRODUCERS = PRODUCERS_, DMA_WAVES = PRODUCERS > 0 ? PRODUCERS : WAVES;
    static constexpr int THREADS = 64 * (WAVES + PRODUCERS);
    static constexpr bool A_KMAJOR = A_KMAJOR_, B_KMAJOR = B_KMAJOR_;
    static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N, FM = WTM / 16, FN = WTN / 16;
    static constexpr int A_ROW = A_KMAJOR ? BM * 2 : BK * 2, B_ROW = B_KMAJOR ? BN * 2 : BK * 2;
    static constexpr int A_STAGE = BM * BK * 2, B_STAGE = BN * BK * 2, B_REGION = STAGES * A_STAGE;
    static constexpr int LDS_BYTES = STAGES * (A_STAGE + B_STAGE);
    static constexpr bool C_STAGED = WTN % 64 == 0 && WTM % 32 == 0 && LDS_BYTES + WAVES * 4096 <= 160 * 1024;
    static constexpr int C_STAGE_BYTES = C_STAGED ? WAVES * 4096 : 0;
    // Adapters stage V there too, or in strips of their own.
    static constexpr int ADAPT_BYTES = C_STAGED ? 0 : WAVES * kAdapterStrip<FN>;
    static_assert(!C_STAGED || kAdapterStrip<FN> <= 4096, "V's strip");
    static constexpr int QA = A_STAGE / 1024 / DMA_WAVES, QB = B_STAGE / 1024 / DMA_WAVES, NQ = QA + QB;
    static_assert(QA * DMA_WAVES * 1024 == A_STAGE && QB * DMA_WAVES * 1024 == B_STAGE, "whole DMA instructions");
    static_assert((STAGES & (STAGES - 1)) == 0 && STAGES >= 2 && LDS_BYTES <= 160 * 1024, "ring");
    static_assert((STAGES - 1) * NQ < 64, "vmcnt range");
};

// One output tile: rows m0 .. m_end - 1 (at most BM) and columns n0 .. of C,
// summed over k0 .. k_end - 1, with the weights (or output) of `group`.
// adapter >= 0: the sum starts from the rows' low-rank terms with that adapter.
struct DmaUnit {
    int m0, m_end, n0, group, k0, k_end, adapter;
};

// The rows' products: unit -> row tile of a group (from the row table) and
// column tile.  Lane l keeps where group l ends and how many tiles there are up
// to it; with more than 64 groups a lookup scans `ends` again.
template <class Cfg>
struct RowUnits {
    const int* ends;
    int groups, M, K, tiles_n, lane;
    int listed;              // groups with tiles: all, and with `rest` the rows of none as one more
    int end, incl;           // per lane, at most 64 groups
    int row_tiles, rows;     // tiles of all groups; rows in groups
    const int* ids;          // the groups' adapters, or nullptr
    int adapters;

    __device__ __forceinline__ int tiles_of(const GroupRows& r) const { return (r.end - r.begin + Cfg::BM - 1) / Cfg::BM; }

    __device__ __forceinline__ void init(const RowsArgs& a, const int* ends_, int groups_, bool rest, int lane_)
    {
        ends = ends_;
        groups = groups_;
        listed = groups + (rest ? 1 : 0);
        ids = nullptr;
        M = a.m;
        K = a.k;
        tiles_n = (a.n + Cfg::BN - 1) / Cfg::BN;
        lane = lane_;
        row_tiles = 0;
        rows = 0;
        for (int g0 = 0; g0 < listed; g0 += 64) {
            const GroupRows r = load_group_rows(ends, groups, M, g0, rows, lane);
            const bool real = g0 + lane < listed;
            end = r.end;
            incl = row_tiles + wave_scan_sum(real ? tiles_of(r) : 0, lane);
            row_tiles = __builtin_amdgcn_readlane(incl, 63);
            rows = __builtin_amdgcn_readlane(r.end, min(listed - 1 - g0, 63));
        }
    }
    __device__ __forceinline__ int total() const { return row_tiles * tiles_n; }
    __device__ __forceinline__ DmaUnit unit(int u) const
    {
        int tm, tn;
        tile_coords(u, row_tiles, tiles_n, Cfg::GROUP_M, tm, tn);
        if (listed <= 64) {
            const int l = __builtin_ctzll(__ballot(tm < incl));
            const int e = __builtin_amdgcn_readlane(end, l);
            const int b = l ? __builtin_amdgcn_readlane(end, l - 1) : 0;
            const int before = l ? __builtin_amdgcn_readlane(incl, l - 1) : 0;
            const int m0 = b + (tm - before) * Cfg::BM;
            return DmaUnit{m0, min(m0 + Cfg::BM, e), tn * Cfg::BN, l, 0, K, adapter(l)};
        }
        const RowTile t = find_row_tile(ends, groups, M, Cfg::BM, tm, lane);
        return DmaUnit{t.begin, t.end, tn * Cfg::BN, t.group, 0, K, adapter(t.group)};
    }
    __device__ __forceinline__ int adapter(int group) const
    {
        const int id = ids && group < groups ? ids[group] : -1;
        return id < adapters ? id : -1;
    }
};

// The weights' gradients: unit -> group and tile of its (I, J) output; k runs
// over the group's rows.  An empty group keeps one K-step, of zeros.
template <class Cfg>
struct WeightUnits {
    const int* ends;
    int groups, M, I, tiles_i, tiles_j;

    __device__ __forceinline__ void init(const WeightArgs& a, int)
    {
        ends = a.ends;
        groups = a.groups;
        M = a.m;
        I = a.i;
        tiles_i = (a.i + Cfg::BM - 1) / Cfg::BM;
        tiles_j = (a.j + Cfg::BN - 1) / Cfg::BN;
    }
    __device__ __forceinline__ int total() const { return groups * tiles_i * tiles_j; }
    __device__ __forceinline__ DmaUnit unit(int u) const
    {
        // Each XCD takes a contiguous range of units, as tile_coords gives it
        // the tiles of one output; here that is whole groups, mostly.
        const int all = total(), per_xcd = all / 8;
        const int pid = u < per_xcd * 8 ? (u % 8) * per_xcd + u / 8 : u;
        const int tiles = tiles_i * tiles_j, g = pid / tiles;
        int ti, tj;
        tile_coords(pid - g * tiles, tiles_i, tiles_j, Cfg::GROUP_M, ti, tj, false);
        const int b = g ? min(max(ends[g - 1], 0), M) : 0;
        const int e = max(min(max(ends[g], 0), M), b);
        return DmaUnit{ti * Cfg::BM, I, tj * Cfg::BN, g, b, e, -1};
    }
};

// Store a wave's FN x FM blocks through its 4 KiB LDS strip as whole 128-byte
// row pieces, 32 rows x 64 columns at a time: store_tile_staged16 with the
// activation as an argument and the rows ending at m_end.
template <int DT, int FN, int FM>
__device__ __forceinline__ void store_rows_staged(uint16_t* __restrict__ C, const floatx4 (&acc)[FN][FM],
                                                  uint8_t* strip, int lane, int m_base, int n_base, int m_end, int N,
                                                  bool relu)
{
    constexpr int kNonTemporal = 2;   // cache policy nt
    const int r16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int jj = 0; jj < FM / 2; ++jj) {
        const int m_strip = m_base + 32 * jj;
        const int rows = max(0, min(32, m_end - m_strip));
        const __amdgpu_buffer_rsrc_t rc =
            make_rsrc(C + (size_t)min(m_strip, m_end) * (size_t)N, (uint32_t)rows * (uint32_t)N * 2u);
#pragma unroll
        for (int p = 0; p < FN / 4; ++p) {
#pragma unroll
            for (int jh = 0; jh < 2; ++jh)
#pragma unroll
                for (int ii = 0; ii < 4; ++ii) {
                    const floatx4& v = acc[4 * p + ii][2 * jj + jh];
                    const int rw = 16 * jh + r16, c = 2 * ii + (g >> 1);
                    const uint32_t lo =
                        (uint32_t)act_cast<DT>(v[0], relu) | ((uint32_t)act_cast<DT>(v[1], relu) << 16);
                    const uint32_t hi =
                        (uint32_t)act_cast<DT>(v[2], relu) | ((uint32_t)act_cast<DT>(v[3], relu) << 16);
                    *reinterpret_cast<u32x2*>(strip + rw * 128 + ((c ^ ((rw >> 1) & 7)) << 4) + 8 * (g & 1)) =
                        u32x2{lo, hi};
                }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 8 * s + (lane >> 3), c = lane & 7;
                const u32x4 v = *reinterpret_cast<const u32x4*>(strip + r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
                const int n = n_base + 64 * p + 8 * c;
                const uint32_t off = n < N ? ((uint32_t)r * (uint32_t)N + (uint32_t)n) * 2u : kOobOffset;
                __builtin_amdgcn_raw_buffer_store_b128(v, rc, off, 0, kNonTemporal);
            }
        }
    }
}

// The product loop.  A's rows are lda long, B's ldb; `b_group` and `c_group`
// are the elements from one group's B and C to the next.  KTAIL: k_end need not
// be a multiple of 64 for k-contiguous operands (but of 8).
//  With adapters, kAdaptAfter adds a finished tile's low-rank terms to its sums
// (add_adapters: tiles may hold rows of many segments).  kAdaptFirst is for
// tiles cut at the segments' ends: before its K-steps over A and B a tile
// streams K-steps over the intermediates (hi, then lo) and V through the same
// ring, multiplies its sums by the rows' factors, and goes on from them, so
// the low-rank product costs its K-steps and nothing else.
enum { kAdaptNone = 0, kAdaptAfter = 1, kAdaptFirst = 2 };
template <class Cfg, int DT, bool KTAIL, int ADAPT, class Units>
__device__ __forceinline__ void dma_product(const Units& units, const uint16_t* __restrict__ A,
                                            const uint16_t* __restrict__ B, uint16_t* __restrict__ C, uint32_t lda,
                                            uint32_t ldb, size_t b_group, size_t c_group, int N, bool relu, int c_vec,
                                            const AdapterArgs& ad, uint8_t* smem)
{
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, S = Cfg::STAGES;
    constexpr int QA = Cfg::QA, QB = Cfg::QB, NQ = Cfg::NQ, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int A_ROW = Cfg::A_ROW, B_ROW = Cfg::B_ROW, NKS = BK / 32;
    constexpr bool AK = Cfg::A_KMAJOR, BKM = Cfg::B_KMAJOR, WS = Cfg::PRODUCERS > 0, FIRST = ADAPT == kAdaptFirst;
    static_assert(!FIRST || (KTAIL && !AK), "the rank need not be a multiple of BK");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
    const bool producer = WS && wave >= Cfg::WAVES;
    const int dwave = WS ? wave - Cfg::WAVES : wave;
    const int total = __builtin_amdgcn_readfirstlane(units.total());
    const int n_units = (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    if (n_units <= 0) return;
    // Units are the same for all lanes; readfirstlane keeps them in scalar registers.
    auto unit_at = [&](int i) {
        const DmaUnit u = units.unit((int)blockIdx.x + i * (int)gridDim.x);
        return DmaUnit{__builtin_amdgcn_readfirstlane(u.m0),    __builtin_amdgcn_readfirstlane(u.m_end),
                       __builtin_amdgcn_readfirstlane(u.n0),    __builtin_amdgcn_readfirstlane(u.group),
                       __builtin_amdgcn_readfirstlane(u.k0),    __builtin_amdgcn_readfirstlane(u.k_end),
                       __builtin_amdgcn_readfirstlane(u.adapter)};
    };

    const uint32_t lds_base = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem);

    // Where each lane's 16 bytes of a DMA instruction come from (gemm_relu_dma),
    // as an offset from the tile's origin.  Two instructions on, the swizzle
    // repeats, so offsets are kept for the first two and the descriptor's base
    // moves on by the rows between.  k-contiguous operands: the same for every
    // tile.  k-major ones: columns past `limit` are sent out of range, so the
    // offsets are set anew for each tile.  pos: the piece's first k or column.
    constexpr int PA = QA < 2 ? QA : 2, PB = QB < 2 ? QB : 2;
    constexpr int A_PAIR = 2048 / A_ROW, B_PAIR = 2048 / B_ROW;    // rows of two instructions
    static_assert(QA <= 2 || (AK ? A_PAIR % 4 == 0 && 16 % (QA * A_PAIR / 2) == 0 : A_PAIR % 16 == 0), "A swizzle period");
    static_assert(QB <= 2 || (BKM ? B_PAIR % 4 == 0 && 16 % (QB * B_PAIR / 2) == 0 : B_PAIR % 16 == 0), "B swizzle period");
    uint32_t a_voff[PA], b_voff[PB];
    int a_pos[PA], b_pos[PB];
    auto piece = [&](int l, int q, int per_wave, auto kmajor, auto row_bytes, uint32_t ld, int limit, uint32_t& voff,
                     int& pos) {
        constexpr int ROW = decltype(row_bytes)::value;
        const int byte = ((dwave * per_wave + q) * 64 + l) * 16;
        const int row = byte / ROW;
        if constexpr (decltype(kmajor)::value)
            pos = (((byte % ROW) / 16) ^ b_swizzle<ROW, 16>(row)) * 8;
        else
            pos = (((byte % ROW) / 16) ^ a_swizzle<ROW>(row)) * 8;
        voff = pos < limit ? ((uint32_t)row * ld + (uint32_t)pos) * 2u : kOobOffset;
    };
    uint32_t f_lda = lda, f_ldb = ldb;      // row lengths of the step's operands
    auto a_pieces = [&](int l, int limit) {
#pragma unroll
        for (int q = 0; q < PA; ++q)
            piece(l, q, QA, std::integral_constant<bool, AK>{}, std::integral_constant<int, A_ROW>{}, f_lda, limit,
                  a_voff[q], a_pos[q]);
    };
    auto b_pieces = [&](int l, int limit) {
#pragma unroll
        for (int q = 0; q < PB; ++q)
            piece(l, q, QB, std::integral_constant<bool, BKM>{}, std::integral_constant<int, B_ROW>{}, f_ldb, limit,
                  b_voff[q], b_pos[q]);
    };
    if constexpr (!AK && !FIRST) a_pieces(lane, BK);
    if constexpr (!BKM && !FIRST) b_pieces(lane, BK);

    // The load side.  f_left: k still to load of the unit; past the last unit it
    // is 0 and the descriptors are empty, so nothing is fetched.  (All of it is
    // set on every path, without branches, which keeps it in scalar registers.)
    // f_rank: K-steps over the intermediates and V still to load (kAdaptFirst).
    int f_unit = 0, f_k = 0, f_left = 0, f_steps = 0, f_rank = 0;
    // k-contiguous: the tile's rows and how many there are; k-major: the step's first row.
    const uint16_t *f_ap = A, *f_bp = B;
    int f_arows = 0, f_brows = 0;
    int f_kb = 0, f_left_b = 0;       // B's place and what it has left, where they differ from f_k and f_left
    const int rank_steps = FIRST ? 2 * ad.rank_pad / BK : 0;
    auto fill_setup = [&](bool start) {
        const int live = f_unit < n_units ? 1 : 0;
        const DmaUnit u = unit_at(live ? f_unit : n_units - 1);
        const bool low = FIRST && start && live && u.adapter >= 0;
        f_rank = low ? rank_steps : 0;
        f_k = u.k0;
        f_left = live * (u.k_end - u.k0);
        const uint16_t *a = A, *b = B + (size_t)u.group * b_group;
        if constexpr (FIRST) {
            f_kb = f_k;
            f_left_b = low ? ad.rank : f_left;
            f_lda = low ? 2u * (uint32_t)ad.rank_pad : lda;
            a = low ? ad.t : A;
            b = low ? ad.v + (size_t)u.adapter * (size_t)ad.rank * (size_t)N : B;
            if constexpr (!BKM) f_ldb = low ? (uint32_t)ad.rank : ldb;
        }
        int l = lane;
        asm volatile("" : "+v"(l));   // computed here for each tile, not kept in registers in between
        if constexpr (AK) {
            f_ap = a + (size_t)u.k0 * lda + u.m0;
            a_pieces(l, u.m_end - u.m0);
        } else {
            f_ap = a + (size_t)u.m0 * f_lda;
            f_arows = live * (u.m_end - u.m0);
            if constexpr (FIRST) a_pieces(l, BK);
        }
        if constexpr (BKM) {
            f_bp = b + (size_t)u.k0 * ldb + u.n0;
            b_pieces(l, N - u.n0);
        } else {
            f_bp = b + (size_t)u.n0 * f_ldb;
            f_brows = live * min(BN, N - u.n0);
            if constexpr (FIRST) b_pieces(l, BK);
        }
    };
    fill_setup(true);
    // The descriptor of the rows from `skip` on of a stage with `rows` rows.
    auto rows_from = [](const uint16_t* p, int rows, int skip, uint32_t ld) {
        const int32x4_t r = rsrc_words(p + (size_t)skip * ld, (uint32_t)max(0, rows - skip) * ld * 2u);
        return int32x4_t{__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]),
                         __builtin_amdgcn_readfirstlane(r[2]), kBufferFlags};
    };
    auto dma = [&](int slot, int q) {
        if (q < QA) {
            const uint32_t lds = lds_base + slot * Cfg::A_STAGE + (dwave * QA + q) * 1024;
            const uint32_t vo = a_voff[q % PA];
            if constexpr (AK)
                dma_b128(rows_from(f_ap, min(BK, f_left), q / 2 * A_PAIR, lda), lds, vo, 0u);
            else   // (the intermediates' rows are whole K-steps)
                dma_b128(rows_from(f_ap, f_arows, q / 2 * A_PAIR, f_lda), lds,
                         KTAIL && !(FIRST && f_rank) && a_pos[q % PA] >= f_left ? kOobOffset : vo, (uint32_t)f_k * 2u);
        } else {
            const int p = q - QA;
            const int left = FIRST ? f_left_b : f_left;
            const uint32_t lds = lds_base + Cfg::B_REGION + slot * Cfg::B_STAGE + (dwave * QB + p) * 1024;
            const uint32_t vo = b_voff[p % PB];
            if constexpr (BKM)
                dma_b128(rows_from(f_bp, min(BK, left), p / 2 * B_PAIR, ldb), lds, vo, 0u);
            else
                dma_b128(rows_from(f_bp, f_brows, p / 2 * B_PAIR, f_ldb), lds,
                         KTAIL && b_pos[p % PB] >= left ? kOobOffset : vo, (uint32_t)(FIRST ? f_kb : f_k) * 2u);
        }
    };
    auto fill_advance = [&]() {
        if (f_unit >= n_units) return;
        ++f_steps;
        if (FIRST && f_rank > 0) {
            if (--f_rank == 0) {
                fill_setup(false);
                return;
            }
            // V's K-steps once for hi, once again for lo
            const int next = f_kb + BK < ad.rank_pad ? f_kb + BK : 0;
            if constexpr (BKM) f_bp += (ptrdiff_t)(next - f_kb) * (ptrdiff_t)ldb;
            f_k += BK;
            f_kb = next;
            f_left_b = ad.rank - next;
        } else if (f_left <= BK) {
            ++f_unit;
            fill_setup(true);
        } else {
            f_k += BK;
            f_left -= BK;
            if constexpr (FIRST) {
                f_kb = f_k;
                f_left_b = f_left;
            }
            if constexpr (AK) f_ap += (size_t)BK * lda;
            if constexpr (BKM) f_bp += (size_t)BK * ldb;
        }
    };

    // Fragment reads (gemm_relu_dma, MF = 16).
    const int kb = kgroup16(lane >> 4), g4 = lane >> 4, j16 = lane & 15;
    uint32_t a_off[AK ? FM : NKS], b_off[BKM ? FN : NKS];
    if constexpr (AK) {
        const int krow = 8 * kgroup16(g4) + (j16 >> 2);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = wm * Cfg::WTM + j * 16 + 4 * (j16 & 3);
            a_off[j] = (uint32_t)(krow * A_ROW + 16 * ((m >> 3) ^ b_swizzle<A_ROW, 16>(krow)) + 8 * (j16 & 1));
        }
    } else {
        const int row = wm * Cfg::WTM + j16;
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks) a_off[ks] = (uint32_t)(row * A_ROW + 16 * ((4 * ks + kb) ^ a_swizzle<A_ROW>(row)));
    }
    if constexpr (BKM) {
        const int krow = 8 * kgroup16(g4) + (j16 >> 2);
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int n = wn * Cfg::WTN + i * 16 + 4 * (j16 & 3);
            b_off[i] = (uint32_t)(Cfg::B_REGION + krow * B_ROW + 16 * ((n >> 3) ^ b_swizzle<B_ROW, 16>(krow)) +
                                  8 * (j16 & 1));
        }
    } else {
        const int row = wn * Cfg::WTN + j16;
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks)
            b_off[ks] = (uint32_t)(Cfg::B_REGION + row * B_ROW + 16 * ((4 * ks + kb) ^ a_swizzle<B_ROW>(row)));
    }
    floatx4 acc[FN][FM];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear();
    u32x4 fb[2][FN], fa[2][FM];
    auto read_tr = [&](const uint8_t* p, int row) {
        const u32x2 lo = ds_read_tr16(p), hi = ds_read_tr16(p + 4 * row);
        return u32x4{lo.x, lo.y, hi.x, hi.y};
    };
    auto read_unit = [&](int buf, int slot, int ks, int u) {
        if (u < FM) {
            const uint8_t* st = smem + slot * Cfg::A_STAGE;
            if constexpr (AK) fa[buf][u] = read_tr(st + a_off[u] + 32 * ks * A_ROW, A_ROW);
            else fa[buf][u] = *reinterpret_cast<const u32x4*>(st + a_off[ks] + u * 16 * A_ROW);
        } else {
            const uint8_t* st = smem + slot * Cfg::B_STAGE;
            if constexpr (BKM) fb[buf][u - FM] = read_tr(st + b_off[u - FM] + 32 * ks * B_ROW, B_ROW);
            else fb[buf][u - FM] = *reinterpret_cast<const u32x4*>(st + b_off[ks] + (u - FM) * 16 * B_ROW);
        }
    };
    constexpr int NF = FM + FN, NMF = FM * FN;

    constexpr int PRO = WS ? S - 1 : S;      // steps the prologue issues
    if (!WS || producer) {
#pragma unroll
        for (int s = 0; s < PRO; ++s) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) dma(s, q);
            fill_advance();
        }
        wait_vmcnt<(PRO - 1) * NQ>();
    }
    lds_barrier();
    if constexpr (WS) {
        if (producer) {
            for (int g = 0; f_unit < n_units || g < f_steps; ++g) {
                const int slot_fill = (g + S - 1) & (S - 1);
#pragma unroll
                for (int q = 0; q < NQ; ++q) dma(slot_fill, q);
                fill_advance();
                wait_vmcnt<(S - 2) * NQ>();
                lds_barrier();
            }
            wait_vmcnt<0>();   // no LDS DMA may outlive the workgroup
            return;
        }
    }
#pragma unroll
    for (int u = 0; u < NF; ++u) read_unit(0, 0, 0, u);
    constexpr int NQC = WS ? 0 : NQ;
    constexpr int BAR_T = (!WS && NMF >= 8) ? 4 : 0;
    // Reads and, with early refill, the DMAs after the step barrier, alternately.
    auto item = [](int u0) {
        constexpr int PAIRS = NQC < NF ? NQC : NF;
        if (u0 < 2 * PAIRS) return (u0 & 1) ? u0 / 2 : NF + u0 / 2;
        return NQC > NF ? NF + (u0 - PAIRS) : u0 - PAIRS;
    };

    int c_unit = 0, slot = 0;
    DmaUnit c = unit_at(0);
    int c_k = c.k0 - (FIRST && c.adapter >= 0 ? rank_steps * BK : 0);
    while (true) {
        const int slot_next = (slot + 1) & (S - 1);
        auto step_barrier = [&]() {
            if constexpr (!WS) wait_vmcnt<(S - 2) * NQ>();
            lds_barrier();
        };
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks) {
            const int cur = ks & 1, nxt = cur ^ 1;
            const bool last = ks == NKS - 1;
            if (last && BAR_T == 0) step_barrier();
            const bool dma_ks = last;
            const int n_items = NF + (dma_ks ? NQC : 0);
#pragma unroll
            for (int t = 0; t < NMF; ++t) {
                if (last && BAR_T > 0 && t == BAR_T) step_barrier();
                const int bi = t / FM, bj = (bi & 1) ? FM - 1 - t % FM : t % FM;
                acc[bi][bj] = mfma_16x16x32<DT>(fb[cur][bi], fa[cur][bj], acc[bi][bj]);
                const int t0 = last ? t - BAR_T : t, span = last ? NMF - BAR_T : NMF;
                if (t0 < 0) {
                    __builtin_amdgcn_sched_barrier(0);
                    continue;
                }
#pragma unroll
                for (int u0 = t0 * n_items / span; u0 < (t0 + 1) * n_items / span; ++u0) {
                    const int u = dma_ks ? item(u0) : u0;
                    if (u < NF) {
                        if (last) read_unit(nxt, slot_next, 0, u);
                        else read_unit(nxt, slot, ks + 1, u);
                    } else {
                        dma(slot, u - NF);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (!WS && dma_ks) fill_advance();
        }
        slot = slot_next;
        c_k += BK;
        if (FIRST && c_k == 0 && c.adapter >= 0) {
            int l = j16;
            asm volatile("" : "+v"(l));
            float f[FM];
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int m = c.m0 + wm * Cfg::WTM + 16 * j + l;
                f[j] = m < c.m_end ? ad.factor[m] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] *= f[j];
        }
        if (c_k >= c.k_end) {
            const int m_base = c.m0 + wm * Cfg::WTM, n_base = c.n0 + wn * Cfg::WTN;
            if constexpr (ADAPT == kAdaptAfter)
                add_adapters<DT, !BKM>(acc, ad, m_base, c.m_end, n_base, N, lane,
                                                  smem + Cfg::LDS_BYTES + wave * kAdapterStrip<FN>);
            uint16_t* out = C + (size_t)c.group * c_group;
            bool staged = false;
            if constexpr (Cfg::C_STAGED) {
                if (c_vec == 2) {
                    store_rows_staged<DT>(out, acc, smem + Cfg::LDS_BYTES + wave * 4096, lane, m_base, n_base, c.m_end, N,
                                          relu);
                    staged = true;
                }
            }
            if (!staged) {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j)
                        store_cols<DT>(out, acc[i][j], m_base + 16 * j + j16, n_base + 16 * i + 4 * g4, c.m_end, N, relu,
                                       c_vec);
            }
            if (++c_unit >= n_units) break;
            clear();
            c = unit_at(c_unit);
            c_k = c.k0 - (FIRST && c.adapter >= 0 ? rank_steps * BK : 0);
            if constexpr (ADAPT == kAdaptAfter) {   // the registers of the next fragments were free meanwhile
#pragma unroll
                for (int u = 0; u < NF; ++u) read_unit(0, slot, 0, u);
            }
        }
    }
    wait_vmcnt<0>();   // no LDS DMA may outlive the workgroup
}

// Rows of no group: this launch's workgroups share their zeros.
__device__ __forceinline__ void zero_rows(const RowsArgs& a, int first)
{
    const size_t n = (size_t)a.n, count = (size_t)(a.m - first) * n;
    uint16_t* p = a.c + (size_t)first * n;
    const size_t stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < count; i += stride) p[i] = 0;
}

template <class Cfg, int DT, bool KTAIL, int ADAPT>
__global__ __launch_bounds__(Cfg::THREADS, 1) void rows_dma(RowsArgs a, AdapterArgs ad)
{
    __shared__ __attribute__((aligned(1024))) uint8_t
        smem[Cfg::LDS_BYTES + Cfg::C_STAGE_BYTES + (ADAPT == kAdaptAfter ? Cfg::ADAPT_BYTES : 0)];
    RowUnits<Cfg> units;
    if constexpr (ADAPT == kAdaptFirst) {
        units.init(a, ad.ends, ad.segments, true, threadIdx.x & 63);
        units.ids = ad.ids;
        units.adapters = ad.adapters;
    } else {
        units.init(a, a.ends, a.groups, false, threadIdx.x & 63);
        if (units.rows < a.m) zero_rows(a, units.rows);
    }
    dma_product<Cfg, DT, KTAIL, ADAPT>(units, a.a, a.b, a.c, (uint32_t)a.k, (uint32_t)(Cfg::B_KMAJOR ? a.n : a.k),
                                       ADAPT == kAdaptFirst ? 0 : (size_t)a.k * (size_t)a.n, 0, a.n, a.relu != 0, a.c_vec,
                                       ad, smem);
}

template <class Cfg, int DT>
__global__ __launch_bounds__(Cfg::THREADS, 1) void weight_dma(WeightArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Cfg::LDS_BYTES + Cfg::C_STAGE_BYTES];
    WeightUnits<Cfg> units;
    units.init(a, 0);
    dma_product<Cfg, DT, false, kAdaptNone>(units, a.p, a.q, a.out, (uint32_t)a.i, (uint32_t)a.j, 0,
                                       (size_t)a.i * (size_t)a.j, a.j, false, a.c_vec, AdapterArgs{}, smem);
}

}  // namespace gemm_relu_hip
