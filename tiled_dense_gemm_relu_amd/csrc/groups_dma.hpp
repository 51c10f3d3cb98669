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

template <int BM_, int BN_, int STAGES_, int WAVES_M_, int WAVES_N_, bool A_KMAJOR_, bool B_KMAJOR_, int PRODUCERS_,
          int SETS_ = 0, int MASKED_ = 0, bool ODD_ = true>
struct GroupDmaConfig {
    static constexpr int BM = BM_, BN = BN_, BK = 64, STAGES = STAGES_, GROUP_M = 4;
    // WAVES compute waves; PRODUCERS > 0 adds waves that only load, else every
    // compute wave loads its share and slots are refilled early (gemm_relu_dma).
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WAVES = WAVES_M * WAVES_N;
    static constexpr int PRODUCERS = PRODUCERS_, DMA_WAVES = PRODUCERS > 0 ? PRODUCERS : WAVES;
    static constexpr int THREADS = 64 * (WAVES + PRODUCERS);
    static constexpr bool A_KMAJOR = A_KMAJOR_, B_KMAJOR = B_KMAJOR_;
    // SETS > 0: the producers load through registers instead (rows of any length
    // and alignment), with that many steps in flight.  MASKED: the operand (1: A,
    // 2: B) that is zero where a second matrix of its shape is not above zero.
    // ODD: elements may start inside a dword (odd row lengths, 2-byte alignment).
    static constexpr int SETS = SETS_, MASKED = MASKED_;
    static constexpr bool ODD = ODD_;
    static constexpr bool STAGED = SETS > 0;
    static_assert(!STAGED || (PRODUCERS > 0 && STAGES_ == 2), "producers fill the other of two stages");
    static_assert(STAGED || MASKED == 0, "DMA cannot mask");
    static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N, FM = WTM / 16, FN = WTN / 16;
    static constexpr int A_ROW = A_KMAJOR ? BM * 2 : BK * 2, B_ROW = B_KMAJOR ? BN * 2 : BK * 2;
    static constexpr int A_STAGE = BM * BK * 2, B_STAGE = BN * BK * 2, B_REGION = STAGES * A_STAGE;
    static constexpr int LDS_BYTES = STAGES * (A_STAGE + B_STAGE);
    // Each compute wave's strip of LDS, 32 rows of its columns of C on their way to
    // memory.  Adapters stage V there.
    static constexpr int STRIP = 32 * WTN * 2, STRIP_BYTES = WAVES * STRIP;
    static_assert(WTM % 32 == 0 && (WTN == 64 || WTN == 32) && LDS_BYTES + STRIP_BYTES <= 160 * 1024, "strips");
    static_assert(kAdapterStrip<FN> <= STRIP, "V's strip");
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

// Where a workgroup finds its units in its XCD's list of them: in turn, every
// second round in the opposite direction, so that the last workgroup of a round,
// whose unit is the shortest, is the first of the next.
struct UnitOrder {
    int xcd, xcds, place, width;      // this workgroup's XCD and place among its workgroups

    __device__ __forceinline__ void init(int block, int blocks)
    {
        xcds = blocks % 8 == 0 ? 8 : 1;
        xcd = block % xcds;
        place = block / xcds;
        width = blocks / xcds;
    }
    // The first of `total` that belong to XCD x and later ones.
    __device__ __forceinline__ int64_t part(int64_t total, int x) const { return xcds == 8 ? total * x / 8 : total * x; }
    // Position of this workgroup's i-th unit in the list.
    __device__ __forceinline__ int position(int i) const { return i * width + ((i & 1) ? width - 1 - place : place); }
    __device__ __forceinline__ int units(int listed) const
    {
        const int whole = listed / width;
        return whole + (position(whole) < listed ? 1 : 0);
    }
};

// The rows' products.  A group's rows are cut into tiles of BM rows, the last of
// them partial.  The groups' output columns are dealt to the XCDs in order, an
// eighth of the work to each (in quarter tiles; a partial tile of at most half
// the rows counts as half; it costs more, 67 to 79% of a whole one with 256 rows,
// but three quarters measured the same in every case), so an XCD has all row tiles of its columns, next to
// each other in its list: they share the group's weights in its L2.  (Whole
// tiles first and partial ones after them would balance a round better, but the
// partial ones then read their weights again, each its own: 1087 against 1003 us
// for 16384 rows in 16 groups, 4096 x 8192 fp16.)  With more rows than all
// groups' columns (tall outputs of few groups), it is the rows of A that are worth
// sharing: then the XCDs get consecutive units of GROUP_M rows of tiles, column by
// column.  Lane l keeps what belongs to
// group l; with more than 64 groups (MANY) a lookup scans `ends` again.
template <class Cfg, bool MANY>
struct RowUnits {
    static constexpr bool RAGGED = true;      // tiles of fewer than BM rows are common
    const int* ends;
    int groups, M, K, tiles_n, lane;
    int listed;              // groups with tiles: all, and with `rest` the rows of none as one more
    int rows;                // rows in groups
    int units;               // this XCD's
    int64_t first, last;     // its part of the work, or of the units
    bool by_rows, rotate;
    const int* ids;          // the groups' adapters, or nullptr
    int adapters;
    UnitOrder order;
    struct Lane {
        int begin, end;      // the group's rows
        int from, count;     // this XCD's columns of its tiles, or units (by_rows)
        int incl;            // units up to this group
    } kept;                  // at most 64 groups

    __device__ __forceinline__ static int cost(int n) { return n / Cfg::BM * 4 + (n % Cfg::BM > Cfg::BM / 2 ? 4 : n % Cfg::BM ? 2 : 0); }

    // 64 groups from g0 on, which start at row `start`; `work` and `before`
    // are what the groups before them have, and are moved on.
    __device__ __forceinline__ Lane scan(int g0, int& start, int64_t& work, int& units_before) const
    {
        const GroupRows r = load_group_rows(ends, groups, M, g0, start, lane);
        const int n = g0 + lane < listed ? r.end - r.begin : 0, c = cost(n);
        const int before = wave_scan_sum(c) - c;      // at most 4 (2^20 / 64 + 65536)
        // the first column whose work starts at or past w
        auto column = [&](int64_t w) {
            const int64_t past = w - (work + (int64_t)before * tiles_n);
            if (past <= 0 || c == 0) return 0;
            return past >= (int64_t)c * tiles_n ? tiles_n : (int)(((uint32_t)past + c - 1u) / (uint32_t)c);   // c tiles_n <= 2^31
        };
        const int tiles = (n + Cfg::BM - 1) / Cfg::BM;
        // the group's units before unit w of all
        const int units_before_group = wave_scan_sum(tiles) - tiles;
        auto unit_at = [&](int64_t w) {
            return (int)min(max(w - (work + (int64_t)units_before_group * tiles_n), (int64_t)0), (int64_t)tiles * tiles_n);
        };
        Lane k;
        k.begin = r.begin;
        k.end = r.end;
        k.from = by_rows ? unit_at(first) : column(first);
        k.count = max(0, (by_rows ? unit_at(last) : column(last)) - k.from);
        k.incl = units_before + wave_scan_sum(by_rows ? k.count : tiles * k.count);
        work += (int64_t)__builtin_amdgcn_readlane(by_rows ? units_before_group + tiles : before + c, 63) * tiles_n;
        units_before = __builtin_amdgcn_readlane(k.incl, 63);
        start = __builtin_amdgcn_readlane(r.end, 63);
        return k;
    }

    __device__ __forceinline__ void init(const RowsArgs& a, const int* ends_, int groups_, bool rest, int lane_, int block,
                                         int blocks)
    {
        ends = ends_;
        groups = groups_;
        listed = groups + (rest ? 1 : 0);
        ids = nullptr;
        M = a.m;
        K = a.k;
        tiles_n = (a.n + Cfg::BN - 1) / Cfg::BN;
        lane = lane_;
        order.init(block, blocks);
        by_rows = M > (int64_t)groups * a.n;
        rotate = M <= 64 * (int64_t)min(groups, M);
        int64_t total = 0;
        rows = 0;
        for (int g0 = 0; g0 < listed; g0 += 64) {
            const GroupRows r = load_group_rows(ends, groups, M, g0, rows, lane);
            const int n = g0 + lane < listed ? r.end - r.begin : 0;
            total += __builtin_amdgcn_readlane(wave_scan_sum(by_rows ? (n + Cfg::BM - 1) / Cfg::BM : cost(n)), 63);
            rows = __builtin_amdgcn_readlane(r.end, min(listed - 1 - g0, 63));
        }
        total *= tiles_n;
        first = order.part(total, order.xcd);
        last = order.part(total, order.xcd + 1);
        int start = 0;
        int64_t work = 0;
        units = 0;
        for (int g0 = 0; g0 < listed; g0 += 64) kept = scan(g0, start, work, units);
    }
    __device__ __forceinline__ int count() const { return order.units(units); }
    __device__ __forceinline__ DmaUnit unit(int i) const
    {
        const int at = order.position(i);
        int g0 = 0;
        Lane k = kept;
        if (MANY && listed > 64) {
            int start = 0, before = 0;
            int64_t work = 0;
            for (;; g0 += 64) {
                k = scan(g0, start, work, before);
                if (at < before) break;
            }
        }
        const int l = __builtin_ctzll(__ballot(at < k.incl));
        const int b = __builtin_amdgcn_readlane(k.begin, l), e = __builtin_amdgcn_readlane(k.end, l);
        const int from = __builtin_amdgcn_readlane(k.from, l), count = __builtin_amdgcn_readlane(k.count, l);
        const int tiles = (e - b + Cfg::BM - 1) / Cfg::BM, past = __builtin_amdgcn_readlane(k.incl, l) - at;
        int tm, tn;
        tile_coords(by_rows ? from + count - past : tiles * count - past, tiles, by_rows ? tiles_n : count, Cfg::GROUP_M, tm, tn, false);
        const int m0 = b + tm * Cfg::BM, id = ids && g0 + l < groups ? ids[g0 + l] : -1;
        return DmaUnit{m0, min(m0 + Cfg::BM, e), (by_rows ? tn : from + tn) * Cfg::BN, g0 + l, 0, K, id < adapters ? id : -1};
    }
};

// The weights' gradients: unit -> group and tile of its (I, J) output; k runs
// over the group's rows.  An empty group keeps one K-step, of zeros.
template <class Cfg>
struct WeightUnits {
    static constexpr bool RAGGED = false;
    const int* ends;
    int groups, M, I, tiles_i, tiles_j;
    int first, listed;       // this XCD's units
    UnitOrder order;

    __device__ __forceinline__ void init(const WeightArgs& a, int block, int blocks)
    {
        ends = a.ends;
        groups = a.groups;
        M = a.m;
        I = a.i;
        tiles_i = (a.i + Cfg::BM - 1) / Cfg::BM;
        tiles_j = (a.j + Cfg::BN - 1) / Cfg::BN;
        order.init(block, blocks);
        const int total = groups * tiles_i * tiles_j;
        first = (int)order.part(total, order.xcd);
        listed = (int)order.part(total, order.xcd + 1) - first;
    }
    __device__ __forceinline__ int count() const { return order.units(listed); }
    __device__ __forceinline__ DmaUnit unit(int i) const
    {
        const int pid = first + order.position(i), tiles = tiles_i * tiles_j, g = pid / tiles;
        int ti, tj;
        tile_coords(pid - g * tiles, tiles_i, tiles_j, Cfg::GROUP_M, ti, tj, false);
        const int b = g ? min(max(ends[g - 1], 0), M) : 0;
        const int e = max(min(max(ends[g], 0), M), b);
        return DmaUnit{ti * Cfg::BM, I, tj * Cfg::BN, g, b, e, -1};
    }
};

// Store a wave's FN x FM blocks through its 4 KiB LDS strip as whole 128-byte
// row pieces, 32 rows x 64 columns at a time: store_tile_staged16 with the
// activation as an argument and the rows ending at m_end, the first FX blocks.
template <int DT, int FX, int FN, int FM>
__device__ __forceinline__ void store_rows_staged(uint16_t* __restrict__ C, const floatx4 (&acc)[FN][FM],
                                                  uint8_t* strip, int lane, int m_base, int n_base, int m_end, int N,
                                                  bool relu)
{
    constexpr int kNonTemporal = 2;   // cache policy nt
    asm volatile("" : "+v"(lane));    // as in store_rows_any
    const int r16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int jj = 0; jj < FX / 2; ++jj) {
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

// The same for rows of any length and alignment: dwords that lie on their
// boundaries, 32 consecutive ones of a row to half a wave (16 where the wave has
// 32 columns), and single elements at a piece's ends where a row starts inside a
// dword.
template <int DT, int FX, int FN, int FM>
__device__ __forceinline__ void store_rows_any(uint16_t* __restrict__ C, const floatx4 (&acc)[FN][FM], uint8_t* strip,
                                               int lane, int m_base, int n_base, int m_end, int N, bool relu)
{
    constexpr int ROW = FN * 32, CHUNKS = ROW / 16, LANES = FN * 8;    // bytes and 16-byte chunks of a strip's row; dwords
    asm volatile("" : "+v"(lane));   // what follows from it is computed here, not kept through the caller's loop
    const int r16 = lane & 15, g = lane >> 4;
    auto at = [](int row, int chunk) { return row * ROW + ((chunk ^ ((row >> 1) & (CHUNKS - 1))) << 4); };
#pragma unroll
    for (int jj = 0; jj < (FX + 1) / 2; ++jj) {
#pragma unroll
        for (int jh = 0; jh < 2 && 2 * jj + jh < FX; ++jh)
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const floatx4& v = acc[i][2 * jj + jh];
                *reinterpret_cast<u32x2*>(strip + at(16 * jh + r16, 2 * i + (g >> 1)) + 8 * (g & 1)) =
                    u32x2{(uint32_t)act_cast<DT>(v[0], relu) | ((uint32_t)act_cast<DT>(v[1], relu) << 16),
                          (uint32_t)act_cast<DT>(v[2], relu) | ((uint32_t)act_cast<DT>(v[3], relu) << 16)};
            }
        const int rows = min(2 * jj + 1 < FX ? 32 : 16, m_end - (m_base + 32 * jj)), cols = min(16 * FN, N - n_base);
        for (int r = lane / LANES; r < rows; r += 64 / LANES) {
            uint16_t* const p = C + (size_t)(m_base + 32 * jj + r) * (size_t)N + n_base;
            const int odd = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1, e = 2 * (lane % LANES) + odd;
            auto element = [&](int x) { return *reinterpret_cast<const uint16_t*>(strip + at(r, x >> 3) + 2 * (x & 7)); };
            if (e + 1 < cols)
                *reinterpret_cast<uint32_t*>(p + e) = (uint32_t)element(e) | ((uint32_t)element(e + 1) << 16);
            else if (e < cols)
                p[e] = element(e);
            if (odd && e == 1 && cols > 0) p[0] = element(0);
        }
    }
}

// The product loop.  A's rows are lda long, B's ldb; `b_group` and `c_group`
// are the elements from one group's B and C to the next.  KTAIL 0: k-contiguous
// operands have k_end % 64 == 0.  1: k_end % 8 == 0.  2: rows of any even length
// at 4-byte alignment (the DMA reads 16 bytes from any dword); a piece that holds
// elements past k_end as well is cut off in LDS by the lane that loaded it, once
// it has landed and before the barrier that hands it over, so the products of
// what lies behind a row (another row's infinity) never enter a sum.
//  With adapters, kAdaptAfter adds a finished tile's low-rank terms to its sums
// (add_adapters: tiles may hold rows of many segments).  kAdaptFirst is for
// tiles cut at the segments' ends: before its K-steps over A and B a tile
// streams K-steps over the intermediates (lo, then hi) and V through the same
// ring, multiplies its sums by the rows' factors, and goes on from them, so
// the low-rank product costs its K-steps and nothing else.
enum { kAdaptNone = 0, kAdaptAfter = 1, kAdaptFirst = 2 };
template <class Cfg, int DT, int KTAIL, int ADAPT, class Units>
__device__ __forceinline__ void dma_product(const Units& units, const uint16_t* __restrict__ A,
                                            const uint16_t* __restrict__ B, uint16_t* __restrict__ C, uint32_t lda,
                                            uint32_t ldb, size_t b_group, size_t c_group, int N, bool relu, int c_vec,
                                            const AdapterArgs& ad, const uint16_t* __restrict__ mask, uint8_t* smem)
{
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, S = Cfg::STAGES;
    constexpr int QA = Cfg::QA, QB = Cfg::QB, NQ = Cfg::NQ, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int A_ROW = Cfg::A_ROW, B_ROW = Cfg::B_ROW, NKS = BK / 32;
    constexpr bool AK = Cfg::A_KMAJOR, BKM = Cfg::B_KMAJOR, WS = Cfg::PRODUCERS > 0, FIRST = ADAPT == kAdaptFirst;
    constexpr bool STAGED = Cfg::STAGED;
    static_assert(!FIRST || (KTAIL && !AK), "the rank need not be a multiple of BK");
    constexpr bool EVEN = KTAIL == 2 && !STAGED;
    static_assert(!EVEN || WS, "the producers cut the pieces off");
    static_assert(!FIRST || !STAGED, "V is streamed by DMA");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
    const bool producer = WS && wave >= Cfg::WAVES;
    const int dwave = WS ? wave - Cfg::WAVES : wave;
    const int n_units = __builtin_amdgcn_readfirstlane(units.count());
    if (n_units <= 0) return;
    // Units are the same for all lanes; readfirstlane keeps them in scalar registers.
    auto unit_at = [&](int i) {
        const DmaUnit u = units.unit(i);
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
    constexpr int PA = QA < 2 || STAGED ? QA : 2, PB = QB < 2 || STAGED ? QB : 2;
    constexpr int A_PAIR = 2048 / A_ROW, B_PAIR = 2048 / B_ROW;    // rows of two instructions
    static_assert(STAGED || QA <= 2 || (AK ? A_PAIR % 4 == 0 && 16 % (QA * A_PAIR / 2) == 0 : A_PAIR % 16 == 0), "A swizzle period");
    static_assert(STAGED || QB <= 2 || (BKM ? B_PAIR % 4 == 0 && 16 % (QB * B_PAIR / 2) == 0 : B_PAIR % 16 == 0), "B swizzle period");
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
    int f_arows = 0, f_brows = 0, f_m0 = 0, f_n0 = 0;
    int f_kb = 0, f_left_b = 0;       // B's place and what it has left, where they differ from f_k and f_left
    // With few rows a group and B stored (N, K), the tiles start their K-steps at
    // different places and wrap round: with row lengths of a power of two all rows'
    // pieces of one K-step lie in few memory channels, and tiles in step would all
    // wait for the same ones.  64 tokens over 64 experts, 2048 x 2048 bf16: 61.5
    // against 68 us.
    constexpr bool ROTATE = WS && !STAGED && !AK && !BKM && !FIRST && BM <= 64;
    int f_todo = 0;                   // K-steps still to load of the unit
    const int rank_steps = FIRST ? 2 * ad.rank_pad / BK : 0;
    auto fill_setup = [&](bool start) {
        const int live = f_unit < n_units ? 1 : 0;
        const DmaUnit u = unit_at(live ? f_unit : n_units - 1);
        const bool low = FIRST && start && live && u.adapter >= 0;
        f_rank = low ? rank_steps : 0;
        f_m0 = u.m0;
        f_n0 = u.n0;
        f_k = u.k0;
        f_left = live * (u.k_end - u.k0);
        if constexpr (ROTATE) {
            const int steps = (u.k_end + BK - 1) / BK;
            f_todo = live * steps;
            if (units.rotate) {
                f_k = (u.n0 / BN + u.group) % steps * BK;
                f_left = live * (u.k_end - f_k);
            }
        }
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
    // The descriptor of the rows from `skip` on of a stage with `rows` rows, which
    // start `col` elements into theirs (k-major; with whole pieces no lane reads
    // past the last row's end anyway).
    auto rows_from = [](const uint16_t* p, int rows, int skip, uint32_t ld, int col) {
        uint32_t bytes = (uint32_t)max(0, rows - skip) * ld * 2u;
        if constexpr (EVEN) bytes -= bytes ? 2u * (uint32_t)col : 0u;
        const int32x4_t r = rsrc_words(p + (size_t)skip * ld, bytes);
        return int32x4_t{__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]),
                         __builtin_amdgcn_readfirstlane(r[2]), kBufferFlags};
    };
    auto dma = [&](int slot, int q) {
        if (q < QA) {
            const uint32_t lds = lds_base + slot * Cfg::A_STAGE + (dwave * QA + q) * 1024;
            const uint32_t vo = a_voff[q % PA];
            if constexpr (AK)
                dma_b128(rows_from(f_ap, min(BK, f_left), q / 2 * A_PAIR, lda, f_m0), lds, vo, 0u);
            else   // (the intermediates' rows are whole K-steps)
                dma_b128(rows_from(f_ap, f_arows, q / 2 * A_PAIR, f_lda, 0), lds,
                         KTAIL && !(FIRST && f_rank) && a_pos[q % PA] >= f_left ? kOobOffset : vo, (uint32_t)f_k * 2u);
        } else {
            const int p = q - QA;
            const int left = FIRST ? f_left_b : f_left;
            const uint32_t lds = lds_base + Cfg::B_REGION + slot * Cfg::B_STAGE + (dwave * QB + p) * 1024;
            const uint32_t vo = b_voff[p % PB];
            if constexpr (BKM)
                dma_b128(rows_from(f_bp, min(BK, left), p / 2 * B_PAIR, ldb, f_n0), lds, vo, 0u);
            else
                dma_b128(rows_from(f_bp, f_brows, p / 2 * B_PAIR, f_ldb, 0), lds,
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
            // V's K-steps once for lo, once again for hi
            const int next = f_kb + BK < ad.rank_pad ? f_kb + BK : 0;
            if constexpr (BKM) f_bp += (ptrdiff_t)(next - f_kb) * (ptrdiff_t)ldb;
            f_k += BK;
            f_kb = next;
            f_left_b = ad.rank - next;
        } else if (ROTATE ? --f_todo == 0 : f_left <= BK) {
            ++f_unit;
            fill_setup(true);
        } else if (ROTATE && f_left <= BK) {
            f_left += f_k;            // round to the first k
            f_k = 0;
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

    // Loads through registers, the step's pieces as the DMA would lay them out:
    // dword-aligned 16-byte loads, with ODD also the dword after them, since a
    // piece may start 2 bytes into its first one (`shift` of the operand's
    // descriptor, and its row's number if the rows are odd: *_odd).  What lies
    // past the last k is read as it comes and zeroed on the way into LDS.  Nothing
    // is read past a matrix's last dword.  The producers set the pace here, so a
    // load costs its two address instructions and the way into LDS four shifts: with
    // predicates and shifts computed for each piece, 4000 bf16 rows of 4100 elements
    // times 4100 x 1100 took 129 us instead of 86.
    constexpr bool ODD = Cfg::ODD;
    struct Piece {
        u32x4 v;
        uint32_t next;
    };
    struct LoadSet {
        Piece a[QA], b[QB], m[Cfg::MASKED == 1 ? QA : Cfg::MASKED == 2 ? QB : 1];
        int left;
        uint32_t shift_a, shift_b, shift_m;
    };
    auto load_pieces = [&](auto& to, const uint32_t* voff, const AnyRsrc& r) __attribute__((always_inline)) {
        constexpr int Q = sizeof(to) / sizeof(Piece);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint32_t at = ODD ? (voff[q] + r.shift) & ~3u : voff[q];
            to[q].v = __builtin_amdgcn_raw_buffer_load_b128(r.rsrc, at, 0, 0);
            if constexpr (ODD) to[q].next = __builtin_amdgcn_raw_buffer_load_b32(r.rsrc, at + 16u, 0, 0);
        }
    };
    auto load_set = [&](LoadSet& set) __attribute__((always_inline)) {
        set.left = f_left;
        const uint32_t rows = (uint32_t)min(BK, f_left), past = (uint32_t)f_k * 2u;
        // up to the end of the last row: k-major operands start inside a row
        const uint32_t bytes_a = AK ? (rows ? (rows * lda - (uint32_t)f_m0) * 2u : 0u)
                                    : f_arows ? (uint32_t)f_arows * lda * 2u - past : 0u;
        const uint32_t bytes_b = BKM ? (rows ? (rows * ldb - (uint32_t)f_n0) * 2u : 0u)
                                     : f_brows ? (uint32_t)f_brows * ldb * 2u - past : 0u;
        const uint16_t *pa = AK ? f_ap : f_ap + f_k, *pb = BKM ? f_bp : f_bp + f_k;
        const AnyRsrc ra = make_any_rsrc(pa, bytes_a), rb = make_any_rsrc(pb, bytes_b);
        set.shift_a = ra.shift;
        set.shift_b = rb.shift;
        load_pieces(set.a, a_voff, ra);
        load_pieces(set.b, b_voff, rb);
        if constexpr (Cfg::MASKED != 0) {
            const AnyRsrc rm = Cfg::MASKED == 1 ? make_any_rsrc(mask + (pa - A), bytes_a) : make_any_rsrc(mask + (pb - B), bytes_b);
            set.shift_m = rm.shift;
            load_pieces(set.m, Cfg::MASKED == 1 ? a_voff : b_voff, rm);
        }
    };
    auto piece_value = [&](const Piece& p, uint32_t bits) {
        if constexpr (!ODD) return p.v;
        else return chunk_value(AnyChunk{p.v, p.next, bits});
    };
    auto take_set = [&](const LoadSet& set, int to) __attribute__((always_inline)) {
        const bool tail = set.left < BK;
        uint8_t* const at = smem + lane * 16 + to * Cfg::A_STAGE + dwave * QA * 1024;
        uint8_t* const bt = smem + lane * 16 + Cfg::B_REGION + to * Cfg::B_STAGE + dwave * QB * 1024;
#pragma unroll
        for (int q = 0; q < QA; ++q) {
            const int row = ((dwave * QA + q) * 64 + lane) * 16 / A_ROW;
            const uint32_t odd = (uint32_t)row & lda & 1u;
            u32x4 v = piece_value(set.a[q], ((set.shift_a >> 1) ^ odd) * 16u);
            if constexpr (Cfg::MASKED == 1) v = mask_chunk<DT>(v, piece_value(set.m[q], ((set.shift_m >> 1) ^ odd) * 16u));
            if (tail) v = keep_first(v, AK ? (row < set.left ? 8 : 0) : set.left - a_pos[q]);
            *reinterpret_cast<u32x4*>(at + q * 1024) = v;
        }
#pragma unroll
        for (int q = 0; q < QB; ++q) {
            const int row = ((dwave * QB + q) * 64 + lane) * 16 / B_ROW;
            const uint32_t odd = (uint32_t)row & ldb & 1u;
            u32x4 v = piece_value(set.b[q], ((set.shift_b >> 1) ^ odd) * 16u);
            if constexpr (Cfg::MASKED == 2) v = mask_chunk<DT>(v, piece_value(set.m[q], ((set.shift_m >> 1) ^ odd) * 16u));
            if (tail) v = keep_first(v, BKM ? (row < set.left ? 8 : 0) : set.left - b_pos[q]);
            *reinterpret_cast<u32x4*>(bt + q * 1024) = v;
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
    auto read_tr = [&](const uint8_t* p, int row) {
        const u32x2 lo = ds_read_tr16(p), hi = ds_read_tr16(p + 4 * row);
        return u32x4{lo.x, lo.y, hi.x, hi.y};
    };
    auto read_unit = [&](u32x4 (&fa)[2][FM], u32x4 (&fb)[2][FN], int buf, int slot, int ks, int u) {
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

    if constexpr (STAGED) {
        if (producer) {
            // Set r holds step r, then r + SETS, ...; step 0 goes to LDS before the
            // first barrier, step g + 1 while the others compute step g.
            constexpr int R = Cfg::SETS;
            LoadSet sets[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                load_set(sets[r]);
                fill_advance();
            }
            take_set(sets[0], 0);
            load_set(sets[0]);
            fill_advance();
            lds_barrier();
            // (A round has no way out between its turns, and every load is on every path:
            // else the compiler waits for all loads in flight at each turn.  Steps past
            // the last load nothing and are not stored.)
            int g = 0;
            bool live = true;
            while (live) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    LoadSet& set = sets[(r + 1) % R];
                    live = f_unit < n_units || g < f_steps;
                    ++g;
                    if (live) take_set(set, g & 1);
                    load_set(set);
                    fill_advance();
                    if (live) lds_barrier();
                }
            }
            return;
        }
    }
    constexpr int PRO = WS ? S - 1 : S;      // steps the prologue issues
    // EVEN: of the steps whose stages are in flight, what they had left.
    int lefts[PRO];
    // This wave's pieces that straddle k_end, of a stage that has landed.
    auto cut_off = [&](int slot, int left) __attribute__((always_inline)) {
        if (left >= BK || left % 8 == 0) return;
        auto cut = [&](uint8_t* at, int pos) {
            if (pos < left && left < pos + 8) {
                u32x4* const p = reinterpret_cast<u32x4*>(at + lane * 16);
                *p = keep_first(*p, left - pos);
            }
        };
        if constexpr (!AK) {
#pragma unroll
            for (int q = 0; q < QA; ++q) cut(smem + slot * Cfg::A_STAGE + (dwave * QA + q) * 1024, a_pos[q % PA]);
        }
        if constexpr (!BKM) {
#pragma unroll
            for (int q = 0; q < QB; ++q)
                cut(smem + Cfg::B_REGION + slot * Cfg::B_STAGE + (dwave * QB + q) * 1024, b_pos[q % PB]);
        }
    };
    auto push_left = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s + 1 < PRO; ++s) lefts[s] = lefts[s + 1];
        lefts[PRO - 1] = f_left;
    };
    if (!STAGED && (!WS || producer)) {
        // (One copy of the code for all stages, here and elsewhere: what does not fit
        // the instruction cache is fetched again for every tile.)
#pragma unroll 1
        for (int s = 0; s < PRO; ++s) {
            push_left();
#pragma unroll
            for (int q = 0; q < NQ; ++q) dma(s, q);
            fill_advance();
        }
        wait_vmcnt<(PRO - 1) * NQ>();
        if constexpr (EVEN) cut_off(0, lefts[0]);
    }
    lds_barrier();
    if constexpr (WS && !STAGED) {
        if (producer) {
            for (int g = 0; f_unit < n_units || g < f_steps; ++g) {
                const int slot_fill = (g + S - 1) & (S - 1);
                push_left();
#pragma unroll
                for (int q = 0; q < NQ; ++q) dma(slot_fill, q);
                fill_advance();
                wait_vmcnt<(S - 2) * NQ>();
                if constexpr (EVEN) cut_off((g + 1) & (S - 1), lefts[0]);
                lds_barrier();
            }
            wait_vmcnt<0>();   // no LDS DMA may outlive the workgroup
            return;
        }
    }
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
    // Of a tile with fewer than BM rows a wave computes what it needs of its own
    // rows: all 16-row blocks, the first half or none.  Their products are
    // skipped, and so are their fragment reads (256 rows of 8 waves: a tile of at
    // most 128 rows takes half the matrix instructions, since every SIMD has a
    // wave of each half).  Each kind has code of its own for a whole unit, from its
    // first fragments to its stores, so that nothing in registers passes from
    // one kind to another.
    constexpr bool HALVES = FM > 1 && ADAPT != kAdaptAfter;   // (rows of one group: few tiles are partial)
    int c_blocks = FM;
    auto set_blocks = [&]() {
        if constexpr (Units::RAGGED) {
            const int live = c.m_end - c.m0 - wm * Cfg::WTM;
            c_blocks = live > (HALVES ? Cfg::WTM / 2 : 0) ? FM : live > 0 ? FM / 2 : 0;
        }
    };
    set_blocks();
    auto step_barrier = [&]() {
        if constexpr (!WS) wait_vmcnt<(S - 2) * NQ>();
        lds_barrier();
    };
    // A unit with the first FX of FM blocks of rows.
    auto run = [&](auto blocks) __attribute__((always_inline)) {
        constexpr int FX = decltype(blocks)::value;
        if constexpr (FX == 0) {
            for (; c_k < c.k_end; c_k += BK) {
                step_barrier();
                if constexpr (!WS) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q) dma(slot, q);
                    fill_advance();
                }
                slot = (slot + 1) & (S - 1);
            }
            return;
        } else {
            floatx4 acc[FN][FM];
            u32x4 fb[2][FN], fa[2][FM];
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < NF; ++u)
                if (u < FX || u >= FM) read_unit(fa, fb, 0, slot, 0, u);
            while (true) {
                const int slot_next = (slot + 1) & (S - 1);
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) {
                    const int cur = ks & 1, nxt = cur ^ 1;
                    const bool last = ks == NKS - 1;
                    if (last && BAR_T == 0) step_barrier();
                    const int n_items = NF + (last ? NQC : 0);
#pragma unroll
                    for (int t = 0; t < NMF; ++t) {
                        if (last && BAR_T > 0 && t == BAR_T) step_barrier();
                        const int bi = t / FM, bj = (bi & 1) ? FM - 1 - t % FM : t % FM;
                        if (bj < FX) acc[bi][bj] = mfma_16x16x32<DT>(fb[cur][bi], fa[cur][bj], acc[bi][bj]);
                        const int t0 = last ? t - BAR_T : t, span = last ? NMF - BAR_T : NMF;
                        if (t0 < 0) {
                            __builtin_amdgcn_sched_barrier(0);
                            continue;
                        }
#pragma unroll
                        for (int u0 = t0 * n_items / span; u0 < (t0 + 1) * n_items / span; ++u0) {
                            const int u = last ? item(u0) : u0;
                            if (u < NF) {
                                if (u >= FX && u < FM) continue;
                                if (last) read_unit(fa, fb, nxt, slot_next, 0, u);
                                else read_unit(fa, fb, nxt, slot, ks + 1, u);
                            } else {
                                dma(slot, u - NF);
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (!WS && last) fill_advance();
                }
                slot = slot_next;
                c_k += BK;
                if (FIRST && 2 * c_k == -rank_steps * BK && c.adapter >= 0) {
#pragma unroll
                    for (int j = 0; j < FX; ++j)
#pragma unroll
                        for (int i = 0; i < FN; ++i) acc[i][j] = finite_low(acc[i][j]);
                }
                if (FIRST && c_k == 0 && c.adapter >= 0) {
                    int l = j16;
                    asm volatile("" : "+v"(l));
                    float f[FX];
#pragma unroll
                    for (int j = 0; j < FX; ++j) {
                        const int m = c.m0 + wm * Cfg::WTM + 16 * j + l;
                        f[j] = m < c.m_end ? ad.factor[m] : 1.0f;
                    }
#pragma unroll
                    for (int j = 0; j < FX; ++j)
#pragma unroll
                        for (int i = 0; i < FN; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][e] *= f[j];
                }
                if (c_k >= c.k_end) break;
            }
            const int m_base = c.m0 + wm * Cfg::WTM, n_base = c.n0 + wn * Cfg::WTN;
            if constexpr (ADAPT == kAdaptAfter)
                add_adapters<DT, !BKM, FX>(acc, ad, m_base, c.m_end, n_base, N, lane,
                                           smem + Cfg::LDS_BYTES + wave * Cfg::STRIP);
            uint16_t* out = C + (size_t)c.group * c_group;
            uint8_t* const strip = smem + Cfg::LDS_BYTES + wave * Cfg::STRIP;
            if (c_vec == 0) {
                store_rows_any<DT, FX>(out, acc, strip, lane, m_base, n_base, c.m_end, N, relu);
            } else if (FN % 4 == 0 && c_vec == 2) {
                if constexpr (FN % 4 == 0)
                    store_rows_staged<DT, FX>(out, acc, strip, lane, m_base, n_base, c.m_end, N, relu);
            } else {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FX; ++j)
                        store_cols<DT>(out, acc[i][j], m_base + 16 * j + j16, n_base + 16 * i + 4 * g4, c.m_end, N, relu);
            }
        }
    };
    while (true) {
        if constexpr (Units::RAGGED) {
            if (c_blocks == FM) run(std::integral_constant<int, FM>{});
            else if (HALVES && c_blocks > 0) run(std::integral_constant<int, HALVES ? FM / 2 : 0>{});
            else run(std::integral_constant<int, 0>{});
        } else {
            run(std::integral_constant<int, FM>{});
        }
        if (++c_unit >= n_units) break;
        c = unit_at(c_unit);
        set_blocks();
        c_k = c.k0 - (FIRST && c.adapter >= 0 ? rank_steps * BK : 0);
    }
    wait_vmcnt<0>();   // no LDS DMA may outlive the workgroup
}

// Rows of no group: this launch's workgroups share their zeros.
__device__ __forceinline__ void zero_rows(const RowsArgs& a, int first, int block, int blocks)
{
    const size_t n = (size_t)a.n, count = (size_t)(a.m - first) * n;
    uint16_t* p = a.c + (size_t)first * n;
    const size_t stride = (size_t)blocks * blockDim.x;
    for (size_t i = (size_t)block * blockDim.x + threadIdx.x; i < count; i += stride) p[i] = 0;
}

template <class Cfg, int DT, int KTAIL, int ADAPT, bool MANY = true>
__global__ __launch_bounds__(Cfg::THREADS, 1) void rows_dma(RowsArgs a, AdapterArgs ad)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Cfg::LDS_BYTES + Cfg::STRIP_BYTES];
    RowUnits<Cfg, MANY> units;
    if constexpr (ADAPT == kAdaptFirst) {
        units.init(a, ad.ends, ad.segments, true, threadIdx.x & 63, blockIdx.x, gridDim.x);
        units.ids = ad.ids;   // (init leaves none)
        units.adapters = ad.adapters;
    } else {
        units.init(a, a.ends, a.groups, false, threadIdx.x & 63, blockIdx.x, gridDim.x);
        if (units.rows < a.m) zero_rows(a, units.rows, blockIdx.x, gridDim.x);
    }
    dma_product<Cfg, DT, KTAIL, ADAPT>(units, a.a, a.b, a.c, (uint32_t)a.lda, (uint32_t)a.ldb,
                                       ADAPT == kAdaptFirst ? 0 : (size_t)(Cfg::B_KMAJOR ? a.k : a.n) * (size_t)a.ldb, 0, a.n,
                                       a.relu != 0, a.c_vec, ad, nullptr, smem);
}

template <class Cfg, int DT, int KTAIL>
__global__ __launch_bounds__(Cfg::THREADS, 1) void weight_dma(WeightArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Cfg::LDS_BYTES + Cfg::STRIP_BYTES];
    WeightUnits<Cfg> units;
    units.init(a, blockIdx.x, gridDim.x);
    dma_product<Cfg, DT, KTAIL, kAdaptNone>(units, a.p, a.q, a.out, (uint32_t)a.ldp, (uint32_t)a.ldq, 0,
                                       (size_t)a.i * (size_t)a.j, a.j, false, a.c_vec, AdapterArgs{}, nullptr, smem);
}

// Both gradients of a grouped product in one launch, D = dC masked on the way
// into LDS: workgroups 0 .. blocks_rows - 1 compute dA (`rows`: A is dC), the
// others dB (`weights`: p or q is dC, CfgW::MASKED says which).
template <class CfgR, class CfgW, int DT, bool MANY>
__global__ __launch_bounds__(CfgR::THREADS, 1) void grad_staged(RowsArgs rows, WeightArgs weights, const uint16_t* mask,
                                                                int blocks_rows)
{
    static_assert(CfgR::THREADS == CfgW::THREADS, "one launch");
    constexpr int LDS_R = CfgR::LDS_BYTES + CfgR::STRIP_BYTES, LDS_W = CfgW::LDS_BYTES + CfgW::STRIP_BYTES;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS_R > LDS_W ? LDS_R : LDS_W];
    const int block = (int)blockIdx.x;
    if (block < blocks_rows) {
        RowUnits<CfgR, MANY> units;
        units.init(rows, rows.ends, rows.groups, false, threadIdx.x & 63, block, blocks_rows);
        if (units.rows < rows.m) zero_rows(rows, units.rows, block, blocks_rows);
        dma_product<CfgR, DT, 1, kAdaptNone>(units, rows.a, rows.b, rows.c, (uint32_t)rows.lda, (uint32_t)rows.ldb,
                                                (size_t)(CfgR::B_KMAJOR ? rows.k : rows.n) * (size_t)rows.ldb, 0, rows.n, false, rows.c_vec, AdapterArgs{},
                                                mask, smem);
    } else {
        WeightUnits<CfgW> units;
        units.init(weights, block - blocks_rows, (int)gridDim.x - blocks_rows);
        dma_product<CfgW, DT, 0, kAdaptNone>(units, weights.p, weights.q, weights.out, (uint32_t)weights.ldp,
                                                 (uint32_t)weights.ldq, 0, (size_t)weights.i * (size_t)weights.j, weights.j,
                                                 false, weights.c_vec, AdapterArgs{}, mask, smem);
    }
}

}  // namespace gemm_relu_hip
